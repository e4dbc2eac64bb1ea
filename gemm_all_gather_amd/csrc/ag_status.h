// Status and error-message helpers of the C ABI's entry points (defined in ag_host.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include "ag.h"

namespace ag {

// Clears the calling thread's error message and returns AG_OK.
ag_status_t ok();
// Sets the calling thread's error message and returns s.
ag_status_t fail(ag_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
ag_status_t fail_hip(hipError_t e, const char* what);

}  // namespace ag
