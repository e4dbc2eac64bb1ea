// A kept row's scale s in two factors: a power of two that goes to the codes, whose products with it are exact in 16 bits,
// and the rest, in [1/2, 1) for every scale between the powers' limits, so that a gradient times it does not overflow.
#pragma once

#include <hip/hip_runtime.h>

namespace ag {
namespace {

// fp16: codes up to 128 times 2^8 stay below 65504, and 2^-24 is its smallest number (from scales of 256 on, rows that hold
// 32512 or more, the rest is 1 or more).  bf16 has fp32's exponents: 128 times 2^119 is finite, and codes times 2^-126 are normal.
template <bool BF16>
__device__ __forceinline__ void split_scale(float s, float* power, float* rest)
{
    const int e = static_cast<int>((__float_as_uint(s) >> 23) & 255u) - 126;     // s < 2^e; 129 of a NaN or an infinity
    const int a = BF16 ? min(max(e, -126), 119) : min(max(e, -24), 8);
    *power = __uint_as_float(static_cast<uint32_t>(a + 127) << 23);
    *rest = ldexpf(s, -a);
}

}  // namespace
}  // namespace ag
