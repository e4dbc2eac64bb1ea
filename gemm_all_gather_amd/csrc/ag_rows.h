// Internal interface between the host code of the row operators (ag_rows_host.cpp: codes of 8 bits, the
// root-mean-square norm and its gradients) and their kernels (ag_rows.hip).  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ag {

// A grid's workgroups: with up to 1024 threads each, a launch's threads stay below 2^32.
constexpr int64_t kMaxRowsPrograms = (int64_t{1} << 22) - 1;

// One pass over rows: h = x + residual, its norm, and the row in 16 or 8 bits; without `norm` the row itself in 8 bits.
struct RowsArgs {
    const void* x;
    const void* residual;   // or null
    const void* weight;     // or null
    void* h;                // or null
    void* y;                // or null
    int8_t* q;              // or null
    float* scale;           // with q
    float* rstd;            // or null
    int64_t ldx, ldr, ldh, ldy, ldq;
    int64_t M;
    int32_t K;
    int32_t reserved;
    double eps;
};

// How a row is dealt to threads: `threads` of a workgroup with `vectors` of 8 elements each in registers; vectors 0:
// longer rows, read twice by `threads`.
struct RowsShape {
    int threads, vectors;
    int per_group;          // rows of a workgroup at a time
};
RowsShape rows_shape(int64_t K, bool norm);
RowsShape norm_backward_shape(int64_t K);       // vectors 0: in two passes, launch_norm_backward_long

// norm with dtype AG_F16 or AG_BF16; without it AG_F32 too.
hipError_t launch_rows(const RowsArgs& a, int dtype, bool norm, int programs, hipStream_t stream);

// y = q * scale in dtype; beside the gradients that read it, q * (the scale's power of two) in their 16-bit type, exactly.
struct DequantizeArgs {
    const int8_t* q;
    const float* scale;
    void* y;
    int64_t ldq, ldy;
    int64_t M;
    int32_t K;
    int32_t more = 0;       // further copies of all M rows, one below the other (beside the gradients only)
};
constexpr int kDequantizeVectors = 4;
inline int64_t dequantize_programs(const DequantizeArgs& a)      // workgroups of 256 threads
{
    const int64_t vectors = a.M * ((a.K + 7) / 8), per = 256 * kDequantizeVectors, groups = (vectors + per - 1) / per;
    return groups < kMaxRowsPrograms ? groups : kMaxRowsPrograms;
}
hipError_t launch_dequantize(const DequantizeArgs& a, int dtype, hipStream_t stream);

struct NormBackwardArgs {
    const uint16_t* dy;
    const uint16_t* h;
    const uint16_t* dh;         // or null
    const uint16_t* weight;     // or null
    const float* rstd;
    uint16_t* dx;               // or null; may be dh
    float* sums;                // one row of floats for each workgroup, or null
    float* means;               // M floats, of the two passes over longer rows
    int64_t ldsums;             // a multiple of 32
    int64_t lddy, ldh, lddh, lddx;
    int64_t M;
    int32_t K;
    int32_t reserved;
};
// dw (+)= the sum of `parts` rows of sums.
struct NormDwArgs {
    const float* sums;
    void* dw;
    int64_t ldsums;
    int32_t parts;
    int32_t K;
    int32_t dtype;              // ag_dtype_t of dw
    int32_t accumulate;
};
hipError_t launch_norm_dw(const NormDwArgs& a, hipStream_t stream);
// Both gradients of little work in one launch (rows of up to 4096; no sums).
hipError_t launch_norm_backward_small(const NormBackwardArgs& a, const NormDwArgs& d, int bf16, int dx_programs, hipStream_t stream);
hipError_t launch_norm_backward(const NormBackwardArgs& a, int bf16, int programs, hipStream_t stream);
// Longer rows: `batches` of `rows` rows each, and as many rows of sums.
hipError_t launch_norm_backward_long(const NormBackwardArgs& a, int bf16, int batches, int rows, hipStream_t stream);

}  // namespace ag
