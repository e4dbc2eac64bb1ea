// The activation's gradient from activations that were kept in 8 bits.

#include "ag_dequantize.h"
#include "ag_linear_device.h"
#include "ag_raw.h"
#include "ag_scale.h"

namespace ag {
namespace {

// dz = dy act'(z), where z may be codes, rounded for dx; dz times the factor in [1/2, 1) of its row's x_scale, rounded for dw
// (x's codes times the scale's power of two are exact in 16 bits), with up to two more terms of what that rounding leaves;
// and the column sums of the unrounded dz over a.rows rows.  Threads and sums as in the kernel without codes.
template <bool BF16, int TERMS, bool X8, bool Z8>
__device__ __forceinline__ void slope_body(const LinearSlopeQ8Args& a, uint32_t program)
{
    __shared__ float part[8][264];
    const int c = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const uint32_t col_blocks = static_cast<uint32_t>((a.N + 255) / 256);
    const int64_t bx = program % col_blocks, by = program / col_blocks;
    const int64_t col = (bx * 32 + c) * 8;
    const int64_t row0 = by * a.rows;
    const int n = static_cast<int>(max(int64_t{0}, min(int64_t{8}, a.N - col)));
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (n > 0) {
        constexpr int DTYPE = BF16 ? AG_BF16 : AG_F16, AHEAD = 4;       // rows on their way
        const int64_t end = min(row0 + a.rows, a.M);
        const int at = static_cast<int>(col), N = static_cast<int>(a.N);
        for (int64_t first = row0 + rl; first < end; first += 8 * AHEAD) {
            Raw<DTYPE> dy[AHEAD], z16[AHEAD];
            u32x2 z8[AHEAD];
            float x_scale[AHEAD], z_scale[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {       // past the end: the last row again
                const int64_t row = min(first + 8 * j, end - 1);
                dy[j].template load<true>(a.dy + row * a.lddy, at, N);
                if constexpr (Z8) {
                    z_scale[j] = 0.f;
                    z8[j] = u32x2{0u, 0u};
                    if (a.z) {
                        z_scale[j] = a.z_scale[row];
                        z8[j] = load_codes(reinterpret_cast<const int8_t*>(a.z) + row * a.ldz + col, n);
                    }
                } else if (a.z) {
                    z16[j].template load<true>(a.z + row * a.ldz, at, N);
                }
                if constexpr (X8) x_scale[j] = a.x_scale[row];
            }
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const int64_t row = first + 8 * j;
                if (row >= end) break;
                float v[8], z[8];
                dy[j].get(v);
                if (a.z) {
                    if constexpr (Z8) {
                        code_values(z, z8[j]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) z[e] *= z_scale[j];
                    } else {
                        z16[j].get(z);
                    }
                    apply_slope(v, z, a.act);
                }
                if (a.dz) store_16<BF16>(a.dz + row * a.lddz + col, v, n);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += v[e];
                if constexpr (X8) {
                    float power, rest;
                    split_scale<BF16>(x_scale[j], &power, &rest);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= rest;
                    store_16<BF16>(a.dz_fold + row * a.lddz + col, v, n);
                }
#pragma unroll
                for (int term = 1; term < TERMS; ++term) {      // what the term before leaves
#pragma unroll
                    for (int e = 0; e < 8; ++e) {       // exact in fp32; nothing of what is not finite in 16 bits
                        const float kept = to_f32<BF16>(from_f32<BF16>(v[e]));
                        v[e] = __builtin_isfinite(kept) ? v[e] - kept : 0.f;
                    }
                    store_16<BF16>((term == 1 ? a.dz_rest : a.dz_last) + row * a.lddz + col, v, n);
                }
            }
        }
    }
    if (a.sums) {
#pragma unroll
        for (int e = 0; e < 8; ++e) part[rl][c * 8 + e] = sum[e];
        __syncthreads();
        const int64_t out = bx * 256 + threadIdx.x;
        if (out < a.N) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < 8; ++r) s += part[r][threadIdx.x];
            a.sums[by * a.N + out] = s;
        }
    }
}

// dz, and beside it x's codes as 16-bit numbers for the product that follows (x.M 0: none): two passes over memory in one launch,
// bound by it: 16384 x 3584 (z in codes) beside 16384 x 8192 bf16 132 to 138 us (814 MB, 6 TB/s), dz alone 74.
template <bool BF16, int TERMS, bool X8, bool Z8>
__global__ __launch_bounds__(256) void ag_linear_slope_q8_kernel(LinearSlopeQ8Args a, DequantizeArgs x, uint32_t slope_programs)
{
    if (blockIdx.x < slope_programs) slope_body<BF16, TERMS, X8, Z8>(a, blockIdx.x);
    else if constexpr (X8) dequantize_body<(BF16 ? AG_BF16 : AG_F16), true>(x, blockIdx.x - slope_programs, gridDim.x - slope_programs);
}

using SlopeFn = void (*)(LinearSlopeQ8Args, DequantizeArgs, uint32_t);
template <bool BF16, int TERMS> SlopeFn pick(bool x8, bool z8)
{
    return x8 ? (z8 ? ag_linear_slope_q8_kernel<BF16, TERMS, true, true> : ag_linear_slope_q8_kernel<BF16, TERMS, true, false>)
              : ag_linear_slope_q8_kernel<BF16, TERMS, false, true>;
}

}  // namespace

hipError_t launch_linear_slope_q8(const LinearSlopeQ8Args& a, const DequantizeArgs& x, int bf16, hipStream_t stream)
{
    const int64_t groups = a.rows < 1 ? 0 : (a.N + 255) / 256 * ((a.M + a.rows - 1) / a.rows);
    const bool x8 = a.x_scale != nullptr, z8 = a.z_scale != nullptr;
    const int64_t copies = x8 && x.M > 0 && x.K > 0 ? dequantize_programs(x) : 0;
    if (groups < 1 || groups + copies >= (int64_t{1} << 24) || (!x8 && !z8) || (x8 && !a.dz_fold)) return hipErrorInvalidValue;
    if (a.dz_last && (!a.dz_rest || !bf16)) return hipErrorInvalidValue;
    const SlopeFn fn = a.dz_last ? pick<true, 3>(x8, z8) : a.dz_rest ? (bf16 ? pick<true, 2>(x8, z8) : pick<false, 2>(x8, z8))
                                                                  : (bf16 ? pick<true, 1>(x8, z8) : pick<false, 1>(x8, z8));
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(groups + copies)), dim3(256), 0, stream, a, x, static_cast<uint32_t>(groups));
    return hipGetLastError();
}

}  // namespace ag
