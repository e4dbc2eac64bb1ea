// The activation's gradient from activations that were kept in 8 bits.

#include <algorithm>

#include "ag_dequantize.h"
#include "ag_linear_device.h"
#include "ag_raw.h"
#include "ag_scale.h"

namespace ag {
namespace {

// v in further terms: what the one before leaves, rounded.
template <bool BF16>
__device__ __forceinline__ void next_term(float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {       // exact in fp32; nothing of what is not finite in 16 bits
        const float kept = to_f32<BF16>(from_f32<BF16>(v[e]));
        v[e] = __builtin_isfinite(kept) ? v[e] - kept : 0.f;
    }
}

// dz = dy act'(z), where z may be codes, rounded for dx; X8 (bf16): dz times the rest of its row's x_scale, rounded for dw (x's codes
// times the scale's power of two are exact in 16 bits), with up to two more terms of what that rounding leaves;
// and the column sums of the unrounded dz over a.rows rows.  Threads and sums as in the kernel without codes.
template <bool BF16, int TERMS, bool X8, bool Z8>
__device__ __forceinline__ void slope_body(const LinearSlopeQ8Args& a, uint32_t program)
{
    static_assert(BF16 || !X8, "fp16 folds whole rows");
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
                    split_scale_bf16(x_scale[j], &power, &rest);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= rest;
                    store_16<BF16>(a.dz_fold + row * a.lddz + col, v, n);
                }
#pragma unroll
                for (int term = 1; term < TERMS; ++term) {      // what the term before leaves
                    next_term<BF16>(v);
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
    else if constexpr (X8) dequantize_body<AG_BF16, true>(x, blockIdx.x - slope_programs, gridDim.x - slope_programs);
}

// How fp16's rows are dealt out: `threads` to a row, and `span` of its columns, of dz and of x alike, to a workgroup.
struct FoldShape {
    int64_t items, chunks;      // items: groups of 256 / threads rows times chunks of columns
    int32_t threads, span;
};

// dz times the rest of its row's x_scale, rounded, its second term, and x's codes times the scale's power of two.  Which power that
// is takes the row's largest |dy| (split_scale_f16), so a row's threads read all of dy's row first, and their columns again from the
// caches.  What is not finite in dy is left out of that: it reaches its own elements of dz, and the others keep their bits.
template <int TERMS, bool Z8, int G>
__device__ __forceinline__ void fold_rows(const LinearSlopeQ8Args& a, const DequantizeArgs& x, const FoldShape& f, uint32_t program, uint32_t programs)
{
    constexpr int ROWS = 256 / G, DZ_AHEAD = 2, CODES_AHEAD = 4;
    __shared__ uint32_t tops[2][4];
    const int lane = threadIdx.x % G, N = static_cast<int>(a.N);
    int turn = 0;
    for (int64_t item = program; item < f.items; item += programs) {
        const int64_t group = item / f.chunks, mine = group * ROWS + (ROWS > 1 ? threadIdx.x / G : 0), row = min(mine, a.M - 1);
        const int from = static_cast<int>(item - group * f.chunks) * f.span;
        const bool live = mine < a.M;
        const uint16_t* dys = a.dy + row * a.lddy;
        const float x_scale = a.x_scale[row];
        float z_scale = 0.f;
        if constexpr (Z8) z_scale = a.z_scale[row];
        uint32_t top = 0;
        for (int col = lane * 8; col < N; col += G * 8 * DZ_AHEAD) {
            Raw<AG_F16> dy[DZ_AHEAD];
#pragma unroll
            for (int j = 0; j < DZ_AHEAD; ++j) dy[j].template load<true>(dys, col + j * G * 8, N);      // past the end: zeros
#pragma unroll
            for (int j = 0; j < DZ_AHEAD; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t m = dy[j].v[e >> 1] >> (16 * (e & 1)) & 0x7fffu;
                    top = max(top, m < 0x7c00u ? m : 0u);
                }
        }
#pragma unroll
        for (int d = 1; d < (G < 64 ? G : 64); d *= 2) top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
        if constexpr (G > 64) {     // used in turn: a wave that is an item ahead does not write what others still read
            if ((threadIdx.x & 63) == 0) tops[turn][threadIdx.x >> 6] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < G / 64; ++w) top = max(top, tops[turn][w]);
            turn ^= 1;
        }
        if (!live) continue;
        float power, rest;
        split_scale_f16(x_scale, to_f32<false>(static_cast<uint16_t>(top)), &power, &rest);
        for (int col = from + lane * 8; col < min(from + f.span, N); col += G * 8 * DZ_AHEAD) {
            Raw<AG_F16> dy[DZ_AHEAD], z16[DZ_AHEAD];
            u32x2 z8[DZ_AHEAD];
#pragma unroll
            for (int j = 0; j < DZ_AHEAD; ++j) {
                const int at = col + j * G * 8, end = at < from + f.span ? N : 0;
                dy[j].template load<true>(dys, at, end);
                if constexpr (Z8) {
                    z8[j] = u32x2{0u, 0u};
                    if (at < end) z8[j] = load_codes(reinterpret_cast<const int8_t*>(a.z) + row * a.ldz + at, end - at);
                } else if (a.z) {
                    z16[j].template load<true>(a.z + row * a.ldz, at, end);
                }
            }
#pragma unroll
            for (int j = 0; j < DZ_AHEAD; ++j) {
                const int at = col + j * G * 8, n = N - at;
                if (n <= 0 || at >= from + f.span) break;
                float v[8], z[8];
                dy[j].get(v);
                if (a.z) {
                    if constexpr (Z8) {
                        code_values(z, z8[j]);
#pragma unroll
                        for (int e = 0; e < 8; ++e) z[e] *= z_scale;
                    } else {
                        z16[j].get(z);
                    }
                    apply_slope(v, z, a.act);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= rest;
                store_16<false>(a.dz_fold + row * a.lddz + at, v, n);
                if constexpr (TERMS > 1) {
                    next_term<false>(v);
                    store_16<false>(a.dz_rest + row * a.lddz + at, v, n);
                }
            }
        }
        for (int col = from + lane * 8; col < min(from + f.span, x.K); col += G * 8 * CODES_AHEAD) {
            u32x2 q[CODES_AHEAD];
#pragma unroll
            for (int j = 0; j < CODES_AHEAD; ++j) {
                const int at = col + j * G * 8, end = at < from + f.span ? x.K : 0;
                q[j] = u32x2{0u, 0u};
                if (at < end) q[j] = load_codes(x.q + row * x.ldq + at, end - at);
            }
#pragma unroll
            for (int j = 0; j < CODES_AHEAD; ++j) {
                const int at = col + j * G * 8, n = x.K - at;
                if (n <= 0 || at >= from + f.span) break;
                float v[8];
                code_values(v, q[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= power;
                for (int c = 0; c <= x.more; ++c) store_16<false>(static_cast<uint16_t*>(x.y) + (row + c * x.M) * x.ldy + at, v, n);
            }
        }
    }
}

// dz for dx and db's sums (slope_programs 0: neither), and beside them the rows for dw, which work dz out again.  Bound by memory, with dy
// and z read twice (16384 x 3584, z in codes, beside 16384 x 8192 187 to 196 us, 1000 x 4100 beside 1000 x 4100 17.6), where a power from the
// scale alone needs one pass (135, 12) but loses small gradients: all gradients of 16384 x 3584 x 8192 1621 us for 1578, of 1000 x 4100 x
// 4100 117 for 113, of 16384 x 512 x 1024 100 for 89.
template <int TERMS, bool Z8, int G>
__global__ __launch_bounds__(256) void ag_linear_fold_f16_kernel(LinearSlopeQ8Args a, DequantizeArgs x, FoldShape f, uint32_t slope_programs)
{
    if (blockIdx.x < slope_programs) slope_body<false, 1, false, Z8>(a, blockIdx.x);
    else fold_rows<TERMS, Z8, G>(a, x, f, blockIdx.x - slope_programs, gridDim.x - slope_programs);
}

using SlopeFn = void (*)(LinearSlopeQ8Args, DequantizeArgs, uint32_t);
template <int TERMS> SlopeFn pick_x8_bf16(bool z8)
{
    return z8 ? ag_linear_slope_q8_kernel<true, TERMS, true, true> : ag_linear_slope_q8_kernel<true, TERMS, true, false>;
}
SlopeFn pick_z8(int bf16, bool two)
{
    return two ? (bf16 ? ag_linear_slope_q8_kernel<true, 2, false, true> : ag_linear_slope_q8_kernel<false, 2, false, true>)
               : (bf16 ? ag_linear_slope_q8_kernel<true, 1, false, true> : ag_linear_slope_q8_kernel<false, 1, false, true>);
}

using FoldFn = void (*)(LinearSlopeQ8Args, DequantizeArgs, FoldShape, uint32_t);
template <int TERMS, bool Z8> FoldFn pick_fold(int threads)
{
    return threads == 16 ? ag_linear_fold_f16_kernel<TERMS, Z8, 16> : threads == 64 ? ag_linear_fold_f16_kernel<TERMS, Z8, 64>
                                                                                    : ag_linear_fold_f16_kernel<TERMS, Z8, 256>;
}

constexpr int64_t kMaxGroups = int64_t{1} << 24;        // of 256 threads: fewer than 2^32 in a launch

// Rows of up to 256 elements 16 threads each, up to 2048 a wave, longer ones a workgroup, as the norm's.  Below 1024 workgroups a row's
// columns are dealt to several.
FoldShape fold_shape(int64_t M, int64_t N, int64_t K)
{
    const int64_t width = std::max(N, K), threads = width <= 256 ? 16 : width <= 2048 ? 64 : 256, step = threads * 8;
    const int64_t groups = (M + 256 / threads - 1) / (256 / threads);
    const int64_t most = std::max<int64_t>(1, std::min((width + step - 1) / step, 1024 / groups));
    const int64_t span = ((width + most - 1) / most + step - 1) / step * step, chunks = (width + span - 1) / span;
    return {groups * chunks, chunks, static_cast<int32_t>(threads), static_cast<int32_t>(span)};
}

hipError_t launch_fold_f16(const LinearSlopeQ8Args& a, const DequantizeArgs& x, int64_t slope_groups, hipStream_t stream)
{
    if (!a.dz && !a.sums) slope_groups = 0;
    if (x.M != a.M || x.K < 1 || !a.dz_fold || a.dz_last) return hipErrorInvalidValue;
    const FoldShape f = fold_shape(a.M, a.N, x.K);
    const int64_t grid = slope_groups + std::min(f.items, int64_t{1} << 22);
    if (grid >= kMaxGroups) return hipErrorInvalidValue;
    const FoldFn fn = a.z_scale ? (a.dz_rest ? pick_fold<2, true>(f.threads) : pick_fold<1, true>(f.threads))
                                : (a.dz_rest ? pick_fold<2, false>(f.threads) : pick_fold<1, false>(f.threads));
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(grid)), dim3(256), 0, stream, a, x, f, static_cast<uint32_t>(slope_groups));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_slope_q8(const LinearSlopeQ8Args& a, const DequantizeArgs& x, int bf16, hipStream_t stream)
{
    const int64_t groups = a.rows < 1 ? 0 : (a.N + 255) / 256 * ((a.M + a.rows - 1) / a.rows);
    const bool x8 = a.x_scale != nullptr, z8 = a.z_scale != nullptr;
    if (groups < 1 || (!x8 && !z8) || (x8 && !a.dz_fold)) return hipErrorInvalidValue;
    if (x8 && !bf16) return launch_fold_f16(a, x, groups, stream);
    const int64_t copies = x8 && x.M > 0 && x.K > 0 ? dequantize_programs(x) : 0;
    if (groups + copies >= kMaxGroups || (x8 && (a.dz_rest != nullptr) != (a.dz_last != nullptr))) return hipErrorInvalidValue;
    const SlopeFn fn = !x8 ? pick_z8(bf16, a.dz_rest != nullptr) : a.dz_last ? pick_x8_bf16<3>(z8) : pick_x8_bf16<1>(z8);
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(groups + copies)), dim3(256), 0, stream, a, x, static_cast<uint32_t>(groups));
    return hipGetLastError();
}

}  // namespace ag
