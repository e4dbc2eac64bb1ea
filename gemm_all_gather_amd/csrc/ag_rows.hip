// Kernels that take whole rows: a row in 8 bits with its scale, the root-mean-square norm around it, and the norm's
// gradients.  All are bound by memory, one pass over their operands.

#include "ag_rows.h"
#include "ag_scale.h"
#include "ag_vec.h"

#include "ag.h"

namespace ag {
namespace {

// ---------------------------------------------------------------- rows and codes

// n <= 8 elements from p on, the others 0.
template <int DTYPE>
__device__ __forceinline__ void load_row(float (&v)[8], const void* p, int64_t at, int n)
{
    if constexpr (DTYPE == AG_F32) {
        const float* f = static_cast<const float*>(p) + at;
        if (n >= 8) {
            const f32x4u lo = *reinterpret_cast<const f32x4u*>(f), hi = *reinterpret_cast<const f32x4u*>(f + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = lo[e];
                v[4 + e] = hi[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? f[e] : 0.f;
        }
    } else {
        load_f32<DTYPE == AG_BF16>(v, static_cast<const uint16_t*>(p) + at, n);
    }
}

// A number of codes' steps to the nearest whole number, ties to even, as in exact arithmetic: v and top are exact, t = v
// (127 / top) in fp32 is off by less than 127 (2^-23 + 2^-47) = 1.6e-5, so only a t within 1e-4 of a half is decided
// in fp64, where the quotient of two numbers of up to 31 bits is a half exactly when it is one and else at least 2^-33 of itself off.
__device__ __forceinline__ float nearest_code(float v, float per, float top, bool wide)
{
    const float t = v * per, q = rintf(t);
    if (__builtin_expect(wide || fabsf(t - q) > 0.4999f, 0)) return static_cast<float>(rint(127.0 * v / top));
    return q;
}

__device__ __forceinline__ void store_codes(int8_t* p, const float (&v)[8], uint32_t top_bits, int n)
{
    const float top = __uint_as_float(top_bits);
    uint32_t lo = 0, hi = 0;
    if (top_bits != 0 && top_bits < 0x7f800000u) {      // a row of zeros, or one that is not finite, has codes of zero
        const float per = 127.f / top;
        const bool wide = top < 1e-30f;                 // 127 / top may not be finite
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = static_cast<uint32_t>(static_cast<int>(nearest_code(v[e], per, top, wide))) & 255u;
        lo = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
        hi = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
    }
    if (n >= 8) {
        reinterpret_cast<Any8*>(p)->v = u32x2{lo, hi};
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = static_cast<int8_t>((e < 4 ? lo >> (8 * e) : hi >> (8 * (e - 4))) & 255u);
    }
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }   // NaN above infinity

// A row's sum of squares and largest magnitude, over G threads; every thread gets both.  One barrier where several waves
// share a row: the LDS is used in turn (`turn`), so that a wave that is a row ahead does not write what others still read.
template <int G>
__device__ __forceinline__ void reduce_row(double& sum, uint32_t& top, double (*lds_sum)[16], uint32_t (*lds_top)[16], int turn)
{
#pragma unroll
    for (int d = 1; d < (G < 64 ? G : 64); d *= 2) {
        sum += __shfl_xor(sum, d);
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), d)));
    }
    if constexpr (G > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            lds_sum[turn][wave] = sum;
            lds_top[turn][wave] = top;
        }
        __syncthreads();
        sum = 0;
        top = 0;
#pragma unroll
        for (int w = 0; w < G / 64; ++w) {
            sum += lds_sum[turn][w];
            top = max(top, lds_top[turn][w]);
        }
    }
}

// 1 / sqrt(mean square + eps), to fp32; in fp64 where the mean leaves fp32's range.
__device__ __forceinline__ float root(double sum, int K, double eps)
{
    const double mean = sum / max(K, 1) + eps;
    if (mean > 1e-30 && mean < 1e30) return 1.f / sqrtf(static_cast<float>(mean));
    return static_cast<float>(1.0 / sqrt(mean));
}

__device__ __forceinline__ float scale_of(uint32_t top_bits, float rstd)
{
    if (top_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    return static_cast<float>(static_cast<double>(__uint_as_float(top_bits)) * rstd * (1.0 / 127.0));
}

// h: the sum rounded to its type, in fp32; what the norm is of.
template <int DTYPE>
__device__ __forceinline__ void add_residual(float (&v)[8], const RowsArgs& a, int64_t row, int col, int n)
{
    if constexpr (DTYPE != AG_F32) {
        if (a.residual) {
            float r[8];
            load_row<DTYPE>(r, a.residual, row * a.ldr + col, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = to_f32<DTYPE == AG_BF16>(from_f32<DTYPE == AG_BF16>(v[e] + r[e]));
        }
    }
}

template <int DTYPE>
__device__ __forceinline__ void store_row(void* p, int64_t at, const float (&v)[8], int n)
{
    if constexpr (DTYPE != AG_F32) store_16<DTYPE == AG_BF16>(static_cast<uint16_t*>(p) + at, v, n);
}

// Rows of up to 8 G V elements, G threads to a row, the row in registers between its two uses.
template <int DTYPE, bool NORM, int G, int V>
__global__ __launch_bounds__(G < 256 ? 256 : G) void ag_rows_kernel(RowsArgs a)
{
    constexpr int ROWS = G < 256 ? 256 / G : 1;
    __shared__ double lds_sum[2][16];
    __shared__ uint32_t lds_top[2][16];
    const int lane = threadIdx.x % G;
    float weight[V][8];
    if constexpr (NORM) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (lane + j * G) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) weight[j][e] = 1.f;
            if (a.weight) load_row<DTYPE>(weight[j], a.weight, col, a.K - col);
        }
    }
    int turn = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS; first < a.M; first += static_cast<int64_t>(gridDim.x) * ROWS) {
        const int64_t mine = first + threadIdx.x / G, row = min(mine, a.M - 1);
        const bool live = mine < a.M;
        float v[V][8];
        double sum = 0;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (lane + j * G) * 8, n = a.K - col;
            load_row<DTYPE>(v[j], a.x, row * a.ldx + col, n);
            add_residual<DTYPE>(v[j], a, row, col, n);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (lane + j * G) * 8, n = a.K - col;
            if constexpr (NORM) {
                if (a.h && live) store_row<DTYPE>(a.h, row * a.ldh + col, v[j], n);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sum = fma(static_cast<double>(v[j][e]), static_cast<double>(v[j][e]), sum);
                    v[j][e] *= weight[j][e];
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[j][e]));
        }
        reduce_row<G>(sum, top, lds_sum, lds_top, turn);
        turn ^= 1;
        float rstd = 1.f;
        if constexpr (NORM) rstd = root(sum, a.K, a.eps);
        if (live && lane == 0) {
            if (a.scale) a.scale[row] = scale_of(top, rstd);
            if (a.rstd) a.rstd[row] = rstd;
        }
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (lane + j * G) * 8, n = a.K - col;
            if (a.q) store_codes(a.q + row * a.ldq + col, v[j], top, n);
            if (a.y) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] *= rstd;
                store_row<DTYPE>(a.y, row * a.ldy + col, v[j], n);
            }
        }
    }
}

// Longer rows: a workgroup reads its row twice, the second time from the caches.
constexpr int kLongThreads = 1024;
template <int DTYPE, bool NORM>
__global__ __launch_bounds__(kLongThreads) void ag_rows_long_kernel(RowsArgs a)
{
    __shared__ double lds_sum[2][16];
    __shared__ uint32_t lds_top[2][16];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        auto weighted = [&](float (&v)[8], int col, int n) {
            if (!NORM || !a.weight) return;
            float w[8];
            load_row<DTYPE>(w, a.weight, col, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= w[e];
        };
        double sum = 0;
        uint32_t top = 0;
        for (int col = threadIdx.x * 8; col < a.K; col += kLongThreads * 8) {
            float v[8];
            const int n = a.K - col;
            load_row<DTYPE>(v, a.x, row * a.ldx + col, n);
            add_residual<DTYPE>(v, a, row, col, n);
            if constexpr (NORM) {
                if (a.h) store_row<DTYPE>(a.h, row * a.ldh + col, v, n);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fma(static_cast<double>(v[e]), static_cast<double>(v[e]), sum);
            }
            weighted(v, col, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[e]));
        }
        reduce_row<kLongThreads>(sum, top, lds_sum, lds_top, turn);
        turn ^= 1;
        float rstd = 1.f;
        if constexpr (NORM) rstd = root(sum, a.K, a.eps);
        if (threadIdx.x == 0) {
            if (a.scale) a.scale[row] = scale_of(top, rstd);
            if (a.rstd) a.rstd[row] = rstd;
        }
        if (!a.q && !a.y) continue;
        for (int col = threadIdx.x * 8; col < a.K; col += kLongThreads * 8) {
            float v[8];
            const int n = a.K - col;
            if (NORM && a.h) {      // x or the residual may be overwritten by now; a thread reads what it wrote itself
                load_row<DTYPE>(v, a.h, row * a.ldh + col, n);
            } else {
                load_row<DTYPE>(v, a.x, row * a.ldx + col, n);
                add_residual<DTYPE>(v, a, row, col, n);
            }
            weighted(v, col, n);
            if (a.q) store_codes(a.q + row * a.ldq + col, v, top, n);
            if (a.y) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= rstd;
                store_row<DTYPE>(a.y, row * a.ldy + col, v, n);
            }
        }
    }
}

// The values of codes, 16 to a thread.
template <int DTYPE>
__global__ __launch_bounds__(256) void ag_dequantize_kernel(DequantizeArgs a)
{
    const int64_t per_row = (a.K + 15) / 16, id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t row = id / per_row;
    const int col = static_cast<int>(id - row * per_row) * 16;
    if (row >= a.M) return;
    float s = a.scale[row];
    if (a.by_power) {
        float rest;
        split_scale<DTYPE == AG_BF16>(s, &s, &rest);
    }
    const int8_t* q = a.q + row * a.ldq + col;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int n = a.K - col - 8 * half;
        if (n <= 0) break;
        float v[8];
        load_codes(v, q + 8 * half, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= s;
        const int64_t at = row * a.ldy + col + 8 * half;
        if constexpr (DTYPE == AG_F32) {
            float* p = static_cast<float*>(a.y) + at;
            if (n >= 8) {
                *reinterpret_cast<f32x4u*>(p) = f32x4u{v[0], v[1], v[2], v[3]};
                *reinterpret_cast<f32x4u*>(p + 4) = f32x4u{v[4], v[5], v[6], v[7]};
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < n) p[e] = v[e];
            }
        } else {
            store_row<DTYPE>(a.y, at, v, n);
        }
    }
}

// ---------------------------------------------------------------- the norm's gradients

// One row's sum over G threads; every thread gets it.
template <int G>
__device__ __forceinline__ float sum_row(float s, float (*lds)[16], int turn)
{
#pragma unroll
    for (int d = 1; d < (G < 64 ? G : 64); d *= 2) s += __shfl_xor(s, d);
    if constexpr (G > 64) {
        if ((threadIdx.x & 63) == 0) lds[turn][threadIdx.x >> 6] = s;
        __syncthreads();
        s = 0.f;
#pragma unroll
        for (int w = 0; w < G / 64; ++w) s += lds[turn][w];
    }
    return s;
}

// With n = h rstd and c = mean(g n): dx = rstd (g - n c) + dh, and dy n for dw, which a workgroup sums over its rows in
// registers (its waves' sums joined through LDS where they take rows of their own).
template <bool BF16, int G, int V>
__global__ __launch_bounds__(G < 256 ? 256 : G) void ag_norm_backward_kernel(NormBackwardArgs a)
{
    constexpr int ROWS = G < 256 ? 256 / G : 1;
    __shared__ float lds[2][16];
    __shared__ float join[ROWS > 1 ? ROWS * G * 8 : 1];
    const int lane = threadIdx.x % G;
    float weight[V][8], dw[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int col = (lane + j * G) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            weight[j][e] = 1.f;
            dw[j][e] = 0.f;
        }
        if (a.weight) load_f32<BF16>(weight[j], a.weight + col, a.K - col);
    }
    const float per_k = 1.f / max(a.K, 1);
    int turn = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS; first < a.M; first += static_cast<int64_t>(gridDim.x) * ROWS) {
        const int64_t mine = first + threadIdx.x / G, row = min(mine, a.M - 1);
        const bool live = mine < a.M;
        const float rstd = a.rstd[row];
        float dy[V][8], n[V][8], dh[V][8];
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (lane + j * G) * 8;
            load_f32<BF16>(dy[j], a.dy + row * a.lddy + col, a.K - col);
            load_f32<BF16>(n[j], a.h + row * a.ldh + col, a.K - col);
            if (a.dh && a.dx) load_f32<BF16>(dh[j], a.dh + row * a.lddh + col, a.K - col);
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                n[j][e] *= rstd;
                if (live) dw[j][e] += dy[j][e] * n[j][e];
                dy[j][e] *= weight[j][e];
                s += dy[j][e] * n[j][e];
            }
        if (!a.dx) continue;
        const float c = sum_row<G>(s, lds, turn) * per_k;
        turn ^= 1;
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (lane + j * G) * 8;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = rstd * (dy[j][e] - n[j][e] * c) + (a.dh ? dh[j][e] : 0.f);
            store_16<BF16>(a.dx + row * a.lddx + col, v, a.K - col);
        }
    }
    if (!a.sums) return;
    float* out = a.sums + static_cast<int64_t>(blockIdx.x) * a.K;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if constexpr (ROWS > 1) {
            if (j > 0) __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) join[(threadIdx.x / G) * (G * 8) + lane * 8 + e] = dw[j][e];
            __syncthreads();
            for (int c = threadIdx.x; c < G * 8; c += 256) {
                const int col = j * G * 8 + c;
                float t = 0.f;
#pragma unroll
                for (int r = 0; r < ROWS; ++r) t += join[r * (G * 8) + c];
                if (col < a.K) out[col] = t;
            }
        } else {
            const int col = (lane + j * G) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (col + e < a.K) out[col + e] = dw[j][e];
        }
    }
}

// Longer rows: read twice, and the sums of dw kept in the workgroup's row of `sums`.
template <bool BF16>
__global__ __launch_bounds__(kLongThreads) void ag_norm_backward_long_kernel(NormBackwardArgs a)
{
    __shared__ float lds[2][16];
    const float per_k = 1.f / a.K;
    float* out = a.sums ? a.sums + static_cast<int64_t>(blockIdx.x) * a.K : nullptr;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const float rstd = a.rstd[row];
        float s = 0.f;
        for (int col = threadIdx.x * 8; col < a.K; col += kLongThreads * 8) {
            const int left = a.K - col;
            float dy[8], n[8], w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
            load_f32<BF16>(dy, a.dy + row * a.lddy + col, left);
            load_f32<BF16>(n, a.h + row * a.ldh + col, left);
            if (a.weight) load_f32<BF16>(w, a.weight + col, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                n[e] *= rstd;
                s += dy[e] * w[e] * n[e];
                if (out && e < left) out[col + e] = (row == blockIdx.x ? 0.f : out[col + e]) + dy[e] * n[e];
            }
        }
        if (!a.dx) continue;
        const float c = sum_row<kLongThreads>(s, lds, turn) * per_k;
        turn ^= 1;
        for (int col = threadIdx.x * 8; col < a.K; col += kLongThreads * 8) {
            const int left = a.K - col;
            float dy[8], n[8], w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}, dh[8] = {};
            load_f32<BF16>(dy, a.dy + row * a.lddy + col, left);
            load_f32<BF16>(n, a.h + row * a.ldh + col, left);
            if (a.weight) load_f32<BF16>(w, a.weight + col, left);
            if (a.dh) load_f32<BF16>(dh, a.dh + row * a.lddh + col, left);
#pragma unroll
            for (int e = 0; e < 8; ++e) dy[e] = rstd * (dy[e] * w[e] - n[e] * rstd * c) + dh[e];
            store_16<BF16>(a.dx + row * a.lddx + col, dy, left);
        }
    }
}

// ---------------------------------------------------------------- choice of a kernel

using RowsFn = void (*)(RowsArgs);
template <int DTYPE, bool NORM> RowsFn pick_rows(const RowsShape& s)
{
    switch (s.threads * 8 + s.vectors) {
    case 16 * 8 + 1: return ag_rows_kernel<DTYPE, NORM, 16, 1>;
    case 64 * 8 + 1: return ag_rows_kernel<DTYPE, NORM, 64, 1>;
    case 64 * 8 + 2: return ag_rows_kernel<DTYPE, NORM, 64, 2>;
    case 256 * 8 + 1: return ag_rows_kernel<DTYPE, NORM, 256, 1>;
    case 256 * 8 + 2: return ag_rows_kernel<DTYPE, NORM, 256, 2>;
    case 256 * 8 + 4: return ag_rows_kernel<DTYPE, NORM, 256, 4>;
    case 1024 * 8 + 2: return ag_rows_kernel<DTYPE, NORM, 1024, 2>;
    case 1024 * 8 + 4: return ag_rows_kernel<DTYPE, NORM, 1024, 4>;
    case kLongThreads * 8: return ag_rows_long_kernel<DTYPE, NORM>;
    default: return nullptr;
    }
}

using NormBackwardFn = void (*)(NormBackwardArgs);
template <bool BF16> NormBackwardFn pick_backward(const RowsShape& s)
{
    switch (s.threads * 8 + s.vectors) {
    case 16 * 8 + 1: return ag_norm_backward_kernel<BF16, 16, 1>;
    case 64 * 8 + 1: return ag_norm_backward_kernel<BF16, 64, 1>;
    case 64 * 8 + 2: return ag_norm_backward_kernel<BF16, 64, 2>;
    case 256 * 8 + 1: return ag_norm_backward_kernel<BF16, 256, 1>;
    case 256 * 8 + 2: return ag_norm_backward_kernel<BF16, 256, 2>;
    case 256 * 8 + 4: return ag_norm_backward_kernel<BF16, 256, 4>;
    case 1024 * 8 + 2: return ag_norm_backward_kernel<BF16, 1024, 2>;
    case 1024 * 8 + 4: return ag_norm_backward_kernel<BF16, 1024, 4>;
    case kLongThreads * 8: return ag_norm_backward_long_kernel<BF16>;
    default: return nullptr;
    }
}

}  // namespace

// ---------------------------------------------------------------- launchers

RowsShape rows_shape(int64_t K)
{
    if (K <= 128) return {16, 1, 16};
    if (K <= 512) return {64, 1, 4};
    if (K <= 1024) return {64, 2, 4};
    if (K <= 2048) return {256, 1, 1};
    if (K <= 4096) return {256, 2, 1};
    if (K <= 8192) return {256, 4, 1};
    if (K <= 16384) return {1024, 2, 1};
    if (K <= 32768) return {1024, 4, 1};
    return {kLongThreads, 0, 1};
}

hipError_t launch_rows(const RowsArgs& a, int dtype, bool norm, int programs, hipStream_t stream)
{
    const RowsShape s = rows_shape(a.K);
    const RowsFn fn = norm ? (dtype == AG_BF16 ? pick_rows<AG_BF16, true>(s) : dtype == AG_F16 ? pick_rows<AG_F16, true>(s) : nullptr)
                           : (dtype == AG_BF16 ? pick_rows<AG_BF16, false>(s) : dtype == AG_F16 ? pick_rows<AG_F16, false>(s)
                                                                                                : pick_rows<AG_F32, false>(s));
    if (fn == nullptr || programs < 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(programs)), dim3(static_cast<uint32_t>(s.threads * s.per_group)), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_dequantize(const DequantizeArgs& a, int dtype, hipStream_t stream)
{
    const int64_t groups = (a.M * ((a.K + 15) / 16) + 255) / 256;
    if (groups < 1 || groups > 0x7fffffff) return hipErrorInvalidValue;
    auto fn = dtype == AG_BF16 ? ag_dequantize_kernel<AG_BF16> : dtype == AG_F16 ? ag_dequantize_kernel<AG_F16> : ag_dequantize_kernel<AG_F32>;
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(groups)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_norm_backward(const NormBackwardArgs& a, int bf16, int programs, hipStream_t stream)
{
    const RowsShape s = rows_shape(a.K);
    const NormBackwardFn fn = bf16 ? pick_backward<true>(s) : pick_backward<false>(s);
    if (fn == nullptr || programs < 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(programs)), dim3(static_cast<uint32_t>(s.threads * s.per_group)), 0, stream, a);
    return hipGetLastError();
}

}  // namespace ag
