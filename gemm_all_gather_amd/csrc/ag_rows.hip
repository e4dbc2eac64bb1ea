// Kernels that take whole rows: a row in 8 bits with its scale, the root-mean-square norm around it, and the norm's
// gradients.  All are bound by memory, one pass over their operands.

#include <algorithm>

#include "ag_rows.h"
#include "ag_dequantize.h"
#include "ag_raw.h"
#include "ag_vec.h"

#include "ag.h"

namespace ag {
namespace {

// ---------------------------------------------------------------- rows and codes

// A number of codes' steps to the nearest whole number, ties to even, as in exact arithmetic: v and top are exact, t = v
// (127 / top) in fp32 is off by less than 127 (2^-23 + 2^-47) = 1.6e-5, so only a t within 1e-4 of a half is decided
// in fp64, where the quotient of two numbers of up to 31 bits is a half exactly when it is one and else at least 2^-33 of itself off.
__device__ __forceinline__ float nearest_code(float v, float per, float top, bool wide)
{
    const float t = v * per, q = rintf(t);
    if (__builtin_expect(wide || fabsf(t - q) > 0.4999f, 0)) return static_cast<float>(rint(127.0 * v / top));
    return q;
}

// What a row's codes are made with: 127 over its largest magnitude.
struct Unit {
    float top, per;
    bool none, wide;        // no codes but 0; 127 / top may not be finite
    __device__ __forceinline__ explicit Unit(uint32_t top_bits)
    {
        top = __uint_as_float(top_bits);
        none = top_bits == 0 || top_bits >= 0x7f800000u;        // a row of zeros, or one that is not finite
        per = none ? 0.f : 127.f / top;
        wide = top < 1e-30f;
    }
    __device__ __forceinline__ uint32_t code(float v) const      // in 8 bits
    {
        return none ? 0u : static_cast<uint32_t>(static_cast<int>(nearest_code(v, per, top, wide))) & 255u;
    }
};

__device__ __forceinline__ void store_codes(int8_t* p, const float (&v)[8], const Unit& unit, int n)
{
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = unit.code(v[e]);
    if (n >= 8) {
        reinterpret_cast<Any8*>(p)->v = u32x2{c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24};
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = static_cast<int8_t>(c[e]);
    }
}

// One element, for the up to seven behind a row's last whole vector.
template <int DTYPE> __device__ __forceinline__ float element(const void* row, int col)
{
    if constexpr (DTYPE == AG_F32) return static_cast<const float*>(row)[col];
    else return to_f32<DTYPE == AG_BF16>(static_cast<const uint16_t*>(row)[col]);
}
template <int DTYPE> __device__ __forceinline__ void put_element(void* p, int64_t at, float v)
{
    if constexpr (DTYPE == AG_F32) static_cast<float*>(p)[at] = v;
    else static_cast<uint16_t*>(p)[at] = from_f32<DTYPE == AG_BF16>(v);
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }   // NaN above infinity

// x combined with all lanes' of each group of G <= 64, in every lane: rotations within rows of 16 lanes, then swaps of rows and
// of halves, none of which goes through LDS.
template <int D> __device__ __forceinline__ uint32_t rotated(uint32_t x)      // within 16 lanes, by D
{
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x120 + D, 0xf, 0xf, true));
}
template <int D, class T> __device__ __forceinline__ T rotated_as(T x)
{
    if constexpr (sizeof(T) == 8) {
        u32x2 w = __builtin_bit_cast(u32x2, x);
        w.x = rotated<D>(w.x);
        w.y = rotated<D>(w.y);
        return __builtin_bit_cast(T, w);
    } else {
        return __builtin_bit_cast(T, rotated<D>(__builtin_bit_cast(uint32_t, x)));
    }
}
// Both rows of a pair (SIZE 16), both halves (32): each lane gets its own side's and the other side's, in the lanes' order.
template <int SIZE> __device__ __forceinline__ u32x2 swapped(uint32_t x)
{
    if constexpr (SIZE == 16) return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(x, x, false, false));
    else return __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(x, x, false, false));
}
template <int SIZE, class T, class F> __device__ __forceinline__ T across(T x, F f)
{
    if constexpr (sizeof(T) == 8) {
        const u32x2 w = __builtin_bit_cast(u32x2, x), lo = swapped<SIZE>(w.x), hi = swapped<SIZE>(w.y);
        return f(__builtin_bit_cast(T, u32x2{lo.x, hi.x}), __builtin_bit_cast(T, u32x2{lo.y, hi.y}));
    } else {
        const u32x2 w = swapped<SIZE>(__builtin_bit_cast(uint32_t, x));
        const uint32_t one = w.x, other = w.y;      // a bit cast of a vector's element takes its first one
        return f(__builtin_bit_cast(T, one), __builtin_bit_cast(T, other));
    }
}
template <int G, class T, class F> __device__ __forceinline__ T combine(T x, F f)
{
    static_assert(G == 16 || G == 64, "whole rows or whole waves");
    x = f(x, rotated_as<8>(x));
    x = f(x, rotated_as<4>(x));
    x = f(x, rotated_as<2>(x));
    x = f(x, rotated_as<1>(x));
    if constexpr (G == 64) {
        x = across<16>(x, f);
        x = across<32>(x, f);
    }
    return x;
}

// A row's sum of squares (of a norm) and largest magnitude, over G threads; every thread gets both.  One barrier where several
// waves share a row: the LDS is used in turn (`turn`), so that a wave that is a row ahead does not write what others still read.
template <bool NORM, int G>
__device__ __forceinline__ void reduce_row(double& sum, uint32_t& top, double (*lds_sum)[16], uint32_t (*lds_top)[16], int turn)
{
    constexpr int LANES = G < 64 ? G : 64;
    if constexpr (NORM) sum = combine<LANES>(sum, [](double x, double y) { return x + y; });
    top = combine<LANES>(top, [](uint32_t x, uint32_t y) { return max(x, y); });
    if constexpr (G > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            if constexpr (NORM) lds_sum[turn][wave] = sum;
            lds_top[turn][wave] = top;
        }
        __syncthreads();
        sum = 0;
        top = 0;
#pragma unroll
        for (int w = 0; w < G / 64; ++w) {
            if constexpr (NORM) sum += lds_sum[turn][w];
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

// x becomes h: the sum rounded to its type; what the norm is of.
template <int DTYPE>
__device__ __forceinline__ void add_residual(Raw<DTYPE>& x, const Raw<DTYPE>& residual)
{
    float f[8], r[8];
    x.get(f);
    residual.get(r);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += r[e];
    x.set(f);
}

template <int DTYPE>
__device__ __forceinline__ void store_row(void* p, int64_t at, const float (&v)[8], int n)
{
    if constexpr (DTYPE != AG_F32) store_16<DTYPE == AG_BF16>(static_cast<uint16_t*>(p) + at, v, n);
}

constexpr int group_threads(int G) { return G < 256 ? 256 : G; }

// Rows of up to 8 G V elements, G threads to a row, the row in registers between its two uses: sum of squares (and largest
// element) first, then y = h rstd w or the codes.  Bound by memory, read once and written once; a row to a workgroup, since rows in
// turn leave the reduction's latency open.  Measured of 16384 x 8192 bf16: norm with a residual and codes 172 to 182 us (940 MB, 5.2 to
// 5.5 TB/s), codes alone 62 (403 MB, 6.5); of 1000 x 4100 fp16 with odd strides 10.5, of one row of 8192 3.8, both latency.
template <int DTYPE, bool NORM, int G, int V, bool TAIL>
__global__ __launch_bounds__(group_threads(G)) void ag_rows_kernel(RowsArgs a)
{
    constexpr int ROWS = group_threads(G) / G;
    __shared__ double lds_sum[2][16];
    __shared__ uint32_t lds_top[2][16];
    const int lane = threadIdx.x % G;
    const bool weighted = NORM && a.weight != nullptr, add = NORM && a.residual != nullptr;
    // TAIL: the K % 8 elements behind the last whole vector go to as many lanes, one each
    const int whole = TAIL ? a.K & ~7 : a.K, tail = whole + lane;
    const bool extra = TAIL && tail < a.K;
    int turn = 0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS; first < a.M; first += static_cast<int64_t>(gridDim.x) * ROWS) {
        const int64_t mine = first + (ROWS > 1 ? threadIdx.x / G : 0), row = min(mine, a.M - 1);
        const bool live = mine < a.M;
        const void *xs = row_of<DTYPE>(a.x, row, a.ldx), *rs = row_of<DTYPE>(a.residual, row, a.ldr);
        Raw<DTYPE> x[V], r[V], weight[V];
        float one = 0.f, one_r = 0.f, one_w = 1.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (lane + j * G) * 8;
            x[j].template load<false>(xs, col, whole);
            if (add) r[j].template load<false>(rs, col, whole);
        }
        if (extra) {
            one = element<DTYPE>(xs, tail);
            if (add) one_r = element<DTYPE>(rs, tail);
            if (weighted) one_w = element<DTYPE>(a.weight, tail);
        }
        if (weighted) {
#pragma unroll
            for (int j = 0; j < V; ++j) weight[j].template load<false>(a.weight, (lane + j * G) * 8, whole);
        }
        double sum = 0;
        uint32_t top = 0;
        float kept[NORM ? V : 1][8];        // h times the weight; codes of plain rows are taken from x again
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (lane + j * G) * 8;
            float (&v)[8] = kept[NORM ? j : 0];
            if constexpr (NORM) {
                if (add) add_residual<DTYPE>(x[j], r[j]);
                if (a.h && live && col < whole) x[j].store(a.h, row * a.ldh + col, 8);
            }
            x[j].get(v);
            if constexpr (NORM) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fma(static_cast<double>(v[e]), static_cast<double>(v[e]), sum);
                if (weighted) {
                    float w[8];
                    weight[j].get(w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= w[e];
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[e]));
        }
        if constexpr (TAIL) {
            if constexpr (NORM) {
                if (add) one = to_f32<DTYPE == AG_BF16>(from_f32<DTYPE == AG_BF16>(one + one_r));
                if (a.h && live && extra) put_element<DTYPE>(a.h, row * a.ldh + tail, one);
                sum = fma(static_cast<double>(one), static_cast<double>(one), sum);
                one *= one_w;
            }
            top = max(top, magnitude(one));
        }
        reduce_row<NORM, G>(sum, top, lds_sum, lds_top, turn);
        turn ^= 1;
        float rstd = 1.f;
        if constexpr (NORM) rstd = root(sum, a.K, a.eps);
        if (!live) continue;
        if (lane == 0) {
            if (a.scale) a.scale[row] = scale_of(top, rstd);
            if (a.rstd) a.rstd[row] = rstd;
        }
        const Unit unit(top);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (lane + j * G) * 8;
            if (col >= whole) continue;
            float (&v)[8] = kept[NORM ? j : 0];
            if constexpr (!NORM) x[j].get(v);
            if (a.q) store_codes(a.q + row * a.ldq + col, v, unit, 8);
            if (NORM && a.y) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] *= rstd;
                store_row<DTYPE>(a.y, row * a.ldy + col, v, 8);
            }
        }
        if (extra) {
            if (a.q) a.q[row * a.ldq + tail] = static_cast<int8_t>(unit.code(one));
            if (NORM && a.y) put_element<DTYPE>(a.y, row * a.ldy + tail, one * rstd);
        }
    }
}

// Longer rows: a workgroup reads its row twice, the second time from the caches.  Its registers do not hold the row beside the weight
// and the products (1024 threads with four vectors: 4000 x 20000 185 us, read twice 164); LDS would hold 16-bit rows of up to 80000,
// and holds none here.  Bound by memory and by those second reads: with residual and codes bf16 4000 x 20000 156 us, 2000 x 40000 149, 3.6 to
// 3.8 TB/s of what has to move; codes alone of 2000 x 40000 bf16 64 us, fp32 108, 3.7.
constexpr int kLongThreads = 1024;
template <int DTYPE, bool NORM>
__global__ __launch_bounds__(kLongThreads) void ag_rows_long_kernel(RowsArgs a)
{
    __shared__ double lds_sum[2][16];
    __shared__ uint32_t lds_top[2][16];
    const bool weighted = NORM && a.weight != nullptr, add = NORM && a.residual != nullptr;
    constexpr bool TAIL = true;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        // Two vectors of h times the weight, or of the row itself; `stored`: h from where it was stored (x or the residual may
        // be overwritten by then: a thread reads what it wrote itself).  Past the row's end they are 0.
        auto load = [&](Raw<DTYPE> (&x)[2], Raw<DTYPE> (&w)[2], int col, bool stored) {
            const bool from_h = NORM && stored && a.h;
            Raw<DTYPE> r[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = col + j * kLongThreads * 8;
                x[j].template load<TAIL>(from_h ? row_of<DTYPE>(a.h, row, a.ldh) : row_of<DTYPE>(a.x, row, a.ldx), at, a.K);
                if (add && !from_h) r[j].template load<TAIL>(row_of<DTYPE>(a.residual, row, a.ldr), at, a.K);
                if (weighted) w[j].template load<TAIL>(a.weight, at, a.K);
            }
            if constexpr (NORM) {
                if (add && !from_h) {
                    add_residual<DTYPE>(x[0], r[0]);
                    add_residual<DTYPE>(x[1], r[1]);
                }
            }
        };
        auto weigh = [&](float (&v)[8], const Raw<DTYPE>& w) {
            if (!weighted) return;
            float f[8];
            w.get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= f[e];
        };
        double sum = 0;
        uint32_t top = 0;
        for (int col = threadIdx.x * 8; col < a.K; col += kLongThreads * 16) {
            Raw<DTYPE> x[2], w[2];
            load(x, w, col, false);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = col + j * kLongThreads * 8;
                float v[8];
                x[j].get(v);
                if constexpr (NORM) {
                    if (a.h) x[j].store(a.h, row * a.ldh + at, a.K - at);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum = fma(static_cast<double>(v[e]), static_cast<double>(v[e]), sum);
                }
                weigh(v, w[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, magnitude(v[e]));
            }
        }
        reduce_row<NORM, kLongThreads>(sum, top, lds_sum, lds_top, turn);
        turn ^= 1;
        float rstd = 1.f;
        if constexpr (NORM) rstd = root(sum, a.K, a.eps);
        if (threadIdx.x == 0) {
            if (a.scale) a.scale[row] = scale_of(top, rstd);
            if (a.rstd) a.rstd[row] = rstd;
        }
        if (!a.q && !a.y) continue;
        const Unit unit(top);
        for (int col = threadIdx.x * 8; col < a.K; col += kLongThreads * 16) {
            Raw<DTYPE> x[2], w[2];
            load(x, w, col, true);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = col + j * kLongThreads * 8, n = a.K - at;
                float v[8];
                x[j].get(v);
                weigh(v, w[j]);
                if (a.q) store_codes(a.q + row * a.ldq + at, v, unit, n);
                if (NORM && a.y) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= rstd;
                    store_row<DTYPE>(a.y, row * a.ldy + at, v, n);
                }
            }
        }
    }
}

// Bound by memory: 16384 x 8192 to bf16 60 us (403 MB, 6.7 TB/s), a call 70; to fp32 165 (671 MB, 4.1 TB/s; a wave's
// store leaves every other 16 bytes to its next one).
template <int DTYPE>
__global__ __launch_bounds__(256) void ag_dequantize_kernel(DequantizeArgs a)
{
    dequantize_body<DTYPE>(a, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------- the norm's gradients

// One row's sum over G threads; every thread gets it.
template <int G>
__device__ __forceinline__ float sum_row(float s, float (*lds)[16], int turn)
{
    s = combine<(G < 64 ? G : 64)>(s, [](float x, float y) { return x + y; });
    if constexpr (G > 64) {
        if ((threadIdx.x & 63) == 0) lds[turn][threadIdx.x >> 6] = s;
        __syncthreads();
        s = 0.f;
#pragma unroll
        for (int w = 0; w < G / 64; ++w) s += lds[turn][w];
    }
    return s;
}

// One element of dw: an earlier gradient, rounding, store.
__device__ __forceinline__ void put_dw(const NormDwArgs& a, int col, float t)
{
    if (a.dtype == AG_F32) {
        float* p = static_cast<float*>(a.dw) + col;
        *p = a.accumulate ? *p + t : t;
    } else {
        uint16_t* p = static_cast<uint16_t*>(a.dw) + col;
        if (a.accumulate) t += a.dtype == AG_BF16 ? to_f32<true>(*p) : to_f32<false>(*p);
        *p = a.dtype == AG_BF16 ? from_f32<true>(t) : from_f32<false>(t);
    }
}

// With n = h rstd and c = mean(g n): dx = rstd (g - n c) + dh, and dy n for dw, which a workgroup sums over its rows in
// registers (its waves' sums joined through LDS where they take rows of their own).  The row stays as it was loaded and is
// taken apart twice, so that few registers leave many rows on their way.
template <bool BF16, int G, int V, bool TAIL>
__device__ __forceinline__ void backward_rows(const NormBackwardArgs& a, int program, int programs)
{
    constexpr int ROWS = group_threads(G) / G;
    constexpr int DTYPE = BF16 ? AG_BF16 : AG_F16;
    __shared__ float lds[2][16];
    __shared__ float join[ROWS > 1 ? ROWS * G * 8 : 1];
    const int lane = threadIdx.x % G;
    // TAIL: the K % 8 elements behind the last whole vector go to as many lanes, one each
    const int whole = TAIL ? a.K & ~7 : a.K, tail = whole + lane;
    const bool extra = TAIL && tail < a.K;
    Raw<DTYPE> weight[V], dy[V], h[V], dh[V];
    float dw[V][8], one_w = 1.f, one_dw = 0.f;
    if (extra && a.weight) one_w = element<DTYPE>(a.weight, tail);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int col = (lane + j * G) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.f;
        if (a.weight) weight[j].template load<false>(a.weight, col, whole);
        else weight[j].ones();
    }
    const bool add = a.dh != nullptr && a.dx != nullptr;
    const float per_k = 1.f / max(a.K, 1);
    int turn = 0;
    for (int64_t first = static_cast<int64_t>(program) * ROWS; first < a.M; first += static_cast<int64_t>(programs) * ROWS) {
        const int64_t mine = first + (ROWS > 1 ? threadIdx.x / G : 0), row = min(mine, a.M - 1);
        const bool live = mine < a.M;
        const void *ds = row_of<DTYPE>(a.dy, row, a.lddy), *hs = row_of<DTYPE>(a.h, row, a.ldh), *es = row_of<DTYPE>(a.dh, row, a.lddh);
        const float rstd = a.rstd[row];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (lane + j * G) * 8;
            dy[j].template load<false>(ds, col, whole);
            h[j].template load<false>(hs, col, whole);
        }
        if (add) {
#pragma unroll
            for (int j = 0; j < V; ++j) dh[j].template load<false>(es, (lane + j * G) * 8, whole);
        }
        float one_g = 0.f, one_n = 0.f, one_dh = 0.f;
        if (extra) {
            one_g = element<DTYPE>(ds, tail);
            one_n = element<DTYPE>(hs, tail);
            if (add) one_dh = element<DTYPE>(es, tail);
        }
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float g[8], n[8], w[8];
            dy[j].get(g);
            h[j].get(n);
            weight[j].get(w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = g[e] * (n[e] * rstd);
                dw[j][e] += live ? t : 0.f;
                s += t * w[e];
            }
        }
        if constexpr (TAIL) {
            one_n *= rstd;
            const float t = one_g * one_n;
            one_dw += live ? t : 0.f;
            s += t * one_w;
        }
        if (!a.dx) continue;
        const float c = sum_row<G>(s, lds, turn) * per_k;
        turn ^= 1;
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int col = (lane + j * G) * 8;
            if (col >= whole) continue;
            float g[8], n[8], w[8], d[8] = {};
            dy[j].get(g);
            h[j].get(n);
            weight[j].get(w);
            if (add) dh[j].get(d);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = rstd * (g[e] * w[e] - n[e] * rstd * c) + d[e];
            store_16<BF16>(a.dx + row * a.lddx + col, g, 8);
        }
        if (extra) put_element<DTYPE>(a.dx, row * a.lddx + tail, rstd * (one_g * one_w - one_n * c) + one_dh);
    }
    if (!a.sums) return;
    float* out = a.sums + static_cast<int64_t>(program) * a.ldsums;
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
                if (col < whole) out[col] = t;
            }
        } else {
            const int col = (lane + j * G) * 8;     // the rows of sums are whole vectors
            if (col < whole) {
                *reinterpret_cast<f32x4*>(out + col) = f32x4{dw[j][0], dw[j][1], dw[j][2], dw[j][3]};
                *reinterpret_cast<f32x4*>(out + col + 4) = f32x4{dw[j][4], dw[j][5], dw[j][6], dw[j][7]};
            }
        }
    }
    if constexpr (TAIL) {
        if constexpr (ROWS > 1) {
            __syncthreads();
            join[threadIdx.x] = one_dw;
            __syncthreads();
            if (threadIdx.x < static_cast<unsigned>(a.K - whole)) {
                float t = 0.f;
#pragma unroll
                for (int r = 0; r < ROWS; ++r) t += join[r * G + threadIdx.x];
                out[whole + threadIdx.x] = t;
            }
        } else if (extra) {
            out[tail] = one_dw;
        }
    }
}

// n = h rstd, g = dy w, dx = rstd (g - n mean(g n)) + dh, a row in registers between its mean and its dx; dw's sums of dy n
// stay in registers over the rows that a workgroup takes in turn.  Bound by memory: 16384 x 8192 bf16 with dh 194 to 201 us (1074 MB,
// 5.4 TB/s), the sums' join after it 5.
template <bool BF16, int G, int V, bool TAIL>
__global__ __launch_bounds__(group_threads(G)) void ag_norm_backward_kernel(NormBackwardArgs a)
{
    backward_rows<BF16, G, V, TAIL>(a, blockIdx.x, gridDim.x);
}

// dw of 64 columns straight from dy and h, 8 columns to a thread and every 32nd row: for little work, where a second pass over
// the rows beside the first costs less than a second launch after it.
template <bool BF16>
__device__ __forceinline__ void backward_weight(const NormBackwardArgs& a, const NormDwArgs& d, int block, float (*part)[65])
{
    constexpr int DTYPE = BF16 ? AG_BF16 : AG_F16;
    const int c = (threadIdx.x & 7) * 8, lane = threadIdx.x >> 3, col = block * 64 + c;
    float dw[8] = {};
    if (col < a.K) {
#pragma unroll 1
        for (int64_t first = lane; first < a.M; first += 128) {
            Raw<DTYPE> dy[4], h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {       // past the last row nothing is loaded
                const int64_t row = min(first + 32 * j, a.M - 1);
                const int K = first + 32 * j < a.M ? a.K : 0;
                dy[j].template load<true>(row_of<DTYPE>(a.dy, row, a.lddy), col, K);
                h[j].template load<true>(row_of<DTYPE>(a.h, row, a.ldh), col, K);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (first + 32 * j >= a.M) break;
                const float rstd = a.rstd[first + 32 * j];
                float g[8], n[8];
                dy[j].get(g);
                h[j].get(n);
#pragma unroll
                for (int e = 0; e < 8; ++e) dw[e] += g[e] * (n[e] * rstd);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) part[lane][c + e] = dw[e];
    __syncthreads();
    const int out = block * 64 + threadIdx.x;
    if (threadIdx.x >= 64 || out >= a.K) return;
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += part[r][threadIdx.x];
    put_dw(d, out, t);
}

// Bound by the launch: 80 x 520 fp16 3.5 us.
template <bool BF16, int G, int V, bool TAIL>
__global__ __launch_bounds__(256) void ag_norm_backward_small_kernel(NormBackwardArgs a, NormDwArgs d, int dx_programs)
{
    static_assert(group_threads(G) == 256, "both parts take 256 threads");
    __shared__ float part[32][65];
    const int p = blockIdx.x;
    if (p < dx_programs) backward_rows<BF16, G, V, TAIL>(a, p, dx_programs);
    else backward_weight<BF16>(a, d, p - dx_programs, part);
}

// Longer rows in two passes: mean(g n) of each row, and then columns, 8 to a thread, over `rows` rows each.  Bound by memory, dy and h
// read twice: bf16 with dh and dw in fp32 4000 x 20000 198 us, 2000 x 40000 201 (3.2 TB/s of what has to move, 4.9 of what does).
template <bool BF16>
__global__ __launch_bounds__(kLongThreads) void ag_norm_backward_mean_kernel(NormBackwardArgs a)
{
    constexpr int DTYPE = BF16 ? AG_BF16 : AG_F16;
    __shared__ float lds[2][16];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const float rstd = a.rstd[row];
        const void *ds = row_of<DTYPE>(a.dy, row, a.lddy), *hs = row_of<DTYPE>(a.h, row, a.ldh);
        float s = 0.f;
        for (int col = threadIdx.x * 8; col < a.K; col += kLongThreads * 16) {
            Raw<DTYPE> dy[2], h[2], weight[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {       // past the row's end: zeros
                const int at = col + j * kLongThreads * 8;
                dy[j].template load<true>(ds, at, a.K);
                h[j].template load<true>(hs, at, a.K);
                if (a.weight) weight[j].template load<true>(a.weight, at, a.K);
                else weight[j].ones();
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float g[8], n[8], w[8];
                dy[j].get(g);
                h[j].get(n);
                weight[j].get(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) s += g[e] * (n[e] * rstd) * w[e];
            }
        }
        s = sum_row<kLongThreads>(s, lds, turn);
        turn ^= 1;
        if (threadIdx.x == 0) a.means[row] = s / a.K;
    }
}

template <bool BF16>
__global__ __launch_bounds__(256) void ag_norm_backward_columns_kernel(NormBackwardArgs a, int column_groups, int rows)
{
    constexpr int DTYPE = BF16 ? AG_BF16 : AG_F16, AHEAD = 4;       // rows on their way
    const int group = static_cast<int>(blockIdx.x) % column_groups, batch = static_cast<int>(blockIdx.x) / column_groups;
    const int col = (group * 256 + static_cast<int>(threadIdx.x)) * 8;
    if (col >= a.K) return;
    Raw<DTYPE> weight;
    if (a.weight) weight.template load<true>(a.weight, col, a.K);
    else weight.ones();
    const bool add = a.dh != nullptr && a.dx != nullptr;
    float w[8], dw[8] = {};
    weight.get(w);
    const int64_t from = static_cast<int64_t>(batch) * rows, end = min(from + rows, a.M);
    for (int64_t first = from; first < end; first += AHEAD) {
        Raw<DTYPE> dy[AHEAD], h[AHEAD], dh[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int64_t row = min(first + j, end - 1);
            dy[j].template load<true>(row_of<DTYPE>(a.dy, row, a.lddy), col, a.K);
            h[j].template load<true>(row_of<DTYPE>(a.h, row, a.ldh), col, a.K);
            if (add) dh[j].template load<true>(row_of<DTYPE>(a.dh, row, a.lddh), col, a.K);
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int64_t row = first + j;
            if (row >= end) break;
            const float rstd = a.rstd[row];
            float g[8], n[8], d[8] = {};
            dy[j].get(g);
            h[j].get(n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                n[e] *= rstd;
                dw[e] += g[e] * n[e];
            }
            if (!a.dx) continue;
            const float c = a.means[row];
            if (add) dh[j].get(d);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = rstd * (g[e] * w[e] - n[e] * c) + d[e];
            store_16<BF16>(a.dx + row * a.lddx + col, g, a.K - col);
        }
    }
    if (!a.sums) return;
    float* out = a.sums + batch * a.ldsums + col;
    *reinterpret_cast<f32x4*>(out) = f32x4{dw[0], dw[1], dw[2], dw[3]};
    *reinterpret_cast<f32x4*>(out + 4) = f32x4{dw[4], dw[5], dw[6], dw[7]};
}

// dw(k) (+)= the workgroups' sums, in order within 32 lanes and then over them.  32 columns to a workgroup, 4 to a thread.
__global__ __launch_bounds__(256) void ag_norm_dw_kernel(NormDwArgs a)
{
    __shared__ float part[32][33];
    const int c = (threadIdx.x & 7) * 4, lane = threadIdx.x >> 3;
    const float* from = a.sums + static_cast<int64_t>(blockIdx.x) * 32 + c;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int q = lane; q < a.parts; q += 32) s += *reinterpret_cast<const f32x4*>(from + q * a.ldsums);
#pragma unroll
    for (int e = 0; e < 4; ++e) part[lane][c + e] = s[e];
    __syncthreads();
    const int col = blockIdx.x * 32 + threadIdx.x;
    if (threadIdx.x >= 32 || col >= a.K) return;
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += part[r][threadIdx.x];
    put_dw(a, col, t);
}

// ---------------------------------------------------------------- choice of a kernel

using RowsFn = void (*)(RowsArgs);
template <int DTYPE, bool NORM, bool TAIL> RowsFn pick_rows(const RowsShape& s)
{
    switch (s.threads * 8 + s.vectors) {
    case 16 * 8 + 1: return ag_rows_kernel<DTYPE, NORM, 16, 1, TAIL>;
    case 64 * 8 + 1: return ag_rows_kernel<DTYPE, NORM, 64, 1, TAIL>;
    case 64 * 8 + 2: return ag_rows_kernel<DTYPE, NORM, 64, 2, TAIL>;
    case 256 * 8 + 1: return ag_rows_kernel<DTYPE, NORM, 256, 1, TAIL>;
    case 256 * 8 + 2: return ag_rows_kernel<DTYPE, NORM, 256, 2, TAIL>;
    case 512 * 8 + 2: return ag_rows_kernel<DTYPE, NORM, 512, 2, TAIL>;
    case 1024 * 8 + 2:
        if constexpr (NORM) return ag_rows_kernel<DTYPE, NORM, 1024, 2, TAIL>;
        else return nullptr;
    case 512 * 8 + 4:
        if constexpr (NORM) return nullptr;
        else return ag_rows_kernel<DTYPE, NORM, 512, 4, TAIL>;
    case 1024 * 8 + 4:
        if constexpr (NORM) return nullptr;
        else return ag_rows_kernel<DTYPE, NORM, 1024, 4, TAIL>;
    case kLongThreads * 8: return ag_rows_long_kernel<DTYPE, NORM>;
    default: return nullptr;
    }
}
template <int DTYPE, bool NORM> RowsFn pick_rows(const RowsShape& s, int K)
{
    return K % 8 ? pick_rows<DTYPE, NORM, true>(s) : pick_rows<DTYPE, NORM, false>(s);
}

using NormBackwardFn = void (*)(NormBackwardArgs);
template <bool BF16, bool TAIL> NormBackwardFn pick_backward(const RowsShape& s)
{
    switch (s.threads * 8 + s.vectors) {
    case 16 * 8 + 1: return ag_norm_backward_kernel<BF16, 16, 1, TAIL>;
    case 64 * 8 + 1: return ag_norm_backward_kernel<BF16, 64, 1, TAIL>;
    case 64 * 8 + 2: return ag_norm_backward_kernel<BF16, 64, 2, TAIL>;
    case 256 * 8 + 1: return ag_norm_backward_kernel<BF16, 256, 1, TAIL>;
    case 256 * 8 + 2: return ag_norm_backward_kernel<BF16, 256, 2, TAIL>;
    case 512 * 8 + 2: return ag_norm_backward_kernel<BF16, 512, 2, TAIL>;
    case 1024 * 8 + 2: return ag_norm_backward_kernel<BF16, 1024, 2, TAIL>;
    default: return nullptr;
    }
}
using NormBackwardSmallFn = void (*)(NormBackwardArgs, NormDwArgs, int);
template <bool BF16, bool TAIL> NormBackwardSmallFn pick_backward_small(const RowsShape& s)
{
    switch (s.threads * 8 + s.vectors) {
    case 16 * 8 + 1: return ag_norm_backward_small_kernel<BF16, 16, 1, TAIL>;
    case 64 * 8 + 1: return ag_norm_backward_small_kernel<BF16, 64, 1, TAIL>;
    case 64 * 8 + 2: return ag_norm_backward_small_kernel<BF16, 64, 2, TAIL>;
    case 256 * 8 + 1: return ag_norm_backward_small_kernel<BF16, 256, 1, TAIL>;
    case 256 * 8 + 2: return ag_norm_backward_small_kernel<BF16, 256, 2, TAIL>;
    default: return nullptr;
    }
}
template <bool BF16> NormBackwardSmallFn pick_backward_small(const RowsShape& s, int K)
{
    return K % 8 ? pick_backward_small<BF16, true>(s) : pick_backward_small<BF16, false>(s);
}

template <bool BF16> NormBackwardFn pick_backward(const RowsShape& s, int K)
{
    return K % 8 ? pick_backward<BF16, true>(s) : pick_backward<BF16, false>(s);
}

}  // namespace

// ---------------------------------------------------------------- launchers

// Four vectors a thread where the row itself is all that is kept (codes of 4096 x 16384 bf16: 512 threads with four 39.6 us,
// 1024 with two 47 to 52).  A norm keeps the residual, the weight and products in fp32 too and has no registers for them (with
// 512 threads and four 104 us, 1024 and two 94 to 99; 4000 x 20000: 1024 and four 185, read twice 164).
RowsShape rows_shape(int64_t K, bool norm)
{
    if (K <= 128) return {16, 1, 16};
    if (K <= 512) return {64, 1, 4};
    if (K <= 1024) return {64, 2, 4};
    if (K <= 2048) return {256, 1, 1};
    if (K <= 4096) return {256, 2, 1};
    if (K <= 8192) return {512, 2, 1};
    if (norm && K <= 16384) return {1024, 2, 1};
    if (!norm && K <= 16384) return {512, 4, 1};
    if (!norm && K <= 32768) return {1024, 4, 1};
    return {kLongThreads, 0, 1};
}

RowsShape norm_backward_shape(int64_t K) { return K <= 16384 ? rows_shape(K, true) : RowsShape{256, 0, 1}; }

hipError_t launch_rows(const RowsArgs& a, int dtype, bool norm, int programs, hipStream_t stream)
{
    const RowsShape s = rows_shape(a.K, norm);
    const RowsFn fn = norm ? (dtype == AG_BF16 ? pick_rows<AG_BF16, true>(s, a.K) : dtype == AG_F16 ? pick_rows<AG_F16, true>(s, a.K) : nullptr)
                           : (dtype == AG_BF16 ? pick_rows<AG_BF16, false>(s, a.K) : dtype == AG_F16 ? pick_rows<AG_F16, false>(s, a.K)
                                                                                                : pick_rows<AG_F32, false>(s, a.K));
    if (fn == nullptr || programs < 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(programs)), dim3(static_cast<uint32_t>(s.threads * s.per_group)), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_dequantize(const DequantizeArgs& a, int dtype, hipStream_t stream)
{
    const int64_t groups = dequantize_programs(a);
    if (groups < 1) return hipErrorInvalidValue;
    auto fn = dtype == AG_BF16 ? ag_dequantize_kernel<AG_BF16> : dtype == AG_F16 ? ag_dequantize_kernel<AG_F16> : ag_dequantize_kernel<AG_F32>;
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(groups)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_norm_backward(const NormBackwardArgs& a, int bf16, int programs, hipStream_t stream)
{
    const RowsShape s = norm_backward_shape(a.K);
    const NormBackwardFn fn = bf16 ? pick_backward<true>(s, a.K) : pick_backward<false>(s, a.K);
    if (fn == nullptr || programs < 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(programs)), dim3(static_cast<uint32_t>(s.threads * s.per_group)), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_norm_backward_small(const NormBackwardArgs& a, const NormDwArgs& d, int bf16, int dx_programs, hipStream_t stream)
{
    const RowsShape s = norm_backward_shape(a.K);
    const NormBackwardSmallFn fn = bf16 ? pick_backward_small<true>(s, a.K) : pick_backward_small<false>(s, a.K);
    if (fn == nullptr || dx_programs < 1 || a.sums != nullptr) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(dx_programs + (a.K + 63) / 64)), dim3(256), 0, stream, a, d, dx_programs);
    return hipGetLastError();
}

hipError_t launch_norm_backward_long(const NormBackwardArgs& a, int bf16, int batches, int rows, hipStream_t stream)
{
    const int64_t column_groups = (a.K + 2047) / 2048, grid = column_groups * batches;
    if (batches < 1 || rows < 1 || grid > kMaxRowsPrograms || (a.dx && !a.means)) return hipErrorInvalidValue;
    if (a.dx) {
        hipLaunchKernelGGL((bf16 ? ag_norm_backward_mean_kernel<true> : ag_norm_backward_mean_kernel<false>),
                           dim3(static_cast<uint32_t>(std::min<int64_t>(a.M, kMaxRowsPrograms))), dim3(kLongThreads), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((bf16 ? ag_norm_backward_columns_kernel<true> : ag_norm_backward_columns_kernel<false>),
                       dim3(static_cast<uint32_t>(grid)), dim3(256), 0, stream, a, static_cast<int>(column_groups), rows);
    return hipGetLastError();
}

hipError_t launch_norm_dw(const NormDwArgs& a, hipStream_t stream)
{
    if (a.K < 1 || (a.parts > 0 && (a.ldsums % 32 != 0 || a.ldsums < a.K))) return hipErrorInvalidValue;
    hipLaunchKernelGGL(ag_norm_dw_kernel, dim3(static_cast<uint32_t>((a.K + 31) / 32)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace ag
