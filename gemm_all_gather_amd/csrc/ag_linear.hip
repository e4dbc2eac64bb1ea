// Linear layer kernels beside the tiled products: the join of cut tiles, the row-streaming form for a few rows of
// x, copies to aligned rows, the activation's gradient with the bias gradient's column sums, and the launchers.
// (The tiled products are instantiated in ag_linear_forward_*.hip and ag_linear_grads_*.hip.)

#include "ag_linear_device.h"

namespace ag {
namespace {

// ---------------------------------------------------------------- join of cut tiles

// Adds the parts of a tail tile in order, 8 consecutive columns per thread, then the epilogue: out = epilogue(p_0 +
// p_1 + ..) in fp32.  Bound by memory: it reads every partial tile once, some of it still in the last-level cache.
// 128 tiles of 256 x 256 in two parts each (67 MB read, 34 MB written with z): 19 us, 5.3 TB/s.  A second launch
// and a fixed order instead of a counter and the last workgroup's sum: no atomics, no cleared counters, and the
// result does not depend on timing.
template <bool BF16, bool LAYER>
__global__ __launch_bounds__(256) void ag_linear_join_kernel(LinearGemmArgs a, int tm, int tn)
{
    const int per_tile = tm * tn / 2048;           // workgroups
    const int tail_tile = static_cast<int>(blockIdx.x) / per_tile;
    const int id = (static_cast<int>(blockIdx.x) % per_tile) * 256 + threadIdx.x;
    const int tile_row = id / (tn / 8), tile_col = (id % (tn / 8)) * 8;
    int64_t row, col;
    place_tile(a, a.full_tiles + tail_tile, tm, tn, &row, &col);
    row += tile_row;
    col += tile_col;
    if (row >= a.I || col >= a.J) return;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int64_t part = static_cast<int64_t>(a.tiles_i * a.tiles_j - a.full_tiles) * (tm * tn);
    const float* from = a.partial + static_cast<int64_t>(tail_tile) * (tm * tn) + tile_row * tn + tile_col;
#pragma unroll 4
    for (int q = 0; q < a.splits; ++q, from += part) {
        const f32x4* src = reinterpret_cast<const f32x4*>(from);
        const f32x4 lo = src[0], hi = src[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] += lo[e];
            v[4 + e] += hi[e];
        }
    }
    const int n = static_cast<int>(min(int64_t{8}, a.J - col));
    float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if constexpr (LAYER) {
        if (a.epi.bias) load_f32<BF16>(bias, a.epi.bias + col, n);
        finish_layer<BF16>(v, bias, a.epi, a.epi.act, row, col, n);
    } else {
        finish_gradient<BF16>(v, a.epi, row, col, n);
    }
}

// ---------------------------------------------------------------- a few rows of x

// y for up to 16 MB rows of x: the weights are streamed once, straight into matrix-instruction fragments,
// 16 rows of w per workgroup.  The workgroup's waves share the reduction, 128 wide at a time, and add up
// through LDS in a fixed order.  D rows are rows of w, D columns rows of x.  Matrix instructions though one row of x
// fills a sixteenth of them: they take the dot products off the vector pipe and cost nothing beside the loads.
// Bound by the stream of w (58.7 MB for N x K = 3584 x 8192: 11.4 us at a large copy's 5.14 TB/s) and the start and end
// of a launch: 1 row, bf16, 13.0 us = 4.5 TB/s; 13 rows of 8192 x 3584, fp16, 15.7.
template <bool BF16>
__device__ __forceinline__ typename Mfma<BF16>::V stream_load(const uint16_t* p, int64_t left)
{
    u16x8 t;
    if (left >= 8) {
        t = load8(p);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = e < left ? p[e] : static_cast<uint16_t>(0);
    }
    return __builtin_bit_cast(typename Mfma<BF16>::V, t);
}

template <bool BF16, int MB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void ag_linear_stream_kernel(LinearStreamArgs a)
{
    using V = typename Mfma<BF16>::V;
    __shared__ f32x4 part[WAVES][MB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int64_t row = min(n0 + (lane & 15), a.N - 1);     // rows past N repeat the last one and are not stored
    const int k_lane = (lane >> 4) * 8;
    const uint16_t* w = a.w + row * a.ldw + k_lane;
    const uint16_t* x[MB];
    bool live[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int64_t m = b * 16 + (lane & 15);
        live[b] = m < a.M;
        x[b] = a.x + (live[b] ? m : 0) * a.ldx + k_lane;
    }
    f32x4 acc[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const V zero = __builtin_bit_cast(V, u32x4{0u, 0u, 0u, 0u});

    struct Block {
        V w[4], x[MB][4];
    };
    auto load = [&](Block& t, int64_t k) {
#pragma unroll
        for (int u = 0; u < 4; ++u) t.w[u] = __builtin_bit_cast(V, load8(w + k + u * 32));
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                t.x[b][u] = zero;
                if (live[b]) t.x[b][u] = __builtin_bit_cast(V, load8(x[b] + k + u * 32));
            }
    };
    auto multiply = [&](const Block& t) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int b = 0; b < MB; ++b) acc[b] = Mfma<BF16>::run(t.w[u], t.x[b][u], acc[b]);
    };
    // two 128-wide blocks on their way per wave while a third is multiplied
    constexpr int64_t NEXT = WAVES * 128;
    const int64_t whole = a.K / 128 * 128;
    int64_t k = wave * 128;
    Block even, odd;
    if (k < whole) load(even, k);
    for (; k < whole; k += 2 * NEXT) {
        const bool more = k + NEXT < whole;
        if (more) load(odd, k + NEXT);
        multiply(even);
        if (k + 2 * NEXT < whole) load(even, k + 2 * NEXT);
        if (more) multiply(odd);
    }
    if (whole < a.K && wave == (whole / 128) % WAVES) {   // the last, shorter block
        k = whole;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t left = a.K - k - u * 32 - k_lane;
            const V fw = stream_load<BF16>(w + k + u * 32, left);
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                const V fx = live[b] ? stream_load<BF16>(x[b] + k + u * 32, left) : zero;
                acc[b] = Mfma<BF16>::run(fw, fx, acc[b]);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) part[wave][b][lane] = acc[b];
    __syncthreads();
    // one thread per row of x and 4 rows of w
    const int tid = threadIdx.x;
    if (tid < MB * 64) {
        const int b = tid >> 6, l = tid & 63;
        f32x4 s = part[0][b][l];
#pragma unroll
        for (int wv = 1; wv < WAVES; ++wv) s += part[wv][b][l];
        const int64_t m = b * 16 + (l & 15), col = n0 + (l >> 4) * 4;
        const int n = static_cast<int>(max(int64_t{0}, min(int64_t{4}, a.N - col)));
        if (m < a.M && n > 0) {
            float v[8] = {s[0], s[1], s[2], s[3], 0.f, 0.f, 0.f, 0.f};
            float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (a.epi.bias) load_f32<BF16>(bias, a.epi.bias + col, n);
            finish_layer<BF16>(v, bias, a.epi, a.epi.act, m, col, n);
        }
    }
}

// ---------------------------------------------------------------- rows to aligned rows

// A matrix's rows to rows of 16-byte multiples, for operands that start on an odd element or have odd strides: a copy
// by 8 elements, bound by memory.  Two more launches and twice the operands' bytes, against a tiled product
// that could not use LDS-direct loads at all (they take addresses of 4 bytes).
__global__ __launch_bounds__(256) void ag_linear_pack_kernel(const uint16_t* src, int64_t ld_src, uint16_t* dst,
                                                             int64_t ld_dst, int64_t rows, int64_t cols)
{
    const int64_t per_row = (cols + 7) / 8;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t row = id / per_row, col = (id - row * per_row) * 8;
    if (row >= rows) return;
    const uint16_t* s = src + row * ld_src + col;
    u16x8 t;
    if (cols - col >= 8) {
        t = load8(s);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = e < cols - col ? s[e] : static_cast<uint16_t>(0);
    }
    *reinterpret_cast<u16x8*>(dst + row * ld_dst + col) = t;
}

// ---------------------------------------------------------------- activation's gradient, bias gradient

// dz = dy act'(z), rounded to the products' type, and the column sums of the unrounded dz over a.rows rows (summed on
// by bias_grad_body: two levels in a fixed order, no atomics).  32 column groups of 8 x 8 row lanes; a workgroup takes
// 256 columns.  One pass over dy and z, bound by HBM: 16384 x 3584, gelu_tanh (352 MB): 69 to 71 us, 5.0 TB/s, a copy's
// rate.  A kernel of its own because dz is an operand of both products; in their loads the slope would be computed
// once per tile row and column (14 and 32 times), and they take operands to LDS without passing registers.  REST: dz's
// second term too, as an instantiation of its own (a branch cost the other calls up to 1 us).
template <bool BF16, bool REST>
__global__ __launch_bounds__(256) void ag_linear_slope_kernel(LinearSlopeArgs a)
{
    __shared__ float part[8][264];
    const int c = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const uint32_t col_blocks = static_cast<uint32_t>((a.N + 255) / 256);
    const int64_t bx = blockIdx.x % col_blocks, by = blockIdx.x / col_blocks;
    const int64_t col = (bx * 32 + c) * 8;
    const int64_t row0 = by * a.rows;
    const int n = static_cast<int>(max(int64_t{0}, min(int64_t{8}, a.N - col)));
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (n > 0) {
#pragma unroll 4
        for (int i = rl; i < a.rows; i += 8) {
            const int64_t row = row0 + i;
            if (row >= a.M) break;
            float v[8];
            load_f32<BF16>(v, a.dy + row * a.lddy + col, n);
            if (a.z) {
                float z[8];
                load_f32<BF16>(z, a.z + row * a.ldz + col, n);
                apply_slope(v, z, a.act);
            }
            if (a.dz) store_16<BF16>(a.dz + row * a.lddz + col, v, n);
            if constexpr (REST) {
                float rest[8];      // exact in fp32; nothing of what is not finite in 16 bits
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float kept = to_f32<BF16>(from_f32<BF16>(v[e]));
                    rest[e] = __builtin_isfinite(kept) ? v[e] - kept : 0.f;
                }
                store_16<BF16>(a.dz_rest + row * a.lddz + col, rest, n);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += v[e];
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

// Where only the bias gradient is asked for (else it is summed beside a product).  Bound by a launch's latency: 4 to 5 us.
__global__ __launch_bounds__(256) void ag_linear_bias_grad_kernel(LinearBiasGradArgs a)
{
    __shared__ float part[8 * 33];
    bias_grad_body(a, blockIdx.x, part);
}

}  // namespace

// ---------------------------------------------------------------- launchers

void linear_tile_shape(int tile, int* tm, int* tn, int* threads)
{
    *tm = tile == kLinearTile128 ? Cfg128::TM : Cfg256::TM;
    *tn = tile == kLinearTile256 ? Cfg256::TN : Cfg128::TN;
    *threads = Cfg256::NT;
}

hipError_t launch_linear_gemm(const LinearGemmArgs& a, int bf16, int form, int tile, int programs, hipStream_t stream)
{
    const LinearGemmFn fn = form == kFormNT ? (bf16 ? linear_forward_bf16(a.epi.act, tile) : linear_forward_f16(a.epi.act, tile))
                                            : (bf16 ? linear_gradient_bf16(form, tile) : linear_gradient_f16(form, tile));
    if (fn == nullptr || programs < 1 || a.stages < 1 || a.splits < 1 || a.split_stages < 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(programs)), dim3(Cfg256::NT), 0, stream, a);
    return hipGetLastError();
}

namespace {
bool grid_of(int64_t work, int64_t per, dim3* grid)
{
    const int64_t g = (work + per - 1) / per;
    if (g < 1 || g > 0x7fffffff) return false;
    *grid = dim3(static_cast<uint32_t>(g));
    return true;
}
}  // namespace

hipError_t launch_linear_join(const LinearGemmArgs& a, int bf16, int form, int tile, hipStream_t stream)
{
    int tm, tn, threads;
    linear_tile_shape(tile, &tm, &tn, &threads);
    const int64_t tiles = static_cast<int64_t>(a.tiles_i) * a.tiles_j - a.full_tiles;
    dim3 grid;
    if (!grid_of(tiles * (tm * tn / 2048), 1, &grid)) return hipErrorInvalidValue;
    auto fn = form == kFormNT ? (bf16 ? ag_linear_join_kernel<true, true> : ag_linear_join_kernel<false, true>)
                              : (bf16 ? ag_linear_join_kernel<true, false> : ag_linear_join_kernel<false, false>);
    hipLaunchKernelGGL(fn, grid, dim3(256), 0, stream, a, tm, tn);
    return hipGetLastError();
}

namespace {
using StreamFn = void (*)(LinearStreamArgs);
template <bool BF16, int MB> StreamFn pick_stream(bool wide)
{
    return wide ? ag_linear_stream_kernel<BF16, MB, 16> : ag_linear_stream_kernel<BF16, MB, 8>;
}
}  // namespace

// Sixteen waves a workgroup where there is at most one workgroup per CU, eight where several share one: one row of
// x, bf16, 224 workgroups (N 3584, K 8192) 13.1 against 15.2 us; 13 rows, fp16, 512 workgroups (N 8192, K 3584)
// 15.8 against 14.9.
hipError_t launch_linear_stream(const LinearStreamArgs& a, int bf16, int cus, hipStream_t stream)
{
    dim3 grid;
    if (a.M < 1 || a.M > kLinearStreamRows || !grid_of(a.N, 16, &grid)) return hipErrorInvalidValue;
    const bool wide = static_cast<int64_t>(grid.x) <= cus;
    const StreamFn fn = a.M <= 16 ? (bf16 ? pick_stream<true, 1>(wide) : pick_stream<false, 1>(wide))
                                  : (bf16 ? pick_stream<true, 2>(wide) : pick_stream<false, 2>(wide));
    hipLaunchKernelGGL(fn, grid, dim3(wide ? 1024 : 512), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_linear_pack(const uint16_t* src, int64_t ld_src, uint16_t* dst, int64_t ld_dst, int64_t rows,
                              int64_t cols, hipStream_t stream)
{
    dim3 grid;
    if (!grid_of(rows * ((cols + 7) / 8), 256, &grid)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(ag_linear_pack_kernel, grid, dim3(256), 0, stream, src, ld_src, dst, ld_dst, rows, cols);
    return hipGetLastError();
}

hipError_t launch_linear_slope(const LinearSlopeArgs& a, int bf16, hipStream_t stream)
{
    dim3 grid;
    if (a.rows < 1 || !grid_of((a.N + 255) / 256 * ((a.M + a.rows - 1) / a.rows), 1, &grid)) return hipErrorInvalidValue;
    auto fn = a.dz_rest ? (bf16 ? ag_linear_slope_kernel<true, true> : ag_linear_slope_kernel<false, true>)
                        : (bf16 ? ag_linear_slope_kernel<true, false> : ag_linear_slope_kernel<false, false>);
    hipLaunchKernelGGL(fn, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_linear_bias_grad(const LinearBiasGradArgs& a, hipStream_t stream)
{
    dim3 grid;
    if (!grid_of(a.N, 32, &grid)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(ag_linear_bias_grad_kernel, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_linear_grads_in_turn(const LinearGemmArgs& dx, const LinearGemmArgs& dw, bool dx_first, int programs,
                                       const LinearBiasGradArgs& db, int bf16, hipStream_t stream)
{
    if (programs < 1 || dx.splits != 1 || dw.splits != 1 || dx.heavy >= programs || dw.heavy >= programs) return hipErrorInvalidValue;
    const LinearInTurnFn fn = bf16 ? linear_in_turn_bf16(dx_first) : linear_in_turn_f16(dx_first);
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(programs)), dim3(Cfg256::NT), 0, stream, dx, dw, db);
    return hipGetLastError();
}

hipError_t launch_linear_grads(const LinearGemmArgs& dx, const LinearGemmArgs& dw, int dx_programs, int dw_programs,
                               const LinearBiasGradArgs& db, int bf16, hipStream_t stream)
{
    const int64_t db_programs = db.db ? (db.N + 31) / 32 : 0;
    const int64_t grid = dx_programs + dw_programs + db_programs;
    if (dx_programs < 1 || dw_programs < 1 || grid > 0x7fffffff || dx.splits != 1 || dw.splits != 1)
        return hipErrorInvalidValue;
    static_assert(Cfg128::NT == 256, "the bias gradient takes 256 threads");
    hipLaunchKernelGGL((bf16 ? linear_side_by_side_bf16() : linear_side_by_side_f16()), dim3(static_cast<uint32_t>(grid)), dim3(Cfg128::NT), 0, stream, dx, dw, dx_programs, dw_programs, db);
    return hipGetLastError();
}

}  // namespace ag
