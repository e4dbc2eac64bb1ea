// Kernels of the linear layer on 8-bit integers beside its tiled products: the join of cut tiles, the row-streaming form
// for a few rows of x, copies to aligned rows, and the launchers.

#include "ag_linear_device.h"

namespace ag {
namespace {

// ---------------------------------------------------------------- join of cut tiles

// Adds the parts of a tail tile, 8 consecutive columns per thread: sums of integers, exact in any order; then the epilogue.
// Bound by memory as the join of 16-bit products: 256 tiles of 256 x 256 in two parts 17 to 18 us (8 of 128 x 128 in 11 parts, latency, 5.5).
template <bool BF16>
__global__ __launch_bounds__(256) void ag_linear_i8_join_kernel(LinearI8GemmArgs a, int tm, int tn)
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
    uint32_t s[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    const int64_t part = static_cast<int64_t>(a.tiles_i * a.tiles_j - a.full_tiles) * (tm * tn);
    const float* from = a.partial + static_cast<int64_t>(tail_tile) * (tm * tn) + tile_row * tn + tile_col;
#pragma unroll 4
    for (int q = 0; q < a.splits; ++q, from += part) {
        const u32x4* src = reinterpret_cast<const u32x4*>(from);
        const u32x4 lo = src[0], hi = src[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[e] += lo[e];
            s[4 + e] += hi[e];
        }
    }
    const int n = static_cast<int>(min(int64_t{8}, a.J - col));
    float v[8], scale[8], bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(s[e]);
    load_scales(scale, a.col_scale + col, n);
    apply_scales(v, a.row_scale[row], scale);
    if (a.epi.bias) load_f32<BF16>(bias, a.epi.bias + col, n);
    finish_layer<BF16>(v, bias, a.epi, a.epi.act, row, col, n);
}

// ---------------------------------------------------------------- a few rows of x

typedef int i32x4 __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(1))) AnyBytes16 { i32x4 v; };

__device__ __forceinline__ i32x4 load16(const int8_t* p) { return reinterpret_cast<const AnyBytes16*>(p)->v; }
__device__ __forceinline__ i32x4 load16(const int8_t* p, int64_t left)
{
    if (left >= 16) return load16(p);
    i32x4 t = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (e < left) t[e >> 2] |= static_cast<int>(static_cast<uint32_t>(static_cast<uint8_t>(p[e])) << (8 * (e & 3)));
    return t;
}

// y for up to 16 MB rows of x: the weights are streamed once, straight into matrix-instruction fragments, 16 rows of w per
// workgroup.  The workgroup's waves share the reduction, 256 / MB wide at a time, and add up through LDS; D rows are rows of
// w, D columns rows of x.  Bound by the stream of w and the start and end of a launch: 3584 x 8192 8.2 us of one row (29 MB; 5.3 at a
// large copy's rate), 11.5 of 17, where each workgroup's reads of x weigh as much as those of w.
template <bool BF16, int MB, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void ag_linear_i8_stream_kernel(LinearI8StreamArgs a)
{
    __shared__ i32x4 part[WAVES][MB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int64_t row = min(n0 + (lane & 15), a.N - 1);     // rows past N repeat the last one and are not stored
    const int k_lane = (lane >> 4) * 16;
    const int8_t* w = a.w + row * a.ldw + k_lane;
    const int8_t* x[MB];
    bool live[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int64_t m = b * 16 + (lane & 15);
        live[b] = m < a.M;
        x[b] = a.x + (live[b] ? m : 0) * a.ldx + k_lane;
    }
    // What the epilogue's threads read, one per row of x and 4 rows of w, is on its way before the weights.
    const int tid = threadIdx.x;
    const int64_t my_row = (tid >> 6) * 16 + (tid & 15), my_col = n0 + ((tid & 63) >> 4) * 4;
    const int my_n = tid < MB * 64 && my_row < a.M ? static_cast<int>(max(int64_t{0}, min(int64_t{4}, a.N - my_col))) : 0;
    float scale[8] = {}, bias[8] = {}, residual[8] = {}, x_scale = 0.f;
    if (my_n > 0) {
        x_scale = a.x_scale[my_row];
        load_scales(scale, a.w_scale + my_col, my_n);
        if (a.epi.bias) load_f32<BF16>(bias, a.epi.bias + my_col, my_n);
        if (a.epi.residual) load_f32<BF16>(residual, a.epi.residual + my_row * a.epi.ldr + my_col, my_n);
    }
    i32x4 acc[MB];
    const i32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = zero;

    constexpr int U = linear_i8_stream_width(MB) / 64;       // steps of a block
    struct Block {
        i32x4 w[U], x[MB][U];
    };
    auto load = [&](Block& t, int64_t k) {
#pragma unroll
        for (int u = 0; u < U; ++u) t.w[u] = load16(w + k + u * 64);
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                t.x[b][u] = zero;
                if (live[b]) t.x[b][u] = load16(x[b] + k + u * 64);
            }
    };
    auto multiply = [&](const Block& t) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < MB; ++b) acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(t.w[u], t.x[b][u], acc[b], 0, 0, 0);
    };
    // two blocks on their way per wave while a third is multiplied
    constexpr int64_t WIDE = 64 * U, NEXT = WAVES * WIDE;
    const int64_t whole = a.K / WIDE * WIDE;
    int64_t k = wave * WIDE;
    Block even, odd;
    if (k < whole) load(even, k);
    for (; k < whole; k += 2 * NEXT) {
        const bool more = k + NEXT < whole;
        if (more) load(odd, k + NEXT);
        multiply(even);
        if (k + 2 * NEXT < whole) load(even, k + 2 * NEXT);
        if (more) multiply(odd);
    }
    if (whole < a.K && wave == (whole / WIDE) % WAVES) {   // the last, shorter block
        k = whole;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t left = a.K - k - u * 64 - k_lane;
            const i32x4 fw = load16(w + k + u * 64, left);
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                const i32x4 fx = live[b] ? load16(x[b] + k + u * 64, left) : zero;
                acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw, fx, acc[b], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) part[wave][b][lane] = acc[b];
    __syncthreads();
    if (my_n > 0) {
        const int b = tid >> 6, l = tid & 63;
        i32x4 s = part[0][b][l];
#pragma unroll
        for (int wv = 1; wv < WAVES; ++wv) s += part[wv][b][l];
        float v[8] = {};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __int_as_float(s[e]);
        apply_scales(v, x_scale, scale);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += bias[e];
        if (a.epi.z) store_16<BF16>(a.epi.z + my_row * a.epi.ldz + my_col, v, my_n);
        activate(v, a.epi.act);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += residual[e];
        store_16<BF16>(static_cast<uint16_t*>(a.epi.out) + my_row * a.epi.ldo + my_col, v, my_n);
    }
}

// ---------------------------------------------------------------- rows to aligned rows

// Rows to rows of 16-byte multiples, for operands that do not start on 4 bytes or have other strides: one matrix, or both
// operands one after the other in one launch.  Bound by memory: 1000 x 4100 and 4100 x 4100 9.2 us (42 MB).
__global__ __launch_bounds__(256) void ag_linear_i8_pack_kernel(LinearI8Pack first, LinearI8Pack second, uint32_t first_groups)
{
    const bool one = blockIdx.x < first_groups;
    const LinearI8Pack& p = one ? first : second;
    const uint32_t program = one ? blockIdx.x : blockIdx.x - first_groups, programs = one ? first_groups : gridDim.x - first_groups;
    const int64_t per_row = (p.cols + 15) / 16, all = p.rows * per_row;
    for (int64_t id = static_cast<int64_t>(program) * 256 + threadIdx.x; id < all; id += static_cast<int64_t>(programs) * 256) {
        const int64_t row = id >> 32 ? id / per_row : static_cast<uint32_t>(id) / static_cast<uint32_t>(per_row), col = (id - row * per_row) * 16;
        *reinterpret_cast<i32x4*>(p.dst + row * p.ld_dst + col) = load16(p.src + row * p.ld_src + col, p.cols - col);
    }
}

using StreamFn = void (*)(LinearI8StreamArgs);
template <bool BF16, int MB> StreamFn pick_stream(bool wide)
{
    return wide ? ag_linear_i8_stream_kernel<BF16, MB, 16> : ag_linear_i8_stream_kernel<BF16, MB, 8>;
}

bool grid_of(int64_t work, int64_t per, dim3* grid)
{
    const int64_t g = (work + per - 1) / per;
    if (g < 1 || g > 0x7fffffff) return false;
    *grid = dim3(static_cast<uint32_t>(g));
    return true;
}

}  // namespace

// ---------------------------------------------------------------- launchers

hipError_t launch_linear_i8_gemm(const LinearI8GemmArgs& a, int bf16, int tile, int programs, hipStream_t stream)
{
    const LinearI8GemmFn fn = bf16 ? linear_i8_bf16(a.epi.act, tile) : linear_i8_f16(a.epi.act, tile);
    if (fn == nullptr || programs < 1 || a.stages < 1 || a.splits < 1 || a.split_stages < 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(programs)), dim3(Cfg256::NT), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_linear_i8_join(const LinearI8GemmArgs& a, int bf16, int tile, hipStream_t stream)
{
    int tm, tn, threads;
    linear_tile_shape(tile, &tm, &tn, &threads);
    const int64_t tiles = static_cast<int64_t>(a.tiles_i) * a.tiles_j - a.full_tiles;
    dim3 grid;
    if (!grid_of(tiles * (tm * tn / 2048), 1, &grid)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((bf16 ? ag_linear_i8_join_kernel<true> : ag_linear_i8_join_kernel<false>), grid, dim3(256), 0, stream, a, tm, tn);
    return hipGetLastError();
}

hipError_t launch_linear_i8_stream(const LinearI8StreamArgs& a, int bf16, int cus, hipStream_t stream)
{
    dim3 grid;
    if (a.M < 1 || a.M > kLinearI8StreamRows || !grid_of(a.N, 16, &grid)) return hipErrorInvalidValue;
    const bool wide = static_cast<int64_t>(grid.x) <= cus;
    const int blocks = linear_i8_stream_blocks(a.M);
    const StreamFn fn = blocks == 1 ? (bf16 ? pick_stream<true, 1>(wide) : pick_stream<false, 1>(wide))
                        : blocks == 2 ? (bf16 ? pick_stream<true, 2>(wide) : pick_stream<false, 2>(wide))
                                      : (bf16 ? pick_stream<true, 4>(wide) : pick_stream<false, 4>(wide));
    hipLaunchKernelGGL(fn, grid, dim3(wide ? 1024 : 512), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_linear_i8_pack(const LinearI8Pack& first, const LinearI8Pack& second, hipStream_t stream)
{
    auto groups = [](const LinearI8Pack& p) { return min((p.rows * ((p.cols + 15) / 16) + 255) / 256, int64_t{1} << 22); };
    const int64_t one = groups(first), all = one + groups(second);
    if (all < 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL(ag_linear_i8_pack_kernel, dim3(static_cast<uint32_t>(all)), dim3(256), 0, stream, first, second, static_cast<uint32_t>(one));
    return hipGetLastError();
}

}  // namespace ag
