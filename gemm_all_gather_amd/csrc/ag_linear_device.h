// Device code of the linear layer's kernels for gfx950, shared by the sources that instantiate them: the
// epilogue's arithmetic, and the tiled product in its three operand layouts.
//
// One product is out(i, j) = epilogue(sum_r A(i, r) B(j, r)):
//   y  = x w^T     A = x, B = w, both r-contiguous                     (NT)
//   dx = dz w      A = dz r-contiguous, B = w with j contiguous        (NN)
//   dw = dz^T x    A = dz with i contiguous, B = x with j contiguous   (TN)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "ag.h"
#include "ag_linear.h"
#include "ag_mfma.h"

namespace ag {

// ---------------------------------------------------------------- epilogue

namespace {

template <bool BF16> __device__ __forceinline__ float to_f32(uint16_t v)
{
    if constexpr (BF16) return __builtin_bit_cast(float, static_cast<uint32_t>(v) << 16);
    else return static_cast<float>(__builtin_bit_cast(_Float16, v));
}
template <bool BF16> __device__ __forceinline__ uint16_t from_f32(float v)   // to nearest, ties to even
{
    if constexpr (BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
    else return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

// Vectors at any alignment of their elements (global accesses need none on gfx950).
typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
struct __attribute__((packed, aligned(2))) Any16 { u32x4 v; };

__device__ __forceinline__ u16x8 load8(const uint16_t* p)
{
    return __builtin_bit_cast(u16x8, reinterpret_cast<const Any16*>(p)->v);
}
__device__ __forceinline__ void store8(uint16_t* p, u16x8 v)
{
    reinterpret_cast<Any16*>(p)->v = __builtin_bit_cast(u32x4, v);
}

template <bool BF16>
__device__ __forceinline__ void load_f32(float (&v)[8], const uint16_t* p, int n)
{
    if (n >= 8) {
        const u16x8 t = load8(p);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = to_f32<BF16>(t[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? to_f32<BF16>(p[e]) : 0.f;
    }
}
template <bool BF16>
__device__ __forceinline__ void store_16(uint16_t* p, const float (&v)[8], int n)
{
    u16x8 t;
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = from_f32<BF16>(v[e]);
    if (n >= 8) {
        store8(p, t);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = t[e];
    }
}

constexpr float kGeluK = 0.79788456080286536f;      // sqrt(2/pi)
constexpr float kGeluC = 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + exp(-u)) from the exponential and reciprocal instructions (each within 1 ulp).
__device__ __forceinline__ float sigmoid(float u)
{
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * u));
}

// The normal distribution's integral up to z, and exp(-z^2/2) on the way.  The left tail is exp(-z^2/2) (a1 t + .. +
// a8 t^8) with t = 1/(1 + 0.305 |z|): the a's fit the tail's quotient by exp(-z^2/2), smooth in t, on 0 <= |z| <= 14
// (iteratively reweighted least squares) to 9.4e-8 of itself.  So the tail is right relative to its own small value,
// without cancellation, as far as the exponential is: its exponent's three roundings leave 1.5 z^2 2^-24, 8e-6 at |z| =
// 13, where the tail leaves fp32's normal numbers.  No branches: erff's would not unroll over a tile's epilogue.
__device__ __forceinline__ float normal_integral(float z, float& gauss)
{
    const float t = __builtin_amdgcn_rcpf(1.f + 0.305f * fabsf(z));
    gauss = __builtin_amdgcn_exp2f(-0.5f * kLog2e * z * z);
    const float q = gauss * t *
                    (0.121639736f + t * (0.122466773f + t * (0.103421151f + t * (0.121020712f + t * (-0.0379749462f +
                     t * (0.185714786f + t * (-0.152987048f + t * 0.0366988741f)))))));
    return z < 0.f ? q : 1.f - q;
}

__device__ __forceinline__ void activate(float (&v)[8], int act)
{
    switch (act) {   // uniform
    case AG_ACT_RELU:
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] < 0.f ? 0.f : v[e];
        break;
    case AG_ACT_GELU:
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float gauss;
            v[e] *= normal_integral(v[e], gauss);
        }
        break;
    case AG_ACT_GELU_TANH:   // (1 + tanh(u))/2 = sigmoid(2u)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * sigmoid(2.f * kGeluK * (v[e] + kGeluC * v[e] * v[e] * v[e]));
        break;
    case AG_ACT_SILU:
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * sigmoid(v[e]);
        break;
    default: break;
    }
}

// v <- v * act'(z)
__device__ __forceinline__ void apply_slope(float (&v)[8], const float (&z)[8], int act)
{
    switch (act) {
    case AG_ACT_RELU:
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = z[e] <= 0.f ? 0.f : v[e];
        break;
    case AG_ACT_GELU:
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float gauss;
            const float whole = normal_integral(z[e], gauss);
            v[e] *= whole + z[e] * kInvSqrt2Pi * gauss;
        }
        break;
    case AG_ACT_GELU_TANH:   // with s = sigmoid(2u): s + z s (1 - s) 2u'
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // z^2 overflows from |z| = 1.8e19 on, where s (1 - s) is 0: the factor beside it has to stay finite
            const float zz = fminf(z[e] * z[e], 1e30f);
            const float s = sigmoid(2.f * kGeluK * z[e] * (1.f + kGeluC * zz));
            v[e] *= s + z[e] * s * (1.f - s) * (2.f * kGeluK * (1.f + 3.f * kGeluC * zz));
        }
        break;
    case AG_ACT_SILU:
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float s = sigmoid(z[e]);
            v[e] *= s + z[e] * s * (1.f - s);
        }
        break;
    default: break;
    }
}

// n <= 8 consecutive gradient elements to p: earlier gradient, rounding, store.
template <bool BF16>
__device__ __forceinline__ void put_gradient(float (&v)[8], void* at, int f32, int accumulate, int n)
{
    if (f32) {
        float* p = static_cast<float*>(at);
        if (n >= 8) {
            f32x4u lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
            if (accumulate) {
                lo += *reinterpret_cast<const f32x4u*>(p);
                hi += *reinterpret_cast<const f32x4u*>(p + 4);
            }
            *reinterpret_cast<f32x4u*>(p) = lo;
            *reinterpret_cast<f32x4u*>(p + 4) = hi;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) p[e] = accumulate ? p[e] + v[e] : v[e];
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(at);
        if (accumulate) {
            float o[8];
            load_f32<BF16>(o, p, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        store_16<BF16>(p, v, n);
    }
}
template <bool BF16>
__device__ __forceinline__ void finish_gradient(float (&v)[8], const LinearEpilogue& ep, int64_t row, int64_t col, int n)
{
    put_gradient<BF16>(v, static_cast<char*>(ep.out) + (row * ep.ldo + col) * (ep.out_f32 ? 4 : 2), ep.out_f32, ep.accumulate, n);
}

// n <= 8 consecutive elements of a layer's output: bias, pre-activation, activation, residual, rounding, store.
template <bool BF16>
__device__ __forceinline__ void finish_layer(float (&v)[8], const float (&bias)[8], const LinearEpilogue& ep, int act,
                                             int64_t row, int64_t col, int n)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += bias[e];
    if (ep.z) store_16<BF16>(ep.z + row * ep.ldz + col, v, n);
    activate(v, act);
    if (ep.residual) {
        float r[8];
        load_f32<BF16>(r, ep.residual + row * ep.ldr + col, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += r[e];
    }
    store_16<BF16>(static_cast<uint16_t*>(ep.out) + row * ep.ldo + col, v, n);
}

}  // namespace

// ---------------------------------------------------------------- tiled product

namespace linear_cfg {
// TM x TN output tile, four waves in a 2 x 2 grid (one per SIMD).  The reduction advances 64 at a time; LDS holds
// SA stages of A and SB of B, each operand in a ring of its own.
template <int TM_, int TN_, int SA_, int SB_>
struct Cfg {
    static constexpr int TM = TM_, TN = TN_, SA = SA_, SB = SB_;
    static constexpr int NW = 4, NT = 256;
    static constexpr int WM = TM / 2, WN = TN / 2;         // wave sub-tile
    static constexpr int BM = WM / 16, BN = WN / 16;       // 16 x 16 blocks of it
    static constexpr int PRODUCTS = BM * BN;               // of a 32-wide half stage
    static constexpr int A_BYTES = TM * 128, B_BYTES = TN * 128;   // of a stage
    static constexpr int LDS = SA * A_BYTES + SB * B_BYTES;
    static constexpr int LA = TM / 32, LB = TN / 32;       // loads of a wave per stage
    static constexpr int READ_STEP = PRODUCTS / (2 * (BM + BN)) > 0 ? PRODUCTS / (2 * (BM + BN)) : 1;   // products per read
    // One operand's slot is refilled in the half that follows its last read, the other's (of the deeper ring, B's
    // of equal ones) in the half after that, the first of the next stage.
    static constexpr bool LATE_A = SA > SB;
    static constexpr int STEP_A = PRODUCTS / LA, STEP_B = PRODUCTS / LB;   // products per load
    // Loads still in flight when the next stage has landed: whole groups after it and, with unequal rings, the
    // late operand's loads of its own group.
    static constexpr int S = SA < SB ? SA : SB;
    static constexpr int AHEAD = (S - 2) * (LA + LB) + (SA < SB ? LB : SB < SA ? LA : 0);
    static_assert((BM & (BM - 1)) == 0 && (BN & (BN - 1)) == 0, "transposed fragments address blocks by XOR");
    static_assert(READ_STEP * (BM + BN) <= PRODUCTS && STEP_A >= 1 && STEP_B >= 1, "reads and loads fit between the products");
    static_assert(S >= 2 && SA - SB <= 1 && SB - SA <= 1, "AHEAD counts one extra stage at most");
    static_assert(SA * LA + SB * LB - LA - LB < 64, "vmcnt is 6 bits");
    static_assert(LDS <= 160 * 1024, "gfx950 has 160 KiB of LDS");
};
}  // namespace linear_cfg

namespace {

__device__ __forceinline__ int64_t dword_up(int64_t bytes) { return (bytes + 3) & ~int64_t{3}; }

// One operand's part of an LDS stage.  A wave instruction moves 1 KiB, lane l
// to bytes [16 l, 16 l + 16) of it; the waves share the part's T/8 instructions.
//
// r-contiguous (TR false): the stage holds T rows of 64 r (128 bytes).  The 16-byte chunks of a row
// are XOR-ed with row & 7, so that the fragment reads of 8 rows at one chunk spread over the banks.
// transposed (TR true): 64 rows of r with T columns each (2 T bytes).  The 32-byte units of a row are
// XOR-ed with f(row) = (row & 3) | 4 ((row >> 3) & 1): the eight rows that 32 lanes of a transposing
// read touch (0-3 and 8-11 of a 32-row step) then lie on eight different 32-byte bank groups.
template <int T, bool TR>
struct Part {
    static constexpr int NW = 4;
    static constexpr int J = T / 8 / NW;                // instructions per wave
    static constexpr int RPI = TR ? 512 / T : 8;           // stage rows per instruction
    static constexpr int STEP = RPI * NW;               // stage rows between a wave's instructions
    static constexpr int UNITS = T / 16;                   // transposed: 32-byte units per row

    uint32_t off[J];    // lane's byte offset within the operand tile's stage, per instruction

    __device__ __forceinline__ void init(int lane, int wave, uint32_t ld2)
    {
        if constexpr (TR) {
            constexpr int LPR = 64 / RPI;                  // lanes per stage row
            const uint32_t c = static_cast<uint32_t>(lane % LPR);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const uint32_t row = static_cast<uint32_t>(wave * RPI + lane / LPR + STEP * j);
                const uint32_t f = (row & 3u) | (((row >> 3) & 1u) << 2);
                off[j] = row * ld2 + ((((c >> 1) ^ f) << 5) | ((c & 1u) << 4));
            }
        } else {
            const uint32_t row = static_cast<uint32_t>(lane >> 3);
            const uint32_t chunk = static_cast<uint32_t>(lane & 7) ^ row;
#pragma unroll
            for (int j = 0; j < J; ++j) off[j] = (static_cast<uint32_t>(wave * 8 + STEP * j) + row) * ld2 + chunk * 16u;
        }
    }

    // The operand tile's next stage to load.  Its descriptor starts at the stage and ends with the operand, so that
    // what lies past the operand is neither read nor anything but zero; the end is rounded up to 4 bytes
    // because the range check works on whole dwords (operands are 4-byte aligned: the dword of the last
    // element is the operand's own).
    struct Next {
        uint64_t base;
        int32_t bytes;      // r-contiguous: from base to the end of the tile's rows; transposed: of a row, from base
        int32_t r_left;     // transposed: rows of the reduction from the stage on
        int32_t stages;     // still to load
    };
    // operand: its address; at, size: the tile's first row (column) and the operand's number of them.
    static __device__ __forceinline__ Next start(const uint16_t* operand, int64_t at, int64_t size, int64_t R, uint32_t ld2,
                                                 int first, int count)
    {
        const int64_t r0 = static_cast<int64_t>(first) * 64;
        const int64_t place = TR ? r0 * ld2 + at * 2 : at * ld2 + r0 * 2;
        const int64_t bytes = TR ? dword_up((size - at) * 2) : (min(size - at, int64_t{T}) - 1) * ld2 + dword_up((R - r0) * 2);
        const bool live = count > 0 && R > 0;
        return Next{reinterpret_cast<uint64_t>(operand) + static_cast<uint64_t>(place),
                    live ? static_cast<int32_t>(min(bytes, int64_t{0x7fffffff})) : 0, live ? static_cast<int32_t>(R - r0) : 0, count};
    }
    // The stage's descriptor (base and size); n moves on to the next one.
    struct At {
        uint64_t base;
        uint32_t records;
    };
    static __device__ __forceinline__ At take(Next& n, uint32_t ld2)
    {
        At t;
        t.base = n.base;
        if constexpr (TR) {
            t.records = n.r_left > 0 ? static_cast<uint32_t>(min(n.r_left, 64) - 1) * ld2 + static_cast<uint32_t>(n.bytes) : 0u;
            n.base += static_cast<uint64_t>(ld2) * 64;
            n.r_left -= 64;
        } else {
            t.records = static_cast<uint32_t>(max(n.bytes, 0));
            n.base += 128;
            n.bytes -= 128;
        }
        n.stages -= 1;
        return t;
    }
    __device__ __forceinline__ void load(const At& t, uint8_t* dst, int j) const { fetch(t, dst + NW * j * 1024, off[j]); }
    static __device__ __forceinline__ void fetch(const At& t, uint8_t* dst, uint32_t at)
    {
        const __amdgpu_buffer_rsrc_t r = make_rsrc(t.base, t.records);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (AG_LDS void*)dst, 16, at, 0, 0, 0);
    }
};

// Fragments of 16-row (16-column) blocks for a 32-wide step of the stage.  Lane l receives row
// l & 15 of a block, r = 8 (l >> 4) .. + 7 of the step, from either layout.  The reads are inline assembly:
// the compiler cannot tell them from the LDS-direct loads still landing in the other slot and would
// wait for those; every read is followed by wait_lgkmcnt0() before its use.
template <int T, bool TR>
struct Frags {
    uint32_t base;      // lane's byte offset within the operand's part of the stage, block 0 of step 0

    __device__ __forceinline__ void init(int lane, int first_row)
    {
        if constexpr (TR) {
            // A 16-lane group addresses 4 stage rows x 32 bytes; ds_read_b64_tr_b16 gives lane i column i of them.
            const uint32_t q = static_cast<uint32_t>(lane >> 4), p = static_cast<uint32_t>(lane & 15);
            const uint32_t row = 8u * q + (p >> 2);
            const uint32_t f = (p >> 2) | ((q & 1u) << 2);
            base = row * (2u * T) + (((static_cast<uint32_t>(first_row) >> 4) ^ f) << 5) + ((p & 3u) << 3);
        } else {
            const uint32_t row = static_cast<uint32_t>(lane & 15);
            base = (static_cast<uint32_t>(first_row) + row) * 128u + (((static_cast<uint32_t>(lane) >> 4) ^ (row & 7u)) << 4);
        }
    }
    // Block b of step kk (constants after unrolling).
    template <class V>
    __device__ __forceinline__ void read(V& dst, uint32_t part, int kk, int b) const
    {
        if constexpr (TR) {
            const uint32_t addr = (part + base) ^ (static_cast<uint32_t>(b) << 5);
            u32x2 lo, hi;
            if (kk == 0) {
                asm volatile("ds_read_b64_tr_b16 %0, %1" : "=v"(lo) : "v"(addr));
                asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(hi) : "v"(addr), "i"(8 * T));
            } else {
                asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(lo) : "v"(addr), "i"(64 * T));
                asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(hi) : "v"(addr), "i"(72 * T));
            }
            dst = __builtin_bit_cast(V, u32x4{lo.x, lo.y, hi.x, hi.y});
        } else {
            read_at(dst, (part + base) ^ (static_cast<uint32_t>(kk) << 6), b);   // chunk + 4: bit 2 of the XOR-ed chunk
        }
    }
    template <class V>
    static __device__ __forceinline__ void read_at(V& dst, uint32_t addr, int block)
    {
        switch (block) {   // the offset must be an immediate
#define AG_FRAG_CASE(b) \
    case b: asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(dst) : "v"(addr), "i"(b * 2048)); break;
            AG_FRAG_CASE(0) AG_FRAG_CASE(1) AG_FRAG_CASE(2) AG_FRAG_CASE(3)
            AG_FRAG_CASE(4) AG_FRAG_CASE(5) AG_FRAG_CASE(6) AG_FRAG_CASE(7)
#undef AG_FRAG_CASE
        default: break;
        }
    }
};

// c += b a^T with c in accumulation registers.  Inline assembly keeps the 256 accumulators of a 256 x 256 tile in
// the accumulation half of the register file; left to itself the compiler spread them over both halves and
// spilled.  It does not see these instructions' write latency: c is used again no sooner than BM * BN of them
// later, and settle() stands between them and other uses.
template <bool BF16, class V>
__device__ __forceinline__ void mfma(f32x4& c, V b, V a)
{
    if constexpr (BF16) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
    else asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(b), "v"(a));
}
__device__ __forceinline__ void settle()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ uint32_t lds_address(const uint8_t* p)
{
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((AG_LDS const uint8_t*)p));
}

// Work of a product: the first full_tiles tiles, a tile at a time per workgroup, round by round; then the other
// (tail) tiles' reductions cut into `splits` parts of split_stages 64-wide steps, again a part at a time, all
// tiles' first parts before all second ones: workgroups that run together share operand rows at the same place
// of the reduction (runs of equal length laid end to end over the tiles do not, and took twice the time per
// step: 1024 x 3584 x 8192 over 256 workgroups 129 us, one tile a workgroup 62).  A part's fp32 tile goes to
// partial tile (part, tail tile); a second kernel joins them.
struct Piece {
    int tile, first, count;     // 64-wide steps first .. first + count - 1 of the tile; count 0: no more work
    int unit;                   // of a cut tile: its partial tile
};

__device__ __forceinline__ int spread(int p, int n)
{
    // Workgroup p runs on XCD p % 8: every XCD gets a contiguous run of n consecutive tiles (or
    // runs), so that its L2 serves the rows that neighbouring tiles share.
    return (p & 7) * (n >> 3) + min(p & 7, n & 7) + (p >> 3);
}

// The q-th piece of workgroup p of n.
__device__ __forceinline__ Piece piece_of(const LinearGemmArgs& a, int p, int n, int q)
{
    if (a.heavy > 0) {      // whole tiles: common_rounds rounds on all, then on the workgroups from `heavy` on
        const bool all = q < a.common_rounds;
        const int m = all ? n : n - a.heavy, r = all ? p : p - a.heavy;
        const int at = all ? q * n : a.common_rounds * n + (q - a.common_rounds) * m;
        if (r < 0 || at + r >= a.full_tiles) return Piece{0, 0, 0, 0};
        return Piece{at + spread(r, min(m, a.full_tiles - at)), 0, a.stages, 0};
    }
    const int rounds = a.full_tiles / n + (p < a.full_tiles % n ? 1 : 0);
    if (q < rounds) return Piece{q * n + spread(p, min(n, a.full_tiles - q * n)), 0, a.stages, 0};
    const int tail = a.tiles_i * a.tiles_j - a.full_tiles, units = tail * a.splits;
    const int at = (q - rounds) * n;
    if (at + p >= units) return Piece{0, 0, 0, 0};
    const int unit = at + spread(p, min(n, units - at));
    const int part = unit / tail, first = part * a.split_stages;
    return Piece{a.full_tiles + unit - part * tail, first, min(a.split_stages, a.stages - first), unit};
}

// First row and column of a tile: the order goes 8 tile rows at a time, column by column.
__device__ __forceinline__ void place_tile(const LinearGemmArgs& a, int t, int tm, int tn, int64_t* i0, int64_t* j0)
{
    constexpr int GROUP = 8;
    const int g = t / (GROUP * a.tiles_j);
    const int rows = min(a.tiles_i - g * GROUP, GROUP);
    const int in_group = t - g * GROUP * a.tiles_j;
    *i0 = static_cast<int64_t>(g * GROUP + in_group % rows) * tm;
    *j0 = static_cast<int64_t>(in_group / rows) * tn;
}

// Two neighbouring blocks' accumulators, 4 columns each per lane of each 16-lane row, become 8 consecutive columns:
// row q of the lanes holds columns 8 q .. 8 q + 7 of the blocks' 32.
__device__ __forceinline__ void widen(float (&v)[8], const f32x4& x, const f32x4& y)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t xe, ye;    // moved out of the accumulation registers here, not earlier
        asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(xe) : "a"(x[e]));
        asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(ye) : "a"(y[e]));
        u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(xe, ye, false, false));
        t = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(t.x, t.y, false, false));
        v[e] = __uint_as_float(t.x);
        v[4 + e] = __uint_as_float(t.y);
    }
}

// f(0), .., f(N - 1) with constant arguments: an unrolled loop of any size (the accumulators it indexes stay registers).
template <class F, int... I> __device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F> __device__ __forceinline__ void each(F f) { each_of(std::make_integer_sequence<int, N>{}, f); }

// A lane's place in a matrix, going down 16 rows at a time.
struct Walk {
    char* p;
    int64_t rows16;
    __device__ __forceinline__ Walk(const void* m, int64_t row, int64_t col, int64_t ld, int size)
        : p(static_cast<char*>(const_cast<void*>(m)) + (row * ld + col) * size), rows16(16 * ld * size)
    {
    }
    template <class T> __device__ __forceinline__ T* at(int elements16) const { return reinterpret_cast<T*>(p + 2 * elements16); }
    __device__ __forceinline__ void down() { p += rows16; }
};

template <bool BF16, int FORM, int ACT, class C>
__device__ __forceinline__ void gemm_body(const LinearGemmArgs& a, int program, int programs, uint8_t* ring)
{
    constexpr bool TA = FORM == kFormTN, TB = FORM != kFormNT;
    constexpr int BM = C::BM, BN = C::BN;
    using V = typename Mfma<BF16>::V;
    using PartA = Part<C::TM, TA>;
    using PartB = Part<C::TN, TB>;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const uint32_t lda2 = static_cast<uint32_t>(a.lda) * 2u, ldb2 = static_cast<uint32_t>(a.ldb) * 2u;

    PartA pa;
    PartB pb;
    Frags<C::TM, TA> ra;
    Frags<C::TN, TB> rb;
    pa.init(lane, wave, lda2);
    pb.init(lane, wave, ldb2);
    ra.init(lane, wm * C::WM);
    rb.init(lane, wn * C::WN);

    // The ring takes the parts of all the workgroup's pieces in one stream, so that the next tile's first stages
    // are on their way during a tile's last ones and its epilogue.  A's and B's loads each walk the pieces.
    auto start_a = [&](int q) {
        const Piece w = piece_of(a, program, programs, q);
        int64_t i0, j0;
        place_tile(a, w.tile, C::TM, C::TN, &i0, &j0);
        return PartA::start(a.A, i0, a.I, a.R, lda2, w.first, w.count);
    };
    auto start_b = [&](int q) {
        const Piece w = piece_of(a, program, programs, q);
        int64_t i0, j0;
        place_tile(a, w.tile, C::TM, C::TN, &i0, &j0);
        return PartB::start(a.B, j0, a.J, a.R, ldb2, w.first, w.count);
    };
    int qa = 0, qb = 0;
    typename PartA::Next na = start_a(0);
    typename PartB::Next nb = start_b(0);
    auto take_a = [&] {
        const typename PartA::At t = PartA::take(na, lda2);
        if (na.stages == 0) na = start_a(++qa);     // past the last piece: no stages, nothing more is fetched
        return t;
    };
    auto take_b = [&] {
        const typename PartB::At t = PartB::take(nb, ldb2);
        if (nb.stages == 0) nb = start_b(++qb);
        return t;
    };

    V fa[2][BM], fb[2][BN];   // fragments of the two 32-wide halves of a stage
    uint8_t* ring_b = ring + C::SA * C::A_BYTES;
    auto next_slot = [](int slot, int slots) { return slot + 1 == slots ? 0 : slot + 1; };
    // Where the reduction is no multiple of 64, the last stage of an r-contiguous operand goes on into the next
    // rows: that is set to zero in LDS, once, when a tile's last stage has landed.
    const bool ragged = !(TA && TB) && (a.R & 63) != 0;
    auto clear_tail = [&](int slot_a, int slot_b) {
        const uint32_t from = static_cast<uint32_t>(a.R & 63);
        for (int row = tid; row < C::TM + C::TN; row += C::NT) {
            if ((TA && row < C::TM) || (TB && row >= C::TM)) continue;
            uint8_t* line = row < C::TM ? ring + slot_a * C::A_BYTES + row * 128 : ring_b + slot_b * C::B_BYTES + (row - C::TM) * 128;
            for (uint32_t c = from >> 3; c < 8; ++c) {
                uint8_t* chunk = line + ((c ^ (static_cast<uint32_t>(row) & 7u)) << 4);   // TM is a multiple of 8
                if (c * 8 >= from) {
                    *reinterpret_cast<u32x4*>(chunk) = u32x4{0u, 0u, 0u, 0u};
                } else {
                    for (uint32_t e = from & 7u; e < 8; ++e) reinterpret_cast<uint16_t*>(chunk)[e] = 0;
                }
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    auto read = [&](int f, uint32_t part_a, uint32_t part_b, int kk, int i) {   // i-th fragment: A's blocks, then B's
        if (i < BM) ra.read(fa[f][i], part_a, kk, i);
        else rb.read(fb[f][i - BM], part_b, kk, i - BM);
    };
    const uint32_t lds_a = lds_address(ring), lds_b = lds_address(ring_b);

    // One operand's refill of a slot, spread over a half's products: i-th of them.
    auto refill_a = [&](const typename PartA::At& t, int slot, int i) {
        if (i % C::STEP_A == C::STEP_A - 1 && i / C::STEP_A < C::LA) pa.load(t, ring + slot * C::A_BYTES + wave * 1024, i / C::STEP_A);
    };
    auto refill_b = [&](const typename PartB::At& t, int slot, int i) {
        if (i % C::STEP_B == C::STEP_B - 1 && i / C::STEP_B < C::LB) pb.load(t, ring_b + slot * C::B_BYTES + wave * 1024, i / C::STEP_B);
    };

    // prologue: all slots on their way but the late operand's last (the first stage's first half fills it), the first
    // stage landed and its first fragments read
#pragma unroll
    for (int q = 0; q < max(C::SA, C::SB); ++q) {
        if (q < C::SA - (C::LATE_A ? 1 : 0)) {
            const typename PartA::At la = take_a();
#pragma unroll
            for (int j = 0; j < C::LA; ++j) pa.load(la, ring + q * C::A_BYTES + wave * 1024, j);
        }
        if (q < C::SB - (C::LATE_A ? 0 : 1)) {
            const typename PartB::At lb = take_b();
#pragma unroll
            for (int j = 0; j < C::LB; ++j) pb.load(lb, ring_b + q * C::B_BYTES + wave * 1024, j);
        }
    }
    typename PartA::At la{};
    typename PartB::At lb{};
    if constexpr (C::LATE_A) la = take_a();
    else lb = take_b();
    wait_vmcnt<C::SA * C::LA + C::SB * C::LB - C::LA - C::LB - (C::LATE_A ? C::LA : C::LB)>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    Piece w = piece_of(a, program, programs, 0);
    if (ragged && w.count == 1 && w.first + 1 == a.stages) clear_tail(0, 0);
#pragma unroll
    for (int i = 0; i < BM + BN; ++i) read(0, lds_a, lds_b, 0, i);
    __builtin_amdgcn_sched_barrier(0);
    wait_lgkmcnt0();
    __builtin_amdgcn_sched_barrier(0);

    int sa = 0, sb = 0;         // slots of the stage
    int late = C::LATE_A ? C::SA - 1 : C::SB - 1;   // slot that the late operand fills next
    for (int q = 0; w.count > 0;) {
        const Piece next = piece_of(a, program, programs, q + 1);
        // whether the stage after the piece's last is a tile's last one too
        const bool next_short = next.count > 0 && next.first + 1 == a.stages;
        const bool ends = w.first + w.count == a.stages;

        f32x4 acc[BM][BN];
#pragma unroll
        for (int bm = 0; bm < BM; ++bm)
#pragma unroll
            for (int bn = 0; bn < BN; ++bn) {
                acc[bm][bn] = f32x4{0.f, 0.f, 0.f, 0.f};
                asm volatile("" : "+a"(acc[bm][bn]));
            }
        settle();

        // A stage is two halves of BM x BN products each.  Between the first half's products the second half's
        // fragments are read; then this wave's reads of the stage's slots are complete and the next stage has
        // landed, and one barrier makes both true for all waves.  Between the second half's products the next
        // stage's first fragments are read.  The stage's two slots are refilled with stages SA and SB further on, one
        // operand's between the second half's products, the other's between the next stage's first half's: a
        // wave is held at a load until the CU takes it (about one 1 KiB instruction per 22 cycles per CU, 1408
        // cycles for a 256 x 256 tile's stage of 2048), so they have to lie evenly.  The order is pinned by
        // scheduling barriers (scalar and address arithmetic may cross them); the fragment reads are
        // waited for as a whole before the half that uses them.
#pragma unroll 1
        for (int s = 0; s < w.count; ++s) {
            const int next_a = next_slot(sa, C::SA), next_b = next_slot(sb, C::SB);
            const uint32_t here_a = lds_a + sa * C::A_BYTES, here_b = lds_b + sb * C::B_BYTES;
            const uint32_t there_a = lds_a + next_a * C::A_BYTES, there_b = lds_b + next_b * C::B_BYTES;
#pragma unroll
            for (int i = 0; i < C::PRODUCTS; ++i) {
                if (i % C::READ_STEP == 0 && i / C::READ_STEP < BM + BN) read(1, here_a, here_b, 1, i / C::READ_STEP);
                if constexpr (C::LATE_A) refill_a(la, late, i);
                else refill_b(lb, late, i);
                mfma<BF16>(acc[i / BN][i % BN], fb[0][i % BN], fa[0][i / BN]);
                __builtin_amdgcn_sched_barrier(0x6);
            }
            la = take_a();
            lb = take_b();
            __builtin_amdgcn_sched_barrier(0);
            wait_lgkmcnt0();
            wait_vmcnt<C::AHEAD>();
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            if (ragged && (s + 2 == w.count ? ends : s + 1 == w.count && next_short)) clear_tail(next_a, next_b);
#pragma unroll
            for (int i = 0; i < C::PRODUCTS; ++i) {
                if (i % C::READ_STEP == 0 && i / C::READ_STEP < BM + BN) read(0, there_a, there_b, 0, i / C::READ_STEP);
                if constexpr (C::LATE_A) refill_b(lb, sb, i);
                else refill_a(la, sa, i);
                mfma<BF16>(acc[i / BN][i % BN], fb[1][i % BN], fa[1][i / BN]);
                __builtin_amdgcn_sched_barrier(0x6);
            }
            __builtin_amdgcn_sched_barrier(0);
            wait_lgkmcnt0();
            __builtin_amdgcn_sched_barrier(0);
            late = C::LATE_A ? sa : sb;
            sa = next_a;
            sb = next_b;
        }
        settle();

        // ---- epilogue, from the registers: a lane's accumulators hold 4 consecutive columns of one row of each
        // block; lanes trade halves of neighbouring blocks, and each then has 8 consecutive columns in fp32 for
        // 16-byte accesses (64 bytes of a row together) and the one rounding at the very end.
        int64_t i0, j0;
        place_tile(a, w.tile, C::TM, C::TN, &i0, &j0);
        int own = lane;
        asm volatile("" : "+v"(own));   // opaque: the lane's addresses are made here, not kept across the loop
        const int tile_row = wm * C::WM + (own & 15), tile_col = wn * C::WN + (own >> 4) * 8;
        const int64_t row0 = i0 + tile_row, col0 = j0 + tile_col;
        if (w.count != a.stages) {
            float* d = a.partial + static_cast<int64_t>(w.unit) * (C::TM * C::TN) + tile_row * C::TN + tile_col;
#pragma unroll
            for (int bm = 0; bm < BM; ++bm, d += 16 * C::TN)
#pragma unroll
                for (int b = 0; b < BN / 2; ++b) {
                    float x[8];
                    widen(x, acc[bm][2 * b], acc[bm][2 * b + 1]);
                    *reinterpret_cast<f32x4*>(d + 32 * b) = f32x4{x[0], x[1], x[2], x[3]};
                    *reinterpret_cast<f32x4*>(d + 32 * b + 4) = f32x4{x[4], x[5], x[6], x[7]};
                    __builtin_amdgcn_sched_barrier(0);   // one vector's values at a time
                }
        } else if (i0 + C::TM <= a.I && j0 + C::TN <= a.J) {
            // the whole tile inside: no bounds, and every address one step from the one before
            Walk out(a.epi.out, row0, col0, a.epi.ldo, a.epi.out_f32 ? 4 : 2);
            Walk z(a.epi.z, row0, col0, a.epi.ldz, 2), res(a.epi.residual, row0, col0, a.epi.ldr, 2);
            float bias[BN / 2][8] = {};
            if (FORM == kFormNT && a.epi.bias) {
#pragma unroll
                for (int b = 0; b < BN / 2; ++b) load_f32<BF16>(bias[b], a.epi.bias + col0 + 32 * b, 8);
            }
            each<BM>([&](auto row_block) __attribute__((always_inline)) {
                constexpr int bm = decltype(row_block)::value;
#pragma unroll
                for (int b = 0; b < BN / 2; ++b) {
                    float x[8];
                    widen(x, acc[bm][2 * b], acc[bm][2 * b + 1]);
                    if constexpr (FORM == kFormNT) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] += bias[b][e];
                        if (a.epi.z) store_16<BF16>(z.at<uint16_t>(32 * b), x, 8);
                        activate(x, ACT);
                        if (a.epi.residual) {
                            float r[8];
                            load_f32<BF16>(r, res.at<uint16_t>(32 * b), 8);
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] += r[e];
                        }
                        store_16<BF16>(out.at<uint16_t>(32 * b), x, 8);
                    } else if (FORM == kFormTN && (a.epi.out_f32 || a.epi.accumulate)) {
                        put_gradient<BF16>(x, out.at<void>(a.epi.out_f32 ? 64 * b : 32 * b), a.epi.out_f32, a.epi.accumulate, 8);
                    } else {
                        store_16<BF16>(out.at<uint16_t>(32 * b), x, 8);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                out.down();
                if (FORM == kFormNT) {
                    z.down();
                    res.down();
                }
            });
        } else {
            each<BM>([&](auto row_block) __attribute__((always_inline)) {
                constexpr int bm = decltype(row_block)::value;
                const int64_t row = row0 + 16 * bm;
#pragma unroll
                for (int b = 0; b < BN / 2; ++b) {
                    float x[8];
                    widen(x, acc[bm][2 * b], acc[bm][2 * b + 1]);
                    const int64_t col = col0 + 32 * b;
                    const int n = static_cast<int>(max(int64_t{0}, min(int64_t{8}, a.J - col)));
                    if (row < a.I && n > 0) {
                        if constexpr (FORM == kFormNT) {
                            float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                            if (a.epi.bias) load_f32<BF16>(bias, a.epi.bias + col, n);
                            finish_layer<BF16>(x, bias, a.epi, ACT, row, col, n);
                        } else {
                            finish_gradient<BF16>(x, a.epi, row, col, n);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            });
        }
        w = next;
        ++q;
    }
    wait_vmcnt<0>();   // loads past the last stage write LDS: they end with the workgroup
}

// Sums the partial column sums of 32 columns: 8 row lanes, then a fixed order through LDS (8 x 33 floats).
__device__ __forceinline__ void bias_grad_body(const LinearBiasGradArgs& a, int block, float* part)
{
    const int c = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(block) * 32 + c;
    float s = 0.f;
    if (col < a.N) {
#pragma unroll 8
        for (int64_t q = rl; q < a.parts; q += 8) s += a.sums[q * a.N + col];
    }
    part[rl * 33 + c] = s;
    __syncthreads();
    if (rl == 0 && col < a.N) {
        s = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) s += part[r * 33 + c];
        if (a.kind == 2) {
            float* p = static_cast<float*>(a.db) + col;
            *p = a.accumulate ? *p + s : s;
        } else {
            uint16_t* p = static_cast<uint16_t*>(a.db) + col;
            if (a.accumulate) s += a.kind == 1 ? to_f32<true>(*p) : to_f32<false>(*p);
            *p = a.kind == 1 ? from_f32<true>(s) : from_f32<false>(s);
        }
    }
}

// The bias gradient's column groups after a product's tiles, on the workgroups with the fewest tiles first: a launch of
// its own takes 4 to 5 us and a gap (all gradients of 1024 x 3584 x 8192 with it 132 to 137 us, so 126).
__device__ __forceinline__ void bias_grads_after(const LinearBiasGradArgs& db, int program, int programs, uint8_t* ring)
{
    if (!db.db) return;
    for (int block = programs - 1 - program; block < (db.N + 31) / 32; block += programs) {
        __syncthreads();
        bias_grad_body(db, block, reinterpret_cast<float*>(ring));
    }
}

template <bool BF16, int FORM, int ACT, class C>
__global__ __launch_bounds__(C::NT, 1) void ag_linear_gemm_kernel(LinearGemmArgs a)
{
    __shared__ __attribute__((aligned(1024))) uint8_t ring[C::LDS];
    gemm_body<BF16, FORM, ACT, C>(a, blockIdx.x, gridDim.x, ring);
    if constexpr (FORM != kFormNT) bias_grads_after(a.db, blockIdx.x, gridDim.x, ring);
}

// dx, dw and the bias gradient's sum one after the other on every workgroup: the product with the longer tiles first,
// and those workgroups that have fewer of its tiles take more of the other's.  Two launches round up to
// whole rounds twice (dw 3584 x 8192 of 16384 rows: 448 tiles on 256 CUs, 1.75 rounds).
template <bool BF16, bool DX_FIRST, class C>
__global__ __launch_bounds__(C::NT, 1) void ag_linear_grads_in_turn_kernel(LinearGemmArgs dx, LinearGemmArgs dw, LinearBiasGradArgs db)
{
    __shared__ __attribute__((aligned(1024))) uint8_t ring[C::LDS];
    const int p = blockIdx.x, n = gridDim.x;
    if constexpr (DX_FIRST) {
        gemm_body<BF16, kFormNN, AG_ACT_NONE, C>(dx, p, n, ring);
        __syncthreads();
        gemm_body<BF16, kFormTN, AG_ACT_NONE, C>(dw, p, n, ring);
    } else {
        gemm_body<BF16, kFormTN, AG_ACT_NONE, C>(dw, p, n, ring);
        __syncthreads();
        gemm_body<BF16, kFormNN, AG_ACT_NONE, C>(dx, p, n, ring);
    }
    bias_grads_after(db, p, n, ring);
}

// dx, dw and the bias gradient's sum in one launch, for layers whose tiles together leave CUs free: workgroups
// below dx_programs take dx, the next dw_programs dw, the others 32 columns each of db.
template <bool BF16, class C>
__global__ __launch_bounds__(C::NT, 1) void ag_linear_grads_kernel(LinearGemmArgs dx, LinearGemmArgs dw, int dx_programs,
                                                                   int dw_programs, LinearBiasGradArgs db)
{
    __shared__ __attribute__((aligned(1024))) uint8_t ring[C::LDS];
    const int p = blockIdx.x;
    if (p < dx_programs) gemm_body<BF16, kFormNN, AG_ACT_NONE, C>(dx, p, dx_programs, ring);
    else if (p < dx_programs + dw_programs) gemm_body<BF16, kFormTN, AG_ACT_NONE, C>(dw, p - dx_programs, dw_programs, ring);
    else bias_grad_body(db, p - dx_programs - dw_programs, reinterpret_cast<float*>(ring));
}

// Measured, with one launch's start, epilogue and join:
//   256 x 256  16384 x 3584 x 8192 NT with gelu_tanh and z, bf16, 680 to 709 us, 1.36 to 1.41 PFLOP/s (a library product
//              of the same operands without epilogue 753); its gradients NN 659 and TN 687.  The matrix pipe is
//              busy 72 to 74% of the cycles at the 1.8 GHz that the card's power limit leaves (zero operands 17 to 20% faster).
//   256 x 128  1024 x 8192 x 3584 NN (dx; 256 tiles) 58 us, 1.04 PFLOP/s.
//   128 x 128  1024 x 3584 x 8192 NT with gelu and residual (224 tiles) 72 us, 0.84 PFLOP/s (the library 70 without
//              either); without both, after a long warm-up, 60.  A stage takes 1060 cycles or more of 512 in the
//              matrix pipe.  Not the fragments' latency holds it: reading them a stage before their use, with one
//              stage less on its way, measured the same (34.8 and 35.0 us for 1024 x 4096 x 4096).
// What holds the smaller two is not known.  A 128 x 128 stage needs 704 cycles of a CU's load intake, 768 of LDS and 512
// of the matrix pipe, and takes 1060 to 1420 (181 750 cycles over the 128 stages of 1024 x 3584 x 8192); a 256 x 128 one
// 1056, 1152 and 1024, and takes about 2300 (0.98 to 1.02 us).  All three tiles draw 12 to 15 TB/s from L2.
// 256 x 256: a wave's 128 x 128 sub-tile keeps LDS reads (128 KiB a stage) and the rings' refill (64 KiB) below the
// matrix pipe's 2048 cycles a stage at 128 bytes per cycle; its accumulators take 256 registers.
// 256 x 128 (1152 LDS cycles against 1024) and 128 x 128 (768 against 512): for products with fewer tiles.
using Cfg256 = linear_cfg::Cfg<256, 256, 3, 2>;
using Cfg256x128 = linear_cfg::Cfg<256, 128, 3, 4>;
using Cfg128 = linear_cfg::Cfg<128, 128, 5, 5>;

}  // namespace
}  // namespace ag
