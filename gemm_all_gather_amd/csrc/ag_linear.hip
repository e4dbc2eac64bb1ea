// Linear layer kernels for gfx950: the matrix product with bias, activation
// and residual in its epilogue, in the three operand layouts that a layer and
// its gradients need, a row-streaming form for a few rows of x, and the
// activation's gradient with the bias gradient's column sums.
//
// One product is out(i, j) = epilogue(sum_r A(i, r) B(j, r)):
//   y  = x w^T     A = x, B = w, both r-contiguous                     (NT)
//   dx = dz w      A = dz r-contiguous, B = w with j contiguous        (NN)
//   dw = dz^T x    A = dz with i contiguous, B = x with j contiguous   (TN)

#include <hip/hip_runtime.h>
#include <stdint.h>

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

constexpr float kSqrt1_2 = 0.70710678118654752f;
constexpr float kGeluK = 0.79788456080286536f;      // sqrt(2/pi)
constexpr float kGeluC = 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + exp(-u)) from the exponential and reciprocal instructions (each within 1 ulp).
__device__ __forceinline__ float sigmoid(float u)
{
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * u));
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
        for (int e = 0; e < 8; ++e) v[e] = 0.5f * v[e] * (1.f + erff(v[e] * kSqrt1_2));
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
        for (int e = 0; e < 8; ++e)
            v[e] *= 0.5f * (1.f + erff(z[e] * kSqrt1_2)) +
                    z[e] * kInvSqrt2Pi * __builtin_amdgcn_exp2f(-0.5f * kLog2e * z[e] * z[e]);
        break;
    case AG_ACT_GELU_TANH:   // with s = sigmoid(2u): s + z s (1 - s) 2u'
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float zz = z[e] * z[e];
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

// Bias, pre-activation, activation, residual, earlier gradient, rounding and
// store of n <= 8 consecutive elements (row, col..) in fp32.
template <bool BF16>
__device__ __forceinline__ void finish(float (&v)[8], const float (&bias)[8], const LinearEpilogue& ep, int64_t row,
                                       int64_t col, int n)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += bias[e];
    if (ep.z) store_16<BF16>(ep.z + row * ep.ldz + col, v, n);
    activate(v, ep.act);
    if (ep.residual) {
        float r[8];
        load_f32<BF16>(r, ep.residual + row * ep.ldr + col, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += r[e];
    }
    if (ep.out_f32) {
        float* p = static_cast<float*>(ep.out) + row * ep.ldo + col;
        if (n >= 8) {
            f32x4u lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
            if (ep.accumulate) {
                lo += *reinterpret_cast<const f32x4u*>(p);
                hi += *reinterpret_cast<const f32x4u*>(p + 4);
            }
            *reinterpret_cast<f32x4u*>(p) = lo;
            *reinterpret_cast<f32x4u*>(p + 4) = hi;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) p[e] = ep.accumulate ? p[e] + v[e] : v[e];
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(ep.out) + row * ep.ldo + col;
        if (ep.accumulate) {
            float o[8];
            load_f32<BF16>(o, p, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        store_16<BF16>(p, v, n);
    }
}

}  // namespace

// ---------------------------------------------------------------- tiled product

namespace linear_cfg {
// TM x TN output tile, eight waves in a 4 x 2 grid, the reduction 64 at a time through two LDS slots.
template <int TM_, int TN_, int OCC_>
struct Cfg {
    static constexpr int TM = TM_, TN = TN_;
    static constexpr int WGM = 4, WGN = 2, NW = 8, NT = 512, HALF = 4;
    static constexpr int WTM = TM / WGM, WTN = TN / WGN;   // wave sub-tile
    static constexpr int BM = WTM / 16, BN = WTN / 16;     // 16 x 16 blocks of it
    static constexpr int OCC = OCC_;                       // waves per SIMD
    static constexpr int A_BYTES = TM * 128, STAGE = (TM + TN) * 128;
    static constexpr int C_PITCH = WTN * 4 + 16;           // a staged fp32 row of the epilogue
    static constexpr int LPR = WTN / 8;                    // lanes per staged row
    static constexpr int RPP = 64 / LPR;                   // rows per pass of the wave
    static_assert((BM & (BM - 1)) == 0 && (BN & (BN - 1)) == 0, "transposed fragments address blocks by XOR");
    static_assert(NW * 16 * C_PITCH <= 2 * STAGE, "every wave stages 16 rows of its sub-tile");
    static_assert(2 * STAGE <= 160 * 1024, "gfx950 has 160 KiB of LDS");
};
}  // namespace linear_cfg

namespace {

// One operand's part of an LDS stage.  A wave instruction moves 1 KiB, lane l
// to bytes [16 l, 16 l + 16) of it; HALF waves share the T/8 instructions.
//
// r-contiguous (TR false): the stage holds T rows of 64 r (128 bytes).  The 16-byte chunks of a row
// are XOR-ed with row & 7, so that the fragment reads of 8 rows at one chunk spread over the banks.
// transposed (TR true): 64 rows of r with T columns each (2 T bytes).  The 32-byte units of a row are
// XOR-ed with f(row) = (row & 3) | 4 ((row >> 3) & 1): the eight rows that 32 lanes of a transposing
// read touch (0-3 and 8-11 of a 32-row step) then lie on eight different 32-byte bank groups.
template <class C, int T, bool TR>
struct Part {
    static constexpr int J = T / 8 / C::HALF;              // instructions per loading wave
    static constexpr int RPI = TR ? 512 / T : 8;           // stage rows per instruction
    static constexpr int STEP = RPI * C::HALF;             // stage rows between a wave's instructions
    static constexpr int UNITS = T / 16;                   // transposed: 32-byte units per row

    uint32_t off[TR && STEP == 8 ? 2 : 1];   // lane's byte offset within the operand tile, first instruction
    uint32_t r_lane;                         // r-contiguous: first r of the lane's chunk within the stage

    __device__ __forceinline__ void init(int lane, int wp, uint32_t ld2)
    {
        if constexpr (TR) {
            static_assert(STEP == 8 || STEP == 16, "f changes with the instruction by bit 2 alone, or not");
            constexpr int LPR = 64 / RPI;                  // lanes per stage row
            const uint32_t row = static_cast<uint32_t>(wp * RPI + lane / LPR);   // < STEP
            const uint32_t f = (row & 3u) | (((row >> 3) & 1u) << 2);
            const uint32_t c = static_cast<uint32_t>(lane % LPR);
            const uint32_t col = (((c >> 1) ^ f) << 5) | ((c & 1u) << 4);
            off[0] = row * ld2 + col;
            if constexpr (STEP == 8) off[1] = row * ld2 + (col ^ 128u);          // rows with bit 3 set
            r_lane = 0;
        } else {
            const uint32_t row = static_cast<uint32_t>(lane >> 3);
            const uint32_t chunk = static_cast<uint32_t>(lane & 7) ^ row;
            off[0] = (static_cast<uint32_t>(wp * 8) + row) * ld2 + chunk * 16u;
            r_lane = chunk * 8u;
        }
    }

    // Stage kt of the operand tile at base (its first row or column already applied).  live: false loads
    // nothing (and writes zeros).  The descriptor starts at the stage and ends with the operand, so that what
    // lies past the reduction's or the last column's end reads as zero and nothing past the operand is read; the
    // end is rounded up to 4 bytes because the range check works on whole dwords (operands are 4-byte
    // aligned: the dword of the last element is the operand's own).
    // extent: bytes from base to the operand's end (r-contiguous), bytes of a row from base (transposed).
    __device__ __forceinline__ void load(uint64_t base, int64_t extent, int64_t R, uint32_t ld2, uint8_t* dst, int kt,
                                         int wp, bool live) const
    {
        const int64_t r0 = static_cast<int64_t>(kt) * 64;
        const int64_t skip = TR ? r0 * ld2 : r0 * 2;
        int64_t records = TR ? (R - 1 - r0) * static_cast<int64_t>(ld2) + extent : extent - skip;
        if (!live || r0 >= R || records < 0) records = 0;
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(base + static_cast<uint64_t>(skip), static_cast<uint64_t>(records));
        uint32_t l2 = ld2, o0 = off[0], o1 = off[TR && STEP == 8 ? 1 : 0];
        if constexpr (!TR) o0 = r0 + r_lane < R ? o0 : kOutOfRange;   // chunks past the end belong to the next row
        // opaque copies: the instructions' offsets are not kept in registers across the loop
        asm volatile("" : "+v"(o0), "+v"(o1), "+s"(l2));
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t o = TR && STEP == 8 && (j & 1) ? o1 : o0;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (AG_LDS void*)(dst + (wp + C::HALF * j) * 1024), 16,
                                                     o + static_cast<uint32_t>(STEP * j) * l2, 0, 0, 0);
        }
    }
};

// Fragments of NB 16-row (16-column) blocks for a 32-wide step of the stage.  Lane l receives row
// l & 15 of a block, r = 8 (l >> 4) .. + 7 of the step, from either layout.  The reads are inline assembly:
// the compiler cannot tell them from the LDS-direct loads still landing in the other slot and would
// wait for those; every read is followed by wait_lgkmcnt0() before its use.
template <class C, int T, bool TR, int NB>
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
    template <class V>
    __device__ __forceinline__ void read(V (&dst)[NB], uint32_t part, int kk) const
    {
        if constexpr (TR) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint32_t addr = (part + base) ^ (static_cast<uint32_t>(b) << 5);
                u32x2 lo, hi;
                if (kk == 0) {
                    asm volatile("ds_read_b64_tr_b16 %0, %1" : "=v"(lo) : "v"(addr));
                    asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(hi) : "v"(addr), "i"(8 * T));
                } else {
                    asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(lo) : "v"(addr), "i"(64 * T));
                    asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(hi) : "v"(addr), "i"(72 * T));
                }
                dst[b] = __builtin_bit_cast(V, u32x4{lo.x, lo.y, hi.x, hi.y});
            }
        } else {
            const uint32_t addr = (part + base) ^ (static_cast<uint32_t>(kk) << 6);   // chunk + 4: bit 2 of the XOR-ed chunk
#pragma unroll
            for (int b = 0; b < NB; ++b) read_at(dst[b], addr, b);
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

__device__ __forceinline__ uint32_t lds_address(const uint8_t* p)
{
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((AG_LDS const uint8_t*)p));
}
__device__ __forceinline__ int64_t dword_up(int64_t bytes) { return (bytes + 3) & ~int64_t{3}; }

template <bool BF16, int FORM, class C>
__global__ __launch_bounds__(C::NT, C::OCC) void ag_linear_gemm_kernel(LinearGemmArgs a)
{
    constexpr bool TA = FORM == kFormTN, TB = FORM != kFormNT;
    using M = Mfma<BF16>;
    using V = typename M::V;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[2][C::STAGE];

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WGN, wn = wave % C::WGN;
    const int half = wave / C::HALF, wp = wave % C::HALF;   // waves sit on SIMDs round-robin: each half has one on every SIMD
    const uint32_t lda2 = static_cast<uint32_t>(a.lda) * 2u, ldb2 = static_cast<uint32_t>(a.ldb) * 2u;

    // workgroup -> part of the reduction and tile.  Workgroup p runs on XCD p % 8: every XCD gets a
    // contiguous run of the tile order, which goes 8 tile rows at a time, so that its L2 serves shared rows.
    const int tiles = a.tiles_i * a.tiles_j;
    const int p = blockIdx.x, n = gridDim.x;
    const int xcd = p & 7, per = n >> 3, more = n & 7;
    const int v = xcd * per + min(xcd, more) + (p >> 3);
    const int split = v / tiles;
    const int t = v - split * tiles;
    constexpr int GROUP = 8;
    const int g = t / (GROUP * a.tiles_j);
    const int gm = min(a.tiles_i - g * GROUP, GROUP);
    const int in_group = t - g * GROUP * a.tiles_j;
    const int64_t i0 = static_cast<int64_t>(g * GROUP + in_group % gm) * C::TM;
    const int64_t j0 = static_cast<int64_t>(in_group / gm) * C::TN;

    const uint64_t a_base = reinterpret_cast<uint64_t>(a.A) + static_cast<uint64_t>(TA ? i0 * 2 : i0 * lda2);
    const uint64_t b_base = reinterpret_cast<uint64_t>(a.B) + static_cast<uint64_t>(TB ? j0 * 2 : j0 * ldb2);
    const int64_t a_extent = TA ? dword_up((a.I - i0) * 2) : (a.I - 1 - i0) * lda2 + dword_up(a.R * 2);
    const int64_t b_extent = TB ? dword_up((a.J - j0) * 2) : (a.J - 1 - j0) * ldb2 + dword_up(a.R * 2);

    Part<C, C::TM, TA> pa;
    Part<C, C::TN, TB> pb;
    Frags<C, C::TM, TA, C::BM> ra;
    Frags<C, C::TN, TB, C::BN> rb;
    pa.init(lane, wp, lda2);
    pb.init(lane, wp, ldb2);
    ra.init(lane, wm * C::WTM);
    rb.init(lane, wn * C::WTN);

    const int stages_all = static_cast<int>((a.R + 63) >> 6);
    const int first = split * a.stages_per_split;
    const int count = max(0, min(stages_all - first, a.stages_per_split));

    f32x4 acc[C::BM][C::BN];
#pragma unroll
    for (int bm = 0; bm < C::BM; ++bm)
#pragma unroll
        for (int bn = 0; bn < C::BN; ++bn) acc[bm][bn] = f32x4{0.f, 0.f, 0.f, 0.f};
    V fa[C::BM], fb[C::BN];

    auto load_a = [&](int slot, int s) { pa.load(a_base, a_extent, a.R, lda2, &ring[slot][0], first + s, wp, s < count); };
    auto load_b = [&](int slot, int s) {
        pb.load(b_base, b_extent, a.R, ldb2, &ring[slot][C::A_BYTES], first + s, wp, s < count);
    };
    // The last 16-byte chunk of an r-contiguous row holds elements past the reduction's end when R is no
    // multiple of 8: they are set to zero in LDS, once, when the last stage has landed.
    auto clear_tail = [&](int slot) {
        const uint32_t chunk = static_cast<uint32_t>(a.R & 63) >> 3, from = static_cast<uint32_t>(a.R & 7);
        for (int row = tid; row < C::TM + C::TN; row += C::NT) {
            if ((TA && row < C::TM) || (TB && row >= C::TM)) continue;
            const uint32_t r7 = static_cast<uint32_t>(row < C::TM ? row : row - C::TM) & 7u;
            uint16_t* c = reinterpret_cast<uint16_t*>(&ring[slot][row * 128 + ((chunk ^ r7) << 4)]);
            for (uint32_t e = from; e < 8; ++e) c[e] = 0;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    const bool tail = !(TA && TB) && (a.R & 7) != 0 && first + count == stages_all;

    // Two slots.  Stage s + 2's A part is loaded by half s % 2 of the waves right after the barrier that
    // ends the reads of stage s, into the slot it frees; its B part by the other half at the start of stage
    // s + 1.  A wave that issues loads is held until the CU takes them, so on every SIMD one wave goes on issuing matrix
    // instructions meanwhile; and a wave's loads in flight at a boundary are those of the next stage alone.
    auto stage = [&](int s, int slot) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            if (kk == 0 && s >= 1 && half != ((s - 1) & 1)) load_b(slot ^ 1, s + 1);
            const uint32_t part = lds_address(&ring[slot][0]);
            ra.read(fa, part, kk);
            rb.read(fb, part + C::A_BYTES, kk);
            __builtin_amdgcn_sched_barrier(0);
            wait_lgkmcnt0();
            __builtin_amdgcn_sched_barrier(0);
            if (kk == 1) {
                wait_vmcnt<0>();
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
                if (half == (s & 1)) load_a(slot, s + 2);
            }
#pragma unroll
            for (int bm = 0; bm < C::BM; ++bm)
#pragma unroll
                for (int bn = 0; bn < C::BN; ++bn) acc[bm][bn] = M::run(fb[bn], fa[bm], acc[bm][bn]);
        }
        if (tail && s + 2 == count) clear_tail(slot ^ 1);
    };

    if (half == 0) {
        load_a(0, 0);
        load_b(0, 0);
        wait_vmcnt<0>();
    } else {
        load_a(1, 1);
        load_b(1, 1);
    }
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (tail && count == 1) clear_tail(0);
    for (int s = 0; s < count; s += 2) {
        stage(s, 0);
        if (s + 1 < count) stage(s + 1, 1);
    }

    // ---- epilogue.  A lane's accumulators hold 4 consecutive columns of one row of each block; every wave
    // passes its sub-tile through its own piece of LDS, 16 rows at a time in fp32, and then holds 8
    // consecutive columns per lane and whole row pieces per group of lanes: wide, coalesced accesses for the
    // residual, the pre-activation and the output, and the one rounding at the very end.
    wait_vmcnt<0>();   // loads of stages past the end have landed too
    wait_lgkmcnt0();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    uint8_t* mine = &ring[0][0] + wave * (16 * C::C_PITCH);
    const int64_t col = j0 + wn * C::WTN + (lane % C::LPR) * 8;
    const int n_col = static_cast<int>(max(int64_t{0}, min(int64_t{8}, a.J - col)));
    float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.splits == 1 && a.epi.bias) load_f32<BF16>(bias, a.epi.bias + col, n_col);
#pragma unroll
    for (int bm = 0; bm < C::BM; ++bm) {
#pragma unroll
        for (int bn = 0; bn < C::BN; ++bn)
            *reinterpret_cast<f32x4*>(mine + (lane & 15) * C::C_PITCH + (bn * 16 + (lane >> 4) * 4) * 4) = acc[bm][bn];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
        for (int pass = 0; pass < 16 / C::RPP; ++pass) {
            const int r = pass * C::RPP + lane / C::LPR;
            const f32x4* src = reinterpret_cast<const f32x4*>(mine + r * C::C_PITCH + (lane % C::LPR) * 32);
            const f32x4 lo = src[0], hi = src[1];
            const int64_t row = i0 + wm * C::WTM + bm * 16 + r;
            if (row < a.I && n_col > 0) {
                float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                if (a.splits > 1) {
                    f32x4* d = reinterpret_cast<f32x4*>(a.partial + (split * a.I + row) * a.partial_ld + col);
                    d[0] = lo;      // rows of the parts are padded to whole vectors
                    d[1] = hi;
                } else {
                    finish<BF16>(x, bias, a.epi, row, col, n_col);
                }
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
}

// 128 x 128 tiles take 64 KiB and 128 registers: two workgroups per CU, one computing while the other is at
// its loads, first or last stage.
using Cfg256 = linear_cfg::Cfg<256, 256, 2>;
using Cfg128 = linear_cfg::Cfg<128, 128, 4>;

using LinearFn = void (*)(LinearGemmArgs);
template <bool BF16, class C> LinearFn pick_form(int form)
{
    switch (form) {
    case kFormNT: return ag_linear_gemm_kernel<BF16, kFormNT, C>;
    case kFormNN: return ag_linear_gemm_kernel<BF16, kFormNN, C>;
    case kFormTN: return ag_linear_gemm_kernel<BF16, kFormTN, C>;
    default: return nullptr;
    }
}

// ---------------------------------------------------------------- join of split products

// Adds the parts of 8 consecutive columns per thread in order, then the epilogue.
template <bool BF16>
__global__ __launch_bounds__(256) void ag_linear_join_kernel(LinearGemmArgs a)
{
    const int64_t per_row = a.partial_ld / 8;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t row = id / per_row, col = (id - row * per_row) * 8;
    if (row >= a.I || col >= a.J) return;
    const float* p = a.partial + row * a.partial_ld + col;
    const int64_t step = a.I * a.partial_ld;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
        const f32x4 lo = reinterpret_cast<const f32x4*>(p + s * step)[0];
        const f32x4 hi = reinterpret_cast<const f32x4*>(p + s * step)[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] += lo[e];
            v[4 + e] += hi[e];
        }
    }
    const int n = static_cast<int>(min(int64_t{8}, a.J - col));
    float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.epi.bias) load_f32<BF16>(bias, a.epi.bias + col, n);
    finish<BF16>(v, bias, a.epi, row, col, n);
}

// ---------------------------------------------------------------- a few rows of x

// y for up to 16 MB rows of x: the weights are streamed once, straight into matrix-instruction fragments,
// 16 rows of w per workgroup.  The workgroup's waves share the reduction, 128 wide at a time, and add up
// through LDS in a fixed order.  D rows are rows of w, D columns rows of x.
constexpr int kStreamWaves = 8;

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

template <bool BF16, int MB>
__global__ __launch_bounds__(64 * kStreamWaves) void ag_linear_stream_kernel(LinearStreamArgs a)
{
    using V = typename Mfma<BF16>::V;
    __shared__ f32x4 part[kStreamWaves][MB][64];
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

    int64_t k = wave * 128;
    for (; k + 128 <= a.K; k += kStreamWaves * 128) {
        V fw[4], fx[MB][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) fw[u] = __builtin_bit_cast(V, load8(w + k + u * 32));
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                fx[b][u] = zero;
                if (live[b]) fx[b][u] = __builtin_bit_cast(V, load8(x[b] + k + u * 32));
            }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int b = 0; b < MB; ++b) acc[b] = Mfma<BF16>::run(fw[u], fx[b][u], acc[b]);
    }
    if (k < a.K) {   // the last, shorter 128: one wave's
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
        for (int wv = 1; wv < kStreamWaves; ++wv) s += part[wv][b][l];
        const int64_t m = b * 16 + (l & 15), col = n0 + (l >> 4) * 4;
        const int n = static_cast<int>(max(int64_t{0}, min(int64_t{4}, a.N - col)));
        if (m < a.M && n > 0) {
            float v[8] = {s[0], s[1], s[2], s[3], 0.f, 0.f, 0.f, 0.f};
            float bias[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (a.epi.bias) load_f32<BF16>(bias, a.epi.bias + col, n);
            finish<BF16>(v, bias, a.epi, m, col, n);
        }
    }
}

// ---------------------------------------------------------------- rows to aligned rows

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

// 32 column groups of 8 x 8 row lanes; a workgroup takes 256 columns of kLinearSlopeRows rows.
template <bool BF16>
__global__ __launch_bounds__(256) void ag_linear_slope_kernel(LinearSlopeArgs a)
{
    __shared__ float part[8][264];
    const int c = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const uint32_t col_blocks = static_cast<uint32_t>((a.N + 255) / 256);
    const int64_t bx = blockIdx.x % col_blocks, by = blockIdx.x / col_blocks;
    const int64_t col = (bx * 32 + c) * 8;
    const int64_t row0 = by * kLinearSlopeRows;
    const int n = static_cast<int>(max(int64_t{0}, min(int64_t{8}, a.N - col)));
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (n > 0) {
#pragma unroll 4
        for (int i = rl; i < kLinearSlopeRows; i += 8) {
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

__global__ __launch_bounds__(256) void ag_linear_bias_grad_kernel(const float* sums, int64_t parts, int64_t N, void* db,
                                                                  int kind, int accumulate)
{
    __shared__ float part[8][33];
    const int c = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + c;
    float s = 0.f;
    if (col < N)
        for (int64_t q = rl; q < parts; q += 8) s += sums[q * N + col];
    part[rl][c] = s;
    __syncthreads();
    if (rl == 0 && col < N) {
        s = 0.f;
#pragma unroll
        for (int r = 0; r < 8; ++r) s += part[r][c];
        if (kind == 2) {
            float* p = static_cast<float*>(db) + col;
            *p = accumulate ? *p + s : s;
        } else {
            uint16_t* p = static_cast<uint16_t*>(db) + col;
            if (accumulate) s += kind == 1 ? to_f32<true>(*p) : to_f32<false>(*p);
            *p = kind == 1 ? from_f32<true>(s) : from_f32<false>(s);
        }
    }
}

}  // namespace

// ---------------------------------------------------------------- launchers

void linear_tile_shape(int tile, int* tm, int* tn, int* threads)
{
    *tm = tile == kLinearTile256 ? Cfg256::TM : Cfg128::TM;
    *tn = tile == kLinearTile256 ? Cfg256::TN : Cfg128::TN;
    *threads = Cfg256::NT;
}

hipError_t launch_linear_gemm(const LinearGemmArgs& a, int bf16, int form, int tile, hipStream_t stream)
{
    LinearFn fn = tile == kLinearTile256 ? (bf16 ? pick_form<true, Cfg256>(form) : pick_form<false, Cfg256>(form))
                                         : (bf16 ? pick_form<true, Cfg128>(form) : pick_form<false, Cfg128>(form));
    const int64_t grid = static_cast<int64_t>(a.tiles_i) * a.tiles_j * a.splits;
    if (fn == nullptr || grid < 1 || grid > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(grid)), dim3(Cfg256::NT), 0, stream, a);
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

hipError_t launch_linear_join(const LinearGemmArgs& a, int bf16, hipStream_t stream)
{
    dim3 grid;
    if (!grid_of(a.I * (a.partial_ld / 8), 256, &grid)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(bf16 ? ag_linear_join_kernel<true> : ag_linear_join_kernel<false>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_linear_stream(const LinearStreamArgs& a, int bf16, hipStream_t stream)
{
    dim3 grid;
    if (a.M < 1 || a.M > kLinearStreamRows || !grid_of(a.N, 16, &grid)) return hipErrorInvalidValue;
    auto fn = a.M <= 16 ? (bf16 ? ag_linear_stream_kernel<true, 1> : ag_linear_stream_kernel<false, 1>)
                        : (bf16 ? ag_linear_stream_kernel<true, 2> : ag_linear_stream_kernel<false, 2>);
    hipLaunchKernelGGL(fn, grid, dim3(64 * kStreamWaves), 0, stream, a);
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
    if (!grid_of((a.N + 255) / 256 * ((a.M + kLinearSlopeRows - 1) / kLinearSlopeRows), 1, &grid)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(bf16 ? ag_linear_slope_kernel<true> : ag_linear_slope_kernel<false>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_linear_bias_grad(const float* sums, int64_t parts, int64_t N, void* db, int db_kind, int accumulate,
                                   hipStream_t stream)
{
    dim3 grid;
    if (!grid_of(N, 32, &grid)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(ag_linear_bias_grad_kernel, grid, dim3(256), 0, stream, sums, parts, N, db, db_kind, accumulate);
    return hipGetLastError();
}

}  // namespace ag
