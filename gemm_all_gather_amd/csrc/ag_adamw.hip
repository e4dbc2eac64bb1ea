// AdamW over many tensors in one launch (gfx950).
//
// A workgroup takes one chunk of one tensor, found through a device table made with the handle.  A
// lane holds 8 consecutive elements, so that 32 lanes hold one block of 8-bit states and its maximum needs no
// LDS.  Every element is read once and written once.
//
// 32-bit states are bound by HBM: 117 million bf16 parameters with master weights (28 bytes each) take 623 us, 5.3 TB/s,
// a large copy's rate.  8-bit states (10 bytes each; 228 us at that rate) are bound by the vector pipe: about 72
// instructions an element, 5.5 of them square roots and reciprocals and 15 in fp64, 345 to 356 us.  The states are blended
// in fp64 and doubtful codes decided there, so that the codes are those of exact arithmetic (a blend in fp32 with its
// error added to what counts as doubtful would give the same codes; it is not built).  By the instructions'
// cycles 36% go into the blend and the update, 35% into the two codes, 29% into stochastic rounding's random bits.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ag.h"
#include "ag_adamw.h"

namespace ag {
namespace {

static_assert(AG_ADAMW_BLOCK == 256, "32 lanes of 8 elements");
static_assert(kAdamwChunk % (256 * 8) == 0, "whole passes of a workgroup");

// Vectors of 8 elements at any alignment of the element (global accesses need none on gfx950).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
struct __attribute__((packed, aligned(2))) Any16 { u32x4 v; };
struct __attribute__((packed, aligned(4))) Any16f { u32x4 v; };
struct __attribute__((packed, aligned(1))) Any8 { u32x2 v; };
// The table's addresses are global memory, which the compiler cannot know of a pointer read from memory (it
// would take the slower flat accesses, which count as LDS accesses too).
#define AG_GLOBAL __attribute__((address_space(1)))
template <class T> using Global = AG_GLOBAL T*;
template <class T, class P> __device__ __forceinline__ Global<T> global(P* p) { return (Global<T>)(p); }

template <int DT> struct Type;      // ag_dtype_t
template <> struct Type<AG_F32> {
    using T = float;
    static __device__ __forceinline__ void load(float (&x)[8], Global<const float> p)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 t = ((Global<const Any16f>)(p + 4 * h))->v;
#pragma unroll
            for (int e = 0; e < 4; ++e) x[4 * h + e] = __uint_as_float(t[e]);
        }
    }
    static __device__ __forceinline__ void store(Global<float> p, const float (&x)[8])
    {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            u32x4 t;
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = __float_as_uint(x[4 * h + e]);
            ((Global<Any16f>)(p + 4 * h))->v = t;
        }
    }
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};
template <bool BF16> struct Half {
    using T = uint16_t;
    static __device__ __forceinline__ float get(uint16_t v)
    {
        if constexpr (BF16) return __builtin_bit_cast(float, static_cast<uint32_t>(v) << 16);
        else return static_cast<float>(__builtin_bit_cast(_Float16, v));
    }
    static __device__ __forceinline__ uint16_t put(float v)    // to nearest, ties to even
    {
        if constexpr (BF16) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
        else return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
    }
    static __device__ __forceinline__ void load(float (&x)[8], Global<const uint16_t> p)
    {
        const u32x4 t = ((Global<const Any16>)p)->v;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = get(static_cast<uint16_t>(t[e / 2] >> (16 * (e & 1))));
    }
    static __device__ __forceinline__ void store(Global<uint16_t> p, const float (&x)[8])
    {
        u32x4 t;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            t[e] = static_cast<uint32_t>(put(x[2 * e])) | (static_cast<uint32_t>(put(x[2 * e + 1])) << 16);
        ((Global<Any16>)p)->v = t;
    }
};
template <> struct Type<AG_F16> : Half<false> {};
template <> struct Type<AG_BF16> : Half<true> {};

template <int DT>
__device__ __forceinline__ void load8(float (&x)[8], const void* base, int64_t at, int n)
{
    const Global<const typename Type<DT>::T> p = global<const typename Type<DT>::T>(base) + at;
    if (n >= 8) {
        Type<DT>::load(x, p);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = e < n ? Type<DT>::get(p[e]) : 0.f;
    }
}
template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&x)[8], int n)
{
    const Global<typename Type<DT>::T> p = global<typename Type<DT>::T>(base) + at;
    if (n >= 8) {
        Type<DT>::store(p, x);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = Type<DT>::put(x[e]);
    }
}
__device__ __forceinline__ uint64_t load_codes(const void* base, int64_t at, int n)
{
    const Global<const uint8_t> p = global<const uint8_t>(base) + at;
    if (n >= 8) return __builtin_bit_cast(uint64_t, ((Global<const Any8>)p)->v);
    uint64_t c = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) c |= static_cast<uint64_t>(p[e]) << (8 * e);
    return c;
}
__device__ __forceinline__ void store_codes(void* base, int64_t at, uint64_t c, int n)
{
    const Global<uint8_t> p = global<uint8_t>(base) + at;
    if (n >= 8) {
        ((Global<Any8>)p)->v = __builtin_bit_cast(u32x2, c);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = static_cast<uint8_t>(c >> (8 * e));
    }
}

// The step's scalars: the host's, or made anew from what device scalars hold.
__device__ __forceinline__ AdamwScalars scalars(const AdamwArgs& a)
{
    if (!a.dev_step && !a.dev_lr && !a.dev_grad_scale) return a.scalars;   // uniform
    double lr = a.lr, gs = a.grad_scale, bias1 = a.bias1, bias2 = a.bias2;
    AdamwScalars s = a.scalars;
    if (a.dev_step) {
        const int64_t step = *a.dev_step;
        s.seed = adamw_mix_seed(a.seed + static_cast<uint64_t>(step));
        bias1 = 1.0 - pow(a.beta1, static_cast<double>(step));
        bias2 = 1.0 - pow(a.beta2, static_cast<double>(step));
    }
    if (a.dev_lr) lr = *a.dev_lr;
    if (a.dev_grad_scale) gs *= *a.dev_grad_scale;
    s.decay = static_cast<float>(1.0 - lr * a.weight_decay);
    s.rate = static_cast<float>(lr / bias1);
    s.inv_bias2 = static_cast<float>(1.0 / bias2);
    s.grad_scale = static_cast<float>(gs);
    return s;
}

// The updates of 8 elements, square roots and quotients by the instructions' 1 ulp: 2^-21 of the step, below the
// parameter's own rounding.  The root instruction takes no subnormal numbers: against an eps of 1e-12 and more
// what it loses (below 1e-19) is nothing; with a smaller eps small arguments are scaled by 2^96 first.
__device__ __forceinline__ void update(float (&p)[8], const float (&m)[8], const float (&v)[8], const AdamwScalars& s)
{
    if (s.eps >= 1e-12f) {   // uniform
#pragma unroll
        for (int e = 0; e < 8; ++e)
            p[e] = p[e] * s.decay - s.rate * m[e] * __builtin_amdgcn_rcpf(__builtin_amdgcn_sqrtf(v[e] * s.inv_bias2) + s.eps);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = v[e] * s.inv_bias2;
            const bool small = x < 1e-30f;
            float r = __builtin_amdgcn_sqrtf(small ? x * 0x1p96f : x);
            r = small ? r * 0x1p-48f : r;
            p[e] = p[e] * s.decay - s.rate * m[e] / (r + s.eps);
        }
    }
}

// 32 random bits of the state element at place i (counted over all tensors' blocks): the two multiply and xor-shift
// rounds of a 32-bit mixer that Wellons found by search in 2018, with its multipliers and shifts.  The seed comes in
// mixed (adamw_mix_seed), half before and half between the rounds, so that seeds that count up give unrelated bits at
// every place.
__device__ __forceinline__ uint32_t random_bits(uint64_t mixed_seed, uint64_t i)
{
    uint32_t x = static_cast<uint32_t>(i) ^ (static_cast<uint32_t>(mixed_seed) + static_cast<uint32_t>(i >> 32) * 0x9E3779B1u);
    x = (x ^ (x >> 16)) * 0x7FEB352Du;
    x = (x ^ (x >> 15)) ^ static_cast<uint32_t>(mixed_seed >> 32);
    x = x * 0x846CA68Bu;
    return x ^ (x >> 16);
}

// The code floor(t + u), t = top * r^(1/POWER), of r = value / maximum in [0, 1], u in (0, 1) a multiple of 2^-17.
// guess() finds it in fp32: r is within 2^-22 of itself (value, reciprocal and product rounded), the roots within
// 2^-22 with it, so t + u within 1e-4 (255 (2^-22 + 2^-24) + 2^-16).  Where t + u lies closer than 1.25e-4 to a whole
// number, `near` is set and decide() says which side it is on in fp64, by comparing r top^POWER with (k - u)^POWER:
// the code is that of exact arithmetic, so it depends on no instruction's last bit.
template <int POWER>
__device__ __forceinline__ float guess(float value, float inverse, float u, bool& near)
{
    constexpr float top = POWER == 2 ? 127.f : 255.f;
    float t = __builtin_amdgcn_sqrtf(value * inverse);
    if (POWER == 4) t = __builtin_amdgcn_sqrtf(t);
    const float x = t * top + u;
    near = fabsf(x - rintf(x)) < 1.25e-4f;
    return fminf(floorf(x), top);
}
template <int POWER>
__device__ __forceinline__ float decide(double value, float maximum, float u)
{
    constexpr float top = POWER == 2 ? 127.f : 255.f;
    const double r = value / static_cast<double>(maximum);
    float t = __builtin_amdgcn_sqrtf(static_cast<float>(r));
    if (POWER == 4) t = __builtin_amdgcn_sqrtf(t);
    const float x = t * top + u, k = rintf(x);
    if (!(fabsf(x - k) < 1.25e-4f)) return fminf(floorf(x), top);
    const double b = static_cast<double>(k) - static_cast<double>(u), b2 = b * b;
    const bool reached = b <= 0.0 || (POWER == 2 ? r * (127.0 * 127.0) >= b2 : r * (255.0 * 255.0 * 255.0 * 255.0) >= b2 * b2);
    return fminf(reached ? k : k - 1.f, top);
}

// Largest of the 32 lanes of a block.  Bit patterns of non-negative floats compare as integers, and a NaN's is above all.
template <int CTRL> __device__ __forceinline__ uint32_t max_dpp(uint32_t v)
{
    const uint32_t o = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, true));
    return v > o ? v : o;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v)
{
    v = max_dpp<0xB1>(v);       // quad_perm 1 0 3 2
    v = max_dpp<0x4E>(v);       // quad_perm 2 3 0 1
    v = max_dpp<0x141>(v);      // row_half_mirror
    v = max_dpp<0x140>(v);      // row_mirror
    const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(v, v, false, false));   // rows 0 and 1, 2 and 3
    return t.x > t.y ? t.x : t.y;
}
constexpr uint32_t kInfBits = 0x7f800000u;

constexpr double kCodeM = 1.0 / (127.0 * 127.0), kCodeV = 1.0 / (255.0 * 255.0 * 255.0 * 255.0);

// beta x + y, each operation rounded to fp64 by itself.  A block's maximum often lies exactly between two
// fp32 numbers (0.9 S + 0.1 g of short significands); its side, and with it the codes' scale, is then the
// rounding's, and a fused operation's would differ from what the same formula gives elsewhere.
__device__ __forceinline__ double blend(double beta, double x, double y)
{
#pragma clang fp contract(off)
    const double bx = beta * x;
    return bx + y;
}

template <int P, int G, bool MASTER, bool S8>
__global__ __launch_bounds__(256) void ag_adamw_kernel(AdamwArgs a)
{
    const AdamwChunk c = a.chunks[blockIdx.x];
    const AdamwEntry t = a.entries[c.tensor];
    const AdamwScalars s = scalars(a);
#pragma unroll
    for (int pass = 0; pass < kAdamwChunk / 2048; ++pass) {
        const int64_t at = static_cast<int64_t>(c.chunk) * kAdamwChunk + pass * 2048 + threadIdx.x * 8;
        // lanes past the end take part in their block's maximum with zeros
        const int64_t left = t.n - at;
        const int n = static_cast<int>(left < 0 ? 0 : left > 8 ? 8 : left);
        if (!S8 && n == 0) return;
        float p[8], g[8];
        load8<G>(g, t.grad, n ? at : 0, n);
        if constexpr (MASTER) load8<AG_F32>(p, t.master, n ? at : 0, n);
        else load8<P>(p, t.param, n ? at : 0, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] *= s.grad_scale;

        if constexpr (!S8) {
            float m[8], v[8];
            load8<AG_F32>(m, t.exp_avg, at, n);
            load8<AG_F32>(v, t.exp_avg_sq, at, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                m[e] = s.b1 * m[e] + s.one_minus_b1 * g[e];
                v[e] = s.b2 * v[e] + s.one_minus_b2 * g[e] * g[e];
            }
            update(p, m, v, s);
            store8<AG_F32>(t.exp_avg, at, m, n);
            store8<AG_F32>(t.exp_avg_sq, at, v, n);
        } else {
            const int64_t block = at / AG_ADAMW_BLOCK;
            const bool block_live = block * AG_ADAMW_BLOCK < t.n;
            const uint64_t mc = load_codes(t.exp_avg, n ? at : 0, n), vc = load_codes(t.exp_avg_sq, n ? at : 0, n);
            const double ms = block_live ? global<const float>(t.exp_avg_scale)[block] * kCodeM : 0.0;
            const double vs = block_live ? global<const float>(t.exp_avg_sq_scale)[block] * kCodeV : 0.0;
            double m[8], v[8];
            float mf[8], vf[8];
            uint32_t mmax = 0, vmax = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // c |c| and c^2 are exact in fp32, c^4 in fp64
                const float cm = static_cast<float>(static_cast<int8_t>(mc >> (8 * e)));
                const float cv = static_cast<float>(static_cast<uint8_t>(vc >> (8 * e)));
                const double cv2 = static_cast<double>(cv * cv);
                m[e] = blend(a.beta1, static_cast<double>(cm * fabsf(cm)) * ms, a.one_minus_beta1 * g[e]);
                v[e] = blend(a.beta2, cv2 * cv2 * vs, a.one_minus_beta2 * g[e] * g[e]);
                mf[e] = static_cast<float>(m[e]);
                vf[e] = static_cast<float>(v[e]);
                const uint32_t mb = __float_as_uint(mf[e]) & 0x7fffffffu, vb = __float_as_uint(vf[e]) & 0x7fffffffu;
                mmax = mmax > mb ? mmax : mb;
                vmax = vmax > vb ? vmax : vb;
            }
            update(p, mf, vf, s);
            mmax = block_max(mmax);
            vmax = block_max(vmax);
            // a block that holds an infinity or a NaN reads back as NaN: all codes 0, the maximum NaN
            const bool mfine = mmax < kInfBits, vfine = vmax < kInfBits;
            const float mS = mfine ? __uint_as_float(mmax) : __builtin_nanf("");
            const float vS = vfine ? __uint_as_float(vmax) : __builtin_nanf("");
            // a maximum so small that its reciprocal would overflow leaves the codes to decide()
            const float mi = mfine && mS > 1e-30f ? __builtin_amdgcn_rcpf(mS) : 0.f;
            const float vi = vfine && vS > 1e-30f ? __builtin_amdgcn_rcpf(vS) : 0.f;
            const bool mtiny = mfine && mmax != 0 && mi == 0.f, vtiny = vfine && vmax != 0 && vi == 0.f;
            float km[8], kv[8], um[8], uv[8];
            bool near_m[8], near_v[8], any = false;     // codes for decide()
            const uint64_t place = (static_cast<uint64_t>(t.first_block) * AG_ADAMW_BLOCK) + static_cast<uint64_t>(at);
#pragma unroll
            for (int e = 0; e < 8; ++e) um[e] = uv[e] = 0.5f;
            if (a.stochastic) {   // uniform
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t bits = random_bits(s.seed, place + e);
                    um[e] = static_cast<float>(2 * (bits & 0xffffu) + 1) * (1.f / 131072.f);
                    uv[e] = static_cast<float>(2 * (bits >> 16) + 1) * (1.f / 131072.f);
                }
            }
            const bool mlive = mfine && mmax != 0, vlive = vfine && vmax != 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                km[e] = guess<2>(fabsf(mf[e]), mi, um[e], near_m[e]);
                kv[e] = guess<4>(vf[e], vi, uv[e], near_v[e]);
                any |= near_m[e] | near_v[e];
            }
            if (__any(any | mtiny | vtiny)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if ((near_m[e] | mtiny) & mlive) km[e] = decide<2>(fabs(m[e]), mS, um[e]);
                    if ((near_v[e] | vtiny) & vlive) kv[e] = decide<4>(v[e], vS, uv[e]);
                }
            }
            uint32_t mo[2] = {0, 0}, vo[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                kv[e] = v[e] > 0.0 ? fmaxf(kv[e], 1.f) : kv[e];
                const int cm = static_cast<int>(copysignf(km[e], mf[e])), cv = static_cast<int>(kv[e]);
                mo[e / 4] |= (static_cast<uint32_t>(cm) & 0xffu) << (8 * (e % 4));
                vo[e / 4] |= static_cast<uint32_t>(cv) << (8 * (e % 4));
            }
            if (!mfine) mo[0] = mo[1] = 0;
            if (!vfine) vo[0] = vo[1] = 0;
            store_codes(t.exp_avg, at, mo[0] | static_cast<uint64_t>(mo[1]) << 32, n);
            store_codes(t.exp_avg_sq, at, vo[0] | static_cast<uint64_t>(vo[1]) << 32, n);
            if (block_live && (threadIdx.x & 31) == 0) {
                global<float>(t.exp_avg_scale)[block] = mS;
                global<float>(t.exp_avg_sq_scale)[block] = vS;
            }
        }
        if constexpr (MASTER) store8<AG_F32>(t.master, at, p, n);
        store8<P>(t.param, at, p, n);
    }
}

// The values that codes stand for, 8 per lane: bound by its writes of 8 bytes an element (117 million elements 225 us,
// 5.2 TB/s).
__global__ __launch_bounds__(256) void ag_adamw_read_kernel(AdamwReadArgs a)
{
    int lo = 0, hi = a.count;                 // the tensor whose groups hold this one
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.first_group[mid] <= blockIdx.x) lo = mid;
        else hi = mid;
    }
    const AdamwEntry t = a.entries[lo];
    float* mo = a.exp_avg[lo];
    float* vo = a.exp_avg_sq[lo];
    const int64_t at = (static_cast<int64_t>(blockIdx.x - a.first_group[lo]) * 256 + threadIdx.x) * 8;
    const int64_t left = t.n - at;
    if (left <= 0) return;
    const int n = static_cast<int>(left > 8 ? 8 : left);
    const uint64_t mc = load_codes(t.exp_avg, at, n), vc = load_codes(t.exp_avg_sq, at, n);
    const double ms = global<const float>(t.exp_avg_scale)[at / AG_ADAMW_BLOCK] * kCodeM;
    const double vs = global<const float>(t.exp_avg_sq_scale)[at / AG_ADAMW_BLOCK] * kCodeV;
    float m[8], v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int cm = static_cast<int8_t>(mc >> (8 * e));
        const uint32_t cv = static_cast<uint32_t>(vc >> (8 * e)) & 0xffu;
        m[e] = static_cast<float>(static_cast<double>(cm * abs(cm)) * ms);
        v[e] = static_cast<float>(static_cast<double>(cv * cv * cv * cv) * vs);
    }
    store8<AG_F32>(mo, at, m, n);
    store8<AG_F32>(vo, at, v, n);
}

using AdamwFn = void (*)(AdamwArgs);
template <int P, int G> AdamwFn pick_state(bool master, bool s8)
{
    if constexpr (P == AG_F32) {
        if (master) return nullptr;
        return s8 ? ag_adamw_kernel<P, G, false, true> : ag_adamw_kernel<P, G, false, false>;
    } else {
        if (master) return s8 ? ag_adamw_kernel<P, G, true, true> : ag_adamw_kernel<P, G, true, false>;
        return s8 ? ag_adamw_kernel<P, G, false, true> : ag_adamw_kernel<P, G, false, false>;
    }
}
template <int P> AdamwFn pick_grad(int g, bool master, bool s8)
{
    switch (g) {
    case AG_F16: return pick_state<P, AG_F16>(master, s8);
    case AG_BF16: return pick_state<P, AG_BF16>(master, s8);
    case AG_F32: return pick_state<P, AG_F32>(master, s8);
    default: return nullptr;
    }
}

}  // namespace

hipError_t launch_adamw(const AdamwLaunch& l, hipStream_t stream)
{
    AdamwFn fn = nullptr;
    switch (l.param) {
    case AG_F16: fn = pick_grad<AG_F16>(l.grad, l.master != 0, l.state8 != 0); break;
    case AG_BF16: fn = pick_grad<AG_BF16>(l.grad, l.master != 0, l.state8 != 0); break;
    case AG_F32: fn = pick_grad<AG_F32>(l.grad, l.master != 0, l.state8 != 0); break;
    default: break;
    }
    if (fn == nullptr || l.chunks < 1 || l.chunks > 0x7fffffff) return hipErrorInvalidValue;
    hipLaunchKernelGGL(fn, dim3(static_cast<uint32_t>(l.chunks)), dim3(256), 0, stream, l.args);
    return hipGetLastError();
}

hipError_t launch_adamw_read(const AdamwReadArgs& a, hipStream_t stream)
{
    const uint32_t groups = a.first_group[a.count];
    if (a.count < 1 || groups < 1) return hipErrorInvalidValue;
    hipLaunchKernelGGL(ag_adamw_read_kernel, dim3(groups), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace ag
