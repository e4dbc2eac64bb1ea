// Elements of 16 bits in vectors of eight, at any alignment: loads, stores and roundings.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ag_mfma.h"

namespace ag {
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

// Eight 8-bit codes at any address.
struct __attribute__((packed, aligned(1))) Any8 { u32x2 v; };

__device__ __forceinline__ void code_values(float (&v)[8], u32x2 codes)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = static_cast<float>(static_cast<int8_t>(codes.x >> (8 * e)));
        v[4 + e] = static_cast<float>(static_cast<int8_t>(codes.y >> (8 * e)));
    }
}

// n <= 8 codes, the others 0.
__device__ __forceinline__ u32x2 load_codes(const int8_t* p, int n)
{
    if (n >= 8) return reinterpret_cast<const Any8*>(p)->v;
    uint64_t w = 0;
    for (int e = n - 1; e >= 0; --e) w = w << 8 | static_cast<uint8_t>(p[e]);
    return u32x2{static_cast<uint32_t>(w), static_cast<uint32_t>(w >> 32)};
}

}  // namespace
}  // namespace ag
