// Vectors of eight elements of a row as they lie in memory.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ag.h"
#include "ag_vec.h"

namespace ag {
namespace {

template <int DTYPE> __device__ __forceinline__ const void* row_of(const void* p, int64_t row, int64_t ld)
{
    return static_cast<const char*>(p) + row * ld * (DTYPE == AG_F32 ? 4 : 2);
}

// Eight elements as they lie in memory: loaded early, and taken apart where they are used (a conversion next to its load
// waits for it, one vector after the other).
template <int DTYPE> struct Raw {
    u32x4 v;            // pairs in words: as eight elements the compiler would keep eight registers
    // The elements of a row of K from col on (TAIL false: K is a multiple of 8), those past its end 0.  A row's last, shorter vector is loaded as its last eight
    // elements, moved down: one load instead of up to seven.
    template <bool TAIL> __device__ __forceinline__ void load(const void* row, int col, int K)
    {
        const uint16_t* s = static_cast<const uint16_t*>(row);
        const int n = K - col;
        v = u32x4{0u, 0u, 0u, 0u};
        if (n >= 8) {
            v = reinterpret_cast<const Any16*>(s + col)->v;
        } else if (TAIL && n > 0) {
            uint64_t lo = 0, hi = 0;
            if (K >= 8) {
                const u32x4 t = reinterpret_cast<const Any16*>(s + (K - 8))->v;
                lo = static_cast<uint64_t>(t.y) << 32 | t.x;
                hi = static_cast<uint64_t>(t.w) << 32 | t.z;
                const int bits = 16 * (8 - n);      // 16 to 112
                const bool far = bits >= 64;
                lo = far ? hi >> (bits - 64) : lo >> bits | hi << (64 - bits);
                hi = far ? 0 : hi >> bits;
            } else {
#pragma unroll 1
                for (int e = n - 1; e >= 0; --e) {
                    hi = hi << 16 | lo >> 48;
                    lo = lo << 16 | s[col + e];
                }
            }
            v = u32x4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi), static_cast<uint32_t>(hi >> 32)};
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8])       // rounded
    {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = static_cast<uint32_t>(from_f32<DTYPE == AG_BF16>(f[2 * e + 1])) << 16 | from_f32<DTYPE == AG_BF16>(f[2 * e]);
    }
    __device__ __forceinline__ void store(void* p, int64_t at, int n) const
    {
        uint16_t* s = static_cast<uint16_t*>(p) + at;
        if (n >= 8) {
            reinterpret_cast<Any16*>(s)->v = v;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) s[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
        }
    }
    __device__ __forceinline__ void ones()
    {
        const uint32_t one = DTYPE == AG_BF16 ? 0x3f80u : 0x3c00u;
        v = u32x4{one << 16 | one, one << 16 | one, one << 16 | one, one << 16 | one};
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        u32x4 w = v;
        asm volatile("" : "+v"(w));     // taken apart here: not at the load, nor once before a loop
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = to_f32<DTYPE == AG_BF16>(static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1))));
    }
};
template <> struct Raw<AG_F32> {
    f32x4u lo, hi;
    template <bool TAIL> __device__ __forceinline__ void load(const void* row, int col, int K)
    {
        const float* s = static_cast<const float*>(row) + col;
        const int n = K - col;
        lo = hi = f32x4u{0.f, 0.f, 0.f, 0.f};
        if (n >= 8) {
            lo = *reinterpret_cast<const f32x4u*>(s);
            hi = *reinterpret_cast<const f32x4u*>(s + 4);
        } else if (TAIL && n > 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) (e < 4 ? lo : hi)[e & 3] = s[e];
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = lo[e];
            f[4 + e] = hi[e];
        }
    }
};

}  // namespace
}  // namespace ag
