// Device building blocks of the linear layer's matrix kernels: buffer descriptors, waits on single counters,
// and the 16x16x32 matrix instruction of each 16-bit type.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#define AG_LDS __attribute__((address_space(3)))

namespace ag {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

__device__ inline __amdgpu_buffer_rsrc_t make_rsrc(uint64_t base, uint32_t records)
{
    constexpr int kRawBufferWord3 = 0x00020000;
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), static_cast<short>(0),
                                             static_cast<int>(records), kRawBufferWord3);
}

// s_waitcnt with only the vector-memory counter limited (gfx9 encoding).
template <int N>
__device__ inline void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
__device__ inline void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt(0xC07F); }

template <bool BF16> struct Mfma;
template <> struct Mfma<false> {
    using V = f16x8;
    static __device__ f32x4 run(V a, V b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
};
template <> struct Mfma<true> {
    using V = bf16x8;
    static __device__ f32x4 run(V a, V b, f32x4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
};

}  // namespace
}  // namespace ag
