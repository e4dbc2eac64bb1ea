// Codes to values, for the sources that launch it alone or beside other work.
#pragma once

#include <hip/hip_runtime.h>

#include "ag.h"
#include "ag_rows.h"
#include "ag_scale.h"
#include "ag_vec.h"

namespace ag {
namespace {

// The values of codes: 8 to a lane, so that a wave's stores are whole lines; a thread takes kDequantizeVectors of them.  POWERS (bf16):
// the codes times the powers of two of their scales, and a.more copies of that.
template <int DTYPE, bool POWERS = false>
__device__ __forceinline__ void dequantize_body(const DequantizeArgs& a, uint32_t program, uint32_t programs)
{
    static_assert(!POWERS || DTYPE == AG_BF16, "fp16's powers depend on the gradients too");
    const uint32_t per_row = (static_cast<uint32_t>(a.K) + 7u) / 8u;
    const uint64_t vectors = static_cast<uint64_t>(a.M) * per_row;
    constexpr uint64_t PER = 256 * kDequantizeVectors;
    for (uint64_t from = program * PER; from < vectors; from += programs * PER) {
        u32x2 q[kDequantizeVectors];
        float s[kDequantizeVectors];
        int64_t row[kDequantizeVectors];
        int col[kDequantizeVectors];
#pragma unroll
        for (int j = 0; j < kDequantizeVectors; ++j) {
            const uint64_t id = min(from + j * 256 + threadIdx.x, vectors - 1);     // past the end: the last one again
            if (vectors >> 32) {
                row[j] = static_cast<int64_t>(id / per_row);
                col[j] = static_cast<int>(id - row[j] * per_row) * 8;
            } else {        // a division of 64 bits takes as long as the rest
                const uint32_t r = static_cast<uint32_t>(id) / per_row;
                row[j] = r;
                col[j] = static_cast<int>(static_cast<uint32_t>(id) - r * per_row) * 8;
            }
            const int8_t* at = a.q + row[j] * a.ldq + col[j];
            const int n = a.K - col[j];
            s[j] = a.scale[row[j]];
            q[j] = load_codes(at, n);
        }
#pragma unroll
        for (int j = 0; j < kDequantizeVectors; ++j) {
            if (from + j * 256 + threadIdx.x >= vectors) break;
            const int n = a.K - col[j];
            float scale = s[j], v[8];
            if constexpr (POWERS) {
                float rest;
                split_scale_bf16(s[j], &scale, &rest);
            }
            code_values(v, q[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= scale;
            const int64_t at = row[j] * a.ldy + col[j];
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
                store_16<DTYPE == AG_BF16>(static_cast<uint16_t*>(a.y) + at, v, n);
                if constexpr (POWERS) {
                    for (int c = 1; c <= a.more; ++c) store_16<DTYPE == AG_BF16>(static_cast<uint16_t*>(a.y) + at + c * a.M * a.ldy, v, n);
                }
            }
        }
    }
}

}  // namespace
}  // namespace ag
