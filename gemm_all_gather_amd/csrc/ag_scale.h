// A kept row's scale s in two factors: a power of two that goes to the codes, whose products with it are exact in 16 bits,
// and the rest, that goes to the row's gradient before its rounding.
#pragma once

#include <hip/hip_runtime.h>

namespace ag {
namespace {

// The exponent e with |v| < 2^e, and not below 2^(e-1) (-126 of what is smaller; 129 of a NaN or an infinity).
__device__ __forceinline__ int exponent_of(float v) { return static_cast<int>((__float_as_uint(v) >> 23) & 255u) - 126; }

__device__ __forceinline__ void split_at(float s, int exponent, float* power, float* rest)
{
    *power = __uint_as_float(static_cast<uint32_t>(exponent + 127) << 23);
    *rest = ldexpf(s, -exponent);
}

// bf16 has fp32's exponents: the rest is in [1/2, 1) for every normal scale, so that a gradient times it neither overflows nor loses
// bits.  128 times 2^119 is finite, and codes times 2^-126 are normal.
__device__ __forceinline__ void split_scale_bf16(float s, float* power, float* rest)
{
    split_at(s, min(max(exponent_of(s), -126), 119), power, rest);
}

// fp16 has 40 binades, and gradients of 1e-4 lie near their end: the rest takes the largest of the row's gradients, `top` for dy, into
// [2^13, 2^15) (no slope is above 1.13, so dz stays below 1.13 2^15), as far as the codes' power can make up for it.  That is 2^8 at
// most, codes up to 128 times which stay below 65504, and 2^-24 at least, fp16's smallest number.  Codes times less than 2^-14 may be
// subnormal, and the matrix instruction adds their products as if they were 2^-14 (six rows of them: 2^-24 of the sum of magnitudes
// to 2^-20, 2^-20 at 2^-24): below 2^-18 the gradients go down first, into [1/2, 2), where a second term still ends at 2^-24 of top.
__device__ __forceinline__ void split_scale_f16(float s, float top, float* power, float* rest)
{
    const int e = exponent_of(s) + max(exponent_of(top), -23) - 15;      // a row of zeros counts as fp16's smallest number
    split_at(s, e >= -18 ? min(e, 8) : max(min(e + 14, -18), -24), power, rest);
}

}  // namespace
}  // namespace ag
