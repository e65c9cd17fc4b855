// fp8_device.hpp -- float32 results to E4M3 codes with one power-of-two scale
// per 32 values, the format of the dispatch payload's rows (fp8.hip), whose
// values are rounded once, from float32 to their codes; and the encoder alone,
// for weights (quantize_weights.hip).
#pragma once

#include "device.hpp"

namespace moe {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// smallest e >= -127 with a <= 448 * 2^e, a >= 0: a = 1.m * 2^(be - 127) fits
// 448 * 2^e = 1.75 * 2^(e + 8) when e = be - 135, or needs one more when the
// mantissa exceeds 0.75. An infinite a gives 120.
__device__ __forceinline__ int32_t fp8_exponent(float a)
{
    const uint32_t bits = __float_as_uint(a);
    return max(-127, (int32_t)(bits >> 23) - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0));
}

// 2^-e for e in [-127, 121]
__device__ __forceinline__ float fp8_multiplier(int32_t e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// four values * mul -> four codes, rounded to nearest even; NaN and infinities
// give the NaN code. Where mul is a power of two, as of the rows, the products
// are exact (a product below float32's normal range lies far below E4M3's
// smallest code); by a weights' 1 / scale they are rounded to float32 first.
__device__ __forceinline__ uint32_t fp8_encode4(float a, float b, float c, float d, float mul)
{
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * mul, b * mul, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * mul, d * mul, w, true);
}

// largest magnitude; NaN does not count
__device__ __forceinline__ float max_abs(float m, float v) { return fmaxf(m, fabsf(v)); }

}  // namespace
}  // namespace moe
