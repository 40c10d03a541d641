// grkan_e4m3.h -- e4m3 codes (4 exponent bits, 3 of mantissa, bias 7, largest
// value 448, no infinity, 0x7f a NaN) and the power-of-two scales of blocks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace grkan {

// |v| if v is finite, else 0.
__device__ static inline float finite_size(float v) {
    const float a = fabsf(v);
    return a < __builtin_inff() ? a : 0.0f;
}

// The smallest 2^e, e >= -126, with amax <= 448 * 2^e; 1 for amax = 0.  448 is
// 1.75 * 2^8: e is amax's exponent less 8, one more for a mantissa above 1.75.
// Subnormal amax has exponent field 0 and takes the least scale.
__device__ static inline float block_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);
    e = e < 1 ? 1 : e;
    return u == 0 ? 1.0f : __uint_as_float((uint32_t)e << 23);
}

// 1 / s for a scale s (a power of two from 2^-126 to 2^120): exact.
__device__ static inline float inverse_scale(float s) { return __uint_as_float(0x7f000000u - __float_as_uint(s)); }

// Codes of four values, rounded to nearest even; |v| <= 448 or not finite (a
// NaN's code: the conversion's own for a NaN, an infinity made one first).
__device__ static inline uint32_t encode4(float a, float b, float c, float d) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
__device__ static inline float scaled(float v, float inv) {
    return fabsf(v) < __builtin_inff() ? v * inv : __builtin_nanf("");
}
typedef unsigned int codes8 __attribute__((ext_vector_type(2)));
__device__ static inline codes8 encode8(const float (&v)[8], float inv) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = scaled(v[e], inv);
    return codes8{encode4(y[0], y[1], y[2], y[3]), encode4(y[4], y[5], y[6], y[7])};
}

}  // namespace grkan
