// grkan_lanes.h -- sums and maxima over the lanes of a wave, and vector
// accesses of a few I/O elements, for the operators of grkan_train.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grkan_device.h"

namespace grkan {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// v of the lane that the DPP control names (every lane names one).
template <int CTRL> __device__ static inline float lane_of(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// Over 16 lanes side by side, the result in each: quads by permutation, then
// the mirrored half and the mirrored whole.
__device__ static inline float sum16(float v) {
    v += lane_of<0xb1>(v);
    v += lane_of<0x4e>(v);
    v += lane_of<0x141>(v);
    v += lane_of<0x140>(v);
    return v;
}
__device__ static inline float max16(float v) {
    v = fmaxf(v, lane_of<0xb1>(v));
    v = fmaxf(v, lane_of<0x4e>(v));
    v = fmaxf(v, lane_of<0x141>(v));
    v = fmaxf(v, lane_of<0x140>(v));
    return v;
}

// Over the 64 lanes of a wave, the same bits in each: swapping the odd rows of 16
// of one copy with the even rows of another leaves each pair of rows side by
// side in both, the halves likewise.
__device__ static inline float sum64(float v) {
    v = sum16(v);
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// One I/O element.
__device__ static inline float load1(const float *p) { return *p; }
__device__ static inline float load1(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ static inline void store1(float *p, float v) { *p = v; }
__device__ static inline void store1(uint16_t *p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

// Four I/O elements side by side, of which the first nv (0..4) exist (the others
// read as 0). VEC: p is aligned to the four, nv is 4 or at most 0.
template <bool VEC> __device__ static inline f32x4 load4(const float *p, int nv) {
    if constexpr (VEC) return nv > 0 ? *reinterpret_cast<const f32x4 *>(p) : f32x4{};
    f32x4 v = {};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < nv) v[e] = p[e];
    return v;
}
template <bool VEC> __device__ static inline f32x4 load4(const uint16_t *p, int nv) {
    f32x4 v = {};
    if constexpr (VEC) {
        if (nv <= 0) return v;
        const u32x2 w = *reinterpret_cast<const u32x2 *>(p);
        return f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                     __uint_as_float(w[1] & 0xffff0000u)};
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < nv) v[e] = load1(p + e);
    return v;
}
template <bool VEC> __device__ static inline void store4(float *p, int nv, f32x4 v) {
    if constexpr (VEC) {
        if (nv > 0) *reinterpret_cast<f32x4 *>(p) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < nv) p[e] = v[e];
}
__device__ static inline u32x2 pack4(f32x4 v) {
    const f32x2 a = {v[0], v[1]}, b = {v[2], v[3]};
    return u32x2{__builtin_bit_cast(unsigned int, __builtin_convertvector(a, bf16x2)),
                 __builtin_bit_cast(unsigned int, __builtin_convertvector(b, bf16x2))};
}
template <bool VEC> __device__ static inline void store4(uint16_t *p, int nv, f32x4 v) {
    if constexpr (VEC) {
        if (nv > 0) *reinterpret_cast<u32x2 *>(p) = pack4(v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < nv) store1(p + e, v[e]);
}

}  // namespace grkan
