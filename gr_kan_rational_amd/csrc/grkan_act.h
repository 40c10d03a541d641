// grkan_act.h -- the elementwise activations of the block operators (group
// norm, linear map with epilogue), forward and derivative, in fp32 registers.
//
//   none      h
//   silu      h s,  s = 1 / (1 + e^-h);          derivative s (1 + h (1 - s))
//   gelu      h Phi(h), Phi the normal distribution function (the exact form,
//             not the tanh approximation);       derivative Phi + h phi
//   rational  the group-rational F(h) = P / (1 + |Q|), degrees (5, 4)
//
// The activation is a run-time value but for the rational, which needs its
// coefficients in registers: RAT selects it at compile time.  The branch on
// the others is the same for every lane and costs nothing measurable beside
// the loads these kernels wait for.
#pragma once

#include "grkan.h"
#include "grkan_block.h"
#include "grkan_device.h"

namespace grkan {

constexpr float kLog2e = 1.44269504088896341f;

// 1 / (1 + e^-h): absolute error below 2^-22 (hardware base-2 exponential and
// reciprocal, 1 ulp each; the exponent's rounding, |h| 2^-24, meets a factor
// s (1 - s) that falls faster).  e^-h = inf gives 0.
__device__ static inline float sigmoid(float h) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * h));
}

// The normal distribution's Phi(h) and, in e, exp(-h^2 / 2).  With u = |h|,
// Phi(-u) = e t p(t), t = 1 / (1 + 0.38 u): a degree-9 polynomial fitted here
// (weighted least squares, iterated towards equal ripple) to
// erfcx(u / sqrt 2) / (2 t) over u in [0, 14], relative error 9e-9, 1e-7 when
// evaluated in fp32.  Beyond 14 e is 0 in fp32.  Phi(u) = 1 - Phi(-u).
__device__ static inline float normal_cdf(float h, float &e) {
    const float u = fabsf(h);
    e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * (h * h));
    const float t = __builtin_amdgcn_rcpf(fmaf(0.38f, u, 1.0f));
    float p = 0.02429252304136753f;
    p = fmaf(p, t, -0.1492505669593811f);
    p = fmaf(p, t, 0.3686513304710388f);
    p = fmaf(p, t, -0.4345865547657013f);
    p = fmaf(p, t, 0.2102862298488617f);
    p = fmaf(p, t, -0.055957868695259094f);
    p = fmaf(p, t, 0.10648509860038757f);
    p = fmaf(p, t, 0.12663328647613525f);
    p = fmaf(p, t, 0.1518578976392746f);
    p = fmaf(p, t, 0.15158861875534058f);
    const float tail = e * (t * p);
    return h < 0.0f ? tail : 1.0f - tail;
}

template <bool RAT>
__device__ static inline float act_value(float h, int act, const Coefs<5, 4> &c) {
    if constexpr (RAT) {
        return rational<5, 4>(h, c);
    } else {
        if (act == GRKAN_ACT_SILU) return h * sigmoid(h);
        if (act == GRKAN_ACT_GELU) {
            float e;
            return h * normal_cdf(h, e);
        }
        return h;
    }
}

// dy act'(h) for the activations without coefficients.
__device__ static inline float act_slope(float h, int act) {
    if (act == GRKAN_ACT_SILU) {
        const float s = sigmoid(h);
        return s * fmaf(h, 1.0f - s, 1.0f);
    }
    if (act == GRKAN_ACT_GELU) {
        float e;
        const float cdf = normal_cdf(h, e);
        return fmaf(h, e * 0.398942280401432678f, cdf);
    }
    return 1.0f;
}

// The rational's backward at an h that is itself the result of fp32
// arithmetic (a normalised value): dy dF/dh, the ten coefficient terms added
// to acc.  Q and its sign are taken in fp32 -- h carries its own rounding, so
// deciding the sign of Q more exactly than h is known would mean nothing --
// with sign(0) = 0.
__device__ static inline float rational_slope(float h, float dy, const Coefs<5, 4> &c, float (&acc)[10]) {
    float P = c.a[5], dP = 5.0f * c.a[5];
#pragma unroll
    for (int i = 4; i >= 0; --i) P = fmaf(P, h, c.a[i]);
#pragma unroll
    for (int i = 4; i >= 1; --i) dP = fmaf(dP, h, (float)i * c.a[i]);
    float q = c.b[3], dQ = 4.0f * c.b[3];
#pragma unroll
    for (int j = 2; j >= 0; --j) q = fmaf(q, h, c.b[j]);
#pragma unroll
    for (int j = 2; j >= 0; --j) dQ = fmaf(dQ, h, (float)(j + 1) * c.b[j]);
    const float Q = h * q;
    const float r = __builtin_amdgcn_rcpf(1.0f + fabsf(Q));
    const float w = dy * r;
    const float v = w * (P * r);
    float sv = Q == 0.0f ? 0.0f : __uint_as_float(__float_as_uint(v) ^ (__float_as_uint(Q) & 0x80000000u));
    const float dh = fmaf(-sv, dQ, w * dP);
    float p = w;
    acc[0] += p;
#pragma unroll
    for (int i = 1; i <= 5; ++i) {
        p *= h;
        acc[i] += p;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        sv *= h;
        acc[6 + j] -= sv;
    }
    return dh;
}

}  // namespace grkan
