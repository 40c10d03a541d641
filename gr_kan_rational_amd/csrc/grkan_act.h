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

// The rational's backward: dy dF/dh, the ten coefficient terms added to acc.
// The powers of h serve the polynomials and the sums (46 instructions; Horner's
// rule with running products for the sums takes 51).  Two forms of Q, by the
// coefficients' type:
//
// SlopeCoefs: h is itself the result of fp32 arithmetic (a normalised value).
// Q and its sign are taken in fp32, with sign(0) = 0: h's own rounding moves Q
// by up to sum j |b_j h^j| 2^-24, as much as the evaluation does, so a better Q
// at a rounded h gains nothing (over six sets of coefficients with real roots of
// Q, dB was off by 1e-7 .. 3e-5 either way, by less with Q in fp64 in two sets
// and by more in four).
//
// ExactSlopeCoefs: h is an exact input (a kept bf16 product).  Then Q's rounding
// is the whole error of D next to a root of Q, and since bf16 values recur it
// does not average out over the rows: with Q in fp32 dB was 1.6 to 34 times
// farther from its fp64 value than with Q as here, by Horner's rule in fp64
// from exact copies, rounded once, as in the activation's own backward (six sets
// as above; four fp64 instructions and two conversions in place of four in
// fp32, at the same rate).  The sign of Q is proven by that backward's guard
// (BwdCoefs), |Q| > 2^-46 (sum |b_j|) (1 + h^4); the rare element within it (h =
// 0 among them) takes the compensated decision.
struct SlopeCoefs {
    static constexpr bool kExact = false;
    Coefs<5, 4> c;
    float da[4], db[3];  // 2 a_2 .. 5 a_5, 2 b_2 .. 4 b_4
    __device__ inline void init(const Coefs<5, 4> &k) {
        c = k;
#pragma unroll
        for (int i = 2; i <= 5; ++i) da[i - 2] = (float)i * k.a[i];
#pragma unroll
        for (int j = 2; j <= 4; ++j) db[j - 2] = (float)j * k.b[j - 1];
    }
};
struct ExactSlopeCoefs : SlopeCoefs {
    static constexpr bool kExact = true;
    QWide<4> wide;
    float guard;
    __device__ inline void init(const Coefs<5, 4> &k) {
        SlopeCoefs::init(k);
        wide = widen<5, 4, false>(k);  // the columns, and with them the group, differ between lanes
        guard = fmaxf((fabsf(k.b[0]) + fabsf(k.b[1]) + fabsf(k.b[2]) + fabsf(k.b[3])) * sign_guard_scale<4>(), kGuardFloor);
    }
};

template <class K>
__device__ static inline float rational_slope(float h, float dy, const K &k, float (&acc)[10]) {
    // One element after another (the asm ties h to every sum so far): left
    // alone, the compiler puts the sums off and holds the powers of all of a
    // lane's elements (270 registers for 12 of them).
    asm volatile("" : "+v"(h) : "v"(acc[0]), "v"(acc[1]), "v"(acc[2]), "v"(acc[3]), "v"(acc[4]), "v"(acc[5]), "v"(acc[6]),
                 "v"(acc[7]), "v"(acc[8]), "v"(acc[9]));
    const float *a = k.c.a, *b = k.c.b;
    const float h2 = h * h, h3 = h2 * h, h4 = h2 * h2, h5 = h4 * h;
    const float P = fmaf(a[5], h5, fmaf(a[4], h4, fmaf(a[3], h3, fmaf(a[2], h2, fmaf(a[1], h, a[0])))));
    const float dP = fmaf(k.da[3], h4, fmaf(k.da[2], h3, fmaf(k.da[1], h2, fmaf(k.da[0], h, a[1]))));
    float Q;
    if constexpr (K::kExact) {
        const double hd = (double)h;
        Q = (float)(hd * fma(fma(fma(k.wide.b[3], hd, k.wide.b[2]), hd, k.wide.b[1]), hd, k.wide.b[0]));
    } else {
        Q = fmaf(b[3], h4, fmaf(b[2], h3, fmaf(b[1], h2, b[0] * h)));
    }
    const float dQ = fmaf(k.db[2], h3, fmaf(k.db[1], h2, fmaf(k.db[0], h, b[0])));
    const float r = __builtin_amdgcn_rcpf(1.0f + fabsf(Q));
    const float w = dy * r;
    const float v = w * (P * r);
    float sv = __uint_as_float(__float_as_uint(v) ^ (__float_as_uint(Q) & 0x80000000u));
    if constexpr (!K::kExact) {
        sv = Q == 0.0f ? 0.0f : sv;
    } else if (!(fabsf(Q) > fmaf(h4, k.guard, k.guard))) {
        const bool zero = h == 0.0f || (b[0] == 0.0f && b[1] == 0.0f && b[2] == 0.0f && b[3] == 0.0f);
        const int s = zero ? 0 : qsign_compensated<4>(h, k.c.b) * (h > 0.0f ? 1 : -1);
        sv = s == 0 ? 0.0f * v : (s > 0 ? v : -v);
    }
    acc[0] += w;
    acc[1] = fmaf(w, h, acc[1]);
    acc[2] = fmaf(w, h2, acc[2]);
    acc[3] = fmaf(w, h3, acc[3]);
    acc[4] = fmaf(w, h4, acc[4]);
    acc[5] = fmaf(w, h5, acc[5]);
    acc[6] = fmaf(-sv, h, acc[6]);
    acc[7] = fmaf(-sv, h2, acc[7]);
    acc[8] = fmaf(-sv, h3, acc[8]);
    acc[9] = fmaf(-sv, h4, acc[9]);
    return fmaf(-sv, dQ, w * dP);
}

}  // namespace grkan
