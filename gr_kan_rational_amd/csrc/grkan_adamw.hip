// grkan_adamw.hip -- the AdamW step over many tensors in one launch, states in
// 32 bits or 8 (gfx950).
//
// The tensors' addresses travel as the kernel's arguments; a workgroup takes 4,096
// elements of one tensor, which it finds from the first workgroups of all (one per
// lane).  Bound: memory with 32-bit states (57 million parameters in bf16 with masters
// 332 us, 5.1 TB/s); with 8-bit ones vector arithmetic beside it, 105 instructions a value
// (division, root, hash, two roundings; busy 0.73), 246 us, 4.2 TB/s.
#include "grkan_adamw.h"

#include <type_traits>

#include "grkan_e4m3.h"
#include "grkan_lanes.h"

namespace grkan {
namespace {

__device__ static inline uint32_t mix(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x6A09E667u;
    h = (h ^ (h >> 15)) * 0xBB67AE85u;
    return h ^ (h >> 16);
}

// beta^step by squaring.
__host__ __device__ static inline double power(double beta, int64_t step) {
    double p = 1.0;
    for (uint64_t k = (uint64_t)step; k; k >>= 1, beta *= beta)
        if (k & 1) p *= beta;
    return p;
}

// The same on the host and on the device: a step that is known before the launch
// has them among the kernel's arguments (on the device they take 4 us of a workgroup's
// time).
__host__ __device__ static inline AdamwFactors factors(double lr, double beta1, double beta2, double decay, double eps,
                                                       int64_t step) {
#pragma clang fp contract(off)
    AdamwFactors f;
    f.beta1 = (float)beta1;
    f.rest1 = (float)(1.0 - beta1);
    f.beta2 = (float)beta2;
    f.rest2 = (float)(1.0 - beta2);
    f.keep = (float)(1.0 - lr * decay);
    f.rate = (float)(lr / (1.0 - power(beta1, step)));
    f.root = (float)(1.0 / sqrt(1.0 - power(beta2, step)));
    f.eps = (float)eps;
    return f;
}

// One value; m is the first moment, v the second.  Each operation is rounded
// by itself.
__device__ static inline float update(const AdamwFactors &f, bool clip, float scale, float w, float g, float &m, float &v) {
#pragma clang fp contract(off)
    if (clip) g = g * scale;
    m = f.beta1 * m + f.rest1 * g;
    v = f.beta2 * v + f.rest2 * g * g;
    const float d = sqrtf(v) * f.root + f.eps;
    return w * f.keep - f.rate * (m / d);
}

// y (|y| <= 448) to an e4m3 value, up with the probability of the remainder; the
// 16 random bits stand at bits 4 to 19, below the 3 bits of mantissa that are
// kept.  Below 2^-6 the values are multiples of 2^-9: adding 2^-6 puts them where
// that is the last bit kept.
__device__ static inline float round_up_sometimes(float y, uint32_t random16) {
#pragma clang fp contract(off)
    const float a = fabsf(y), low = a < 0.015625f ? 0.015625f : 0.0f;
    const uint32_t bits = __float_as_uint(a + low) + (random16 << 4 | 8u);
    return copysignf(__uint_as_float(bits & 0xfff00000u) - low, y);
}

// The weights to step: the master's, but where the parameter is not the master rounded it has
// been written by another (loaded, clamped, set anew) and counts.
template <class T> __device__ static inline f32x4 latest(f32x4 master, f32x4 param) {
    f32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float rounded = sizeof(T) == 2 ? (float)(__bf16)master[e] : master[e];
        w[e] = rounded == param[e] ? master[e] : param[e];
    }
    return w;
}

template <class T, bool VEC>
__device__ static inline void step32(const AdamwArgs &a, const AdamwTensor &t, const AdamwFactors &f, float scale, int64_t base) {
#pragma unroll
    for (int i = 0; i < kAdamwChunk / 1024; ++i) {
        const int64_t at = base + 1024 * i + 4 * (int)threadIdx.x;
        const int nv = (int)min(t.n - at, (int64_t)4);
        if (nv <= 0) continue;
        const bool whole = VEC && nv == 4;
        T *param = static_cast<T *>(t.param) + at;
        const T *grad = static_cast<const T *>(t.grad) + at;
        float *avg = static_cast<float *>(t.avg) + at, *sq = static_cast<float *>(t.sq) + at;
        f32x4 g, w, m, v;
        auto load = [&](auto vec) {
            constexpr bool V = vec();
            g = load4<V>(grad, nv);
            w = load4<V>(param, nv);
            if (t.master) w = latest<T>(load4<V>(t.master + at, nv), w);
            m = load4<V>(avg, nv);
            v = load4<V>(sq, nv);
        };
        auto store = [&](auto vec) {
            constexpr bool V = vec();
            store4<V>(param, nv, w);
            if (t.master) store4<V>(t.master + at, nv, w);
            store4<V>(avg, nv, m);
            store4<V>(sq, nv, v);
        };
        whole ? load(std::true_type{}) : load(std::false_type{});
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float me = m[e], ve = v[e];
            w[e] = update(f, a.grad_scale != nullptr, scale, w[e], g[e], me, ve);
            m[e] = me;
            v[e] = ve;
        }
        whole ? store(std::true_type{}) : store(std::false_type{});
    }
}

// A lane holds 8 values side by side, 16 lanes a block.
template <class T, bool VEC>
__device__ static inline void step8(const AdamwArgs &a, const AdamwTensor &t, const AdamwFactors &f, float scale, int64_t base,
                                    uint32_t block, uint32_t key) {
#pragma unroll
    for (int i = 0; i < kAdamwChunk / 2048; ++i) {
        const int64_t at = base + 2048 * i + 8 * (int)threadIdx.x;
        const int64_t b = at >> 7;
        if (b << 7 >= t.n) continue;
        T *param = static_cast<T *>(t.param) + at;
        const T *grad = static_cast<const T *>(t.grad) + at;
        uint8_t *avg = static_cast<uint8_t *>(t.avg) + at, *sq = static_cast<uint8_t *>(t.sq) + at;
        const u32x2 mc = *reinterpret_cast<const u32x2 *>(avg), rc = *reinterpret_cast<const u32x2 *>(sq);
        const float ms = t.avg_scale[b], rs = t.sq_scale[b];
        float w[8], m[8], r[8];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int64_t p = at + 4 * q;
            const int nv = (int)min(t.n - p, (int64_t)4);
            const bool whole = VEC && nv == 4;
            const f32x4 ge = whole ? load4<true>(grad + 4 * q, 4) : load4<false>(grad + 4 * q, nv);
            f32x4 we = whole ? load4<true>(param + 4 * q, 4) : load4<false>(param + 4 * q, nv);
            if (t.master) we = latest<T>(whole ? load4<true>(t.master + p, 4) : load4<false>(t.master + p, nv), we);
            const f32x2 m01 = __builtin_amdgcn_cvt_pk_f32_fp8(mc[q], false), m23 = __builtin_amdgcn_cvt_pk_f32_fp8(mc[q], true);
            const f32x2 r01 = __builtin_amdgcn_cvt_pk_f32_fp8(rc[q], false), r23 = __builtin_amdgcn_cvt_pk_f32_fp8(rc[q], true);
            const float mv[4] = {m01[0], m01[1], m23[0], m23[1]}, rv[4] = {r01[0], r01[1], r23[0], r23[1]};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool there = e < nv;
                float me = mv[e] * ms, ve = rv[e] * rs;
                ve = ve * ve;
                w[4 * q + e] = update(f, a.grad_scale != nullptr, scale, we[e], ge[e], me, ve);
                m[4 * q + e] = there ? me : 0.0f;
                r[4 * q + e] = there ? sqrtf(ve) : 0.0f;
            }
            const f32x4 out = {w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]};
            if (whole) {
                store4<true>(param + 4 * q, 4, out);
                if (t.master) store4<true>(t.master + p, 4, out);
            } else {
                store4<false>(param + 4 * q, nv, out);
                if (t.master) store4<false>(t.master + p, nv, out);
            }
        }
        float mm = 0.0f, rm = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            mm = fmaxf(mm, finite_size(m[e]));
            rm = fmaxf(rm, finite_size(r[e]));
        }
        const float mscale = block_scale(max16(mm)), rscale = block_scale(max16(rm));
        const float minv = inverse_scale(mscale), rinv = inverse_scale(rscale);
        const uint32_t bk = mix(key + block + (uint32_t)b);
        const uint32_t place = 8 * (threadIdx.x & 15);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t h = mix(bk + place + e);
            const float my = scaled(m[e], minv), ry = scaled(r[e], rinv);
            const float up = round_up_sometimes(ry, h >> 16);
            // (the one NaN that `scaled` gives survives the rounding)
            m[e] = round_up_sometimes(my, h & 0xffffu);
            r[e] = ry > 0.0f ? fmaxf(up, 0.001953125f) : up;
        }
        *reinterpret_cast<u32x2 *>(avg) = u32x2{encode4(m[0], m[1], m[2], m[3]), encode4(m[4], m[5], m[6], m[7])};
        *reinterpret_cast<u32x2 *>(sq) = u32x2{encode4(r[0], r[1], r[2], r[3]), encode4(r[4], r[5], r[6], r[7])};
        if (place == 0) {
            t.avg_scale[b] = mscale;
            t.sq_scale[b] = rscale;
        }
    }
}

template <int BITS> __global__ __launch_bounds__(256) void grkan_adamw_kernel(AdamwArgs a) {
    // the last tensor whose first workgroup is not past this one
    const int lane = (int)threadIdx.x & 63;
    const bool before = lane < a.count && a.first[lane < a.count ? lane : 0] <= blockIdx.x;
    const int i = __popcll(__ballot(before)) - 1;
    const int it = __builtin_amdgcn_readfirstlane(i);
    const AdamwTensor t = a.t[it];
    const int64_t base = (int64_t)(blockIdx.x - a.first[it]) * kAdamwChunk;
    const int64_t step = a.step_ptr ? *a.step_ptr : a.step;
    AdamwFactors f = a.f;
    if (a.lr_ptr || a.step_ptr) f = factors(a.lr_ptr ? (double)*a.lr_ptr : a.lr, a.beta1, a.beta2, a.decay, a.eps, step);
    const float scale = a.grad_scale ? *a.grad_scale : 1.0f;
    const uint8_t flags = a.flags[it];
    auto go = [&](auto type, auto vec) {
        using T = decltype(type);
        if constexpr (BITS == 32)
            step32<T, vec()>(a, t, f, scale, base);
        else
            step8<T, vec()>(a, t, f, scale, base, a.block[it], mix(mix(a.seed) + (uint32_t)step));
    };
    if (flags & kAdamwBf16) {
        if (flags & kAdamwVec)
            go(uint16_t{}, std::true_type{});
        else
            go(uint16_t{}, std::false_type{});
    } else {
        if (flags & kAdamwVec)
            go(float{}, std::true_type{});
        else
            go(float{}, std::false_type{});
    }
}

}  // namespace

void prepare_adamw(AdamwArgs &a) { a.f = factors(a.lr, a.beta1, a.beta2, a.decay, a.eps, a.step); }

hipError_t launch_adamw(const AdamwArgs &a, int bits, hipStream_t s) {
    const unsigned grid = a.first[a.count];
    if (grid == 0) return hipSuccess;
    if (bits == 32)
        hipLaunchKernelGGL((grkan_adamw_kernel<32>), dim3(grid), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((grkan_adamw_kernel<8>), dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace grkan
