// grkan_quantize.hip -- e4m3 codes and power-of-two scales for blocks of 128
// (gfx950).
//
// Bound: memory, one read of x and one byte an element for each layout: 25,216 x 3,072
// bf16 in both layouts 61 us (5.2 TB/s); 25,216 x 768 by rows through the rational 17.8 us
// (3.3 TB/s, half of it the launch and the loads' latency: 50,432 rows take 29).
#include "grkan_fp8.h"
#include "grkan_e4m3.h"
#include "grkan_lanes.h"

#include <type_traits>

namespace grkan {
namespace {

// A lane's 8 columns: their values in a row, F applied.  RAT: 0 no activation, 1 the
// rational with 8 columns in one activation group, 2 with any groups.
template <class T, bool VEC, int RAT> struct Columns8 {
    int c0, nv;   // first column, how many exist (at most 8; 0 or less: none)
    Coefs<5, 4> coef;
    __device__ inline Columns8(const QuantizeArgs &a, int c) : c0(c), nv(a.cols - c) {
        if constexpr (RAT == 1) coef = load_coefs<5, 4>(a.A, a.B, nv > 0 ? c / a.dga : 0);
    }
    // As they lie in memory.
    struct Raw {
        u32x4 w[sizeof(T) / 2];
    };
    __device__ inline Raw fetch(const QuantizeArgs &a, int64_t row) const {
        Raw r = {};
        const T *x = static_cast<const T *>(a.x) + row * a.ldx + c0;
        if (row >= a.rows || nv <= 0) return r;
        if (VEC && nv >= 8) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(x) + i);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e >= nv) continue;
                if constexpr (sizeof(T) == 2)
                    r.w[0][e / 2] |= (uint32_t)x[e] << (16 * (e & 1));
                else
                    r.w[e / 4][e % 4] = __float_as_uint(x[e]);
            }
        }
        return r;
    }
    __device__ inline void values(const QuantizeArgs &a, const Raw &r, bool there, float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (sizeof(T) == 2)
                v[e] = __uint_as_float((e & 1) ? (r.w[0][e / 2] & 0xffff0000u) : (r.w[0][e / 2] << 16));
            else
                v[e] = __uint_as_float(r.w[e / 4][e % 4]);
            // (F(0) need not be 0: what does not exist stays 0)
            if constexpr (RAT == 1) v[e] = there && e < nv ? rational<5, 4>(v[e], coef) : 0.0f;
            if constexpr (RAT == 2)
                v[e] = there && e < nv ? rational<5, 4>(v[e], load_coefs<5, 4>(a.A, a.B, (c0 + e) / a.dga)) : 0.0f;
        }
    }
};

__device__ static inline float finite_max8(const float (&v)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, finite_size(v[e]));
    return m;
}

// Rows alone: 16 lanes a block; a workgroup takes a column block of kQuantizeRows rows,
// so that a lane keeps its columns (and the rational's coefficients), all its loads
// on their way at once.
constexpr int kPasses = kQuantizeRows / 16;

template <class T, bool VEC, int RAT> __global__ __launch_bounds__(256) void grkan_quantize_rows_kernel(QuantizeArgs a) {
    const int t = (int)threadIdx.x, cl = t & 15, rg = t >> 4;
    const int cb = (a.cols + kBlock8 - 1) / kBlock8;
    const int bc = (int)blockIdx.x % cb, br = (int)blockIdx.x / cb;
    const Columns8<T, VEC, RAT> c(a, bc * kBlock8 + cl * 8);
    const int64_t r0 = (int64_t)br * kQuantizeRows + rg;
    typename Columns8<T, VEC, RAT>::Raw raw[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) raw[i] = c.fetch(a, r0 + 16 * i);
    const bool writes = c.c0 < (a.cols + 15) / 16 * 16;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int64_t r = r0 + 16 * i;
        float v[8];
        c.values(a, raw[i], r < a.rows, v);
        const float s = block_scale(max16(finite_max8(v)));
        if (r >= a.rows) continue;
        if (writes) *reinterpret_cast<u32x2 *>(a.q + r * a.ldq + c.c0) = encode8(v, inverse_scale(s));
        if (cl == 0) a.scale[(int64_t)bc * a.lds + r] = s;
    }
}

// The larger of v in each lane and in the lanes 16, 32 and 48 away.
__device__ static inline float max_of_rows(float v) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// Columns, both, or a scale for 128 x 128: a workgroup takes that many, 8 x 8 values
// a thread in registers, so x is read once.  The maxima of rows meet over 16 lanes,
// those of columns over the wave's four groups of rows and then through LDS; the
// transposed codes pass through LDS, so that both layouts leave as whole rows.
template <class T, bool VEC, int RAT, bool TILE>
__global__ __launch_bounds__(256) void grkan_quantize_tile_kernel(QuantizeArgs a) {
    __shared__ __attribute__((aligned(16))) float colmax[4][kBlock8];
    __shared__ __attribute__((aligned(16))) uint8_t codes[kBlock8][kBlock8 + 8];
    const int t = (int)threadIdx.x, cl = t & 15, rg = t >> 4, wave = t >> 6;
    const int cb = (a.cols + kBlock8 - 1) / kBlock8;
    const int bc = (int)blockIdx.x % cb, br = (int)blockIdx.x / cb;
    const Columns8<T, VEC, RAT> c(a, bc * kBlock8 + cl * 8);
    const int64_t r0 = (int64_t)br * kBlock8 + rg * 8;
    typename Columns8<T, VEC, RAT>::Raw raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = c.fetch(a, r0 + i);
    float v[8][8], rm[8], cm[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c.values(a, raw[i], r0 + i < a.rows, v[i]);
        rm[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float m = finite_size(v[i][e]);
            rm[i] = fmaxf(rm[i], m);
            cm[e] = fmaxf(cm[e], m);
        }
    }
    if constexpr (TILE) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, rm[i]);
        m = max_of_rows(max16(m));
        if ((t & 63) == 0) colmax[wave][0] = m;
        __syncthreads();
        m = fmaxf(fmaxf(colmax[0][0], colmax[1][0]), fmaxf(colmax[2][0], colmax[3][0]));
#pragma unroll
        for (int i = 0; i < 8; ++i) rm[i] = cm[i] = m;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) rm[i] = max16(rm[i]);
        if (a.qt) {
#pragma unroll
            for (int e = 0; e < 8; ++e) cm[e] = max_of_rows(cm[e]);
            if ((t & 63) < 16) {
                *reinterpret_cast<f32x4 *>(&colmax[wave][cl * 8]) = f32x4{cm[0], cm[1], cm[2], cm[3]};
                *reinterpret_cast<f32x4 *>(&colmax[wave][cl * 8 + 4]) = f32x4{cm[4], cm[5], cm[6], cm[7]};
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e)
                cm[e] = fmaxf(fmaxf(colmax[0][cl * 8 + e], colmax[1][cl * 8 + e]), fmaxf(colmax[2][cl * 8 + e], colmax[3][cl * 8 + e]));
        }
    }
    if (a.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t r = r0 + i;
            const float s = block_scale(rm[i]);
            if (r >= a.rows) continue;
            if (c.c0 < (a.cols + 15) / 16 * 16) *reinterpret_cast<u32x2 *>(a.q + r * a.ldq + c.c0) = encode8(v[i], inverse_scale(s));
            if (cl == 0 && !TILE) a.scale[(int64_t)bc * a.lds + r] = s;
        }
        if (TILE && t == 0) a.scale[(int64_t)bc * a.lds + br] = block_scale(rm[0]);
    }
    if (a.qt) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float s = block_scale(cm[e]);
            float u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = v[i][e];
            *reinterpret_cast<u32x2 *>(&codes[cl * 8 + e][rg * 8]) = encode8(u, inverse_scale(s));
            if (rg == 0 && !TILE && e < c.nv) a.scale_t[(int64_t)br * a.ldst + c.c0 + e] = s;
        }
        if (TILE && t == 0) a.scale_t[(int64_t)br * a.ldst + bc] = block_scale(rm[0]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // 16 columns a pass, 16 lanes to the 128 rows of one
            const int col = 16 * i + rg, cc = bc * kBlock8 + col;
            const int64_t r = (int64_t)br * kBlock8 + cl * 8;
            if (cc < a.cols && r < ((int64_t)a.rows + 15) / 16 * 16)
                *reinterpret_cast<u32x2 *>(a.qt + (int64_t)cc * a.ldqt + r) = *reinterpret_cast<const u32x2 *>(&codes[col][cl * 8]);
        }
    }
}

template <class T, bool VEC, int RAT> hipError_t launch_kind(const QuantizeArgs &a, hipStream_t s) {
    const int64_t cb = (a.cols + kBlock8 - 1) / kBlock8;
    if (!a.qt && !a.tile) {
        const int64_t rb = ((int64_t)a.rows + kQuantizeRows - 1) / kQuantizeRows;
        hipLaunchKernelGGL((grkan_quantize_rows_kernel<T, VEC, RAT>), dim3((unsigned)(cb * rb)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)(cb * (((int64_t)a.rows + kBlock8 - 1) / kBlock8)));
    if (a.tile)
        hipLaunchKernelGGL((grkan_quantize_tile_kernel<T, VEC, RAT, true>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((grkan_quantize_tile_kernel<T, VEC, RAT, false>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

template <class T> hipError_t launch_type(const QuantizeArgs &a, hipStream_t s) {
    const bool vec = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.ldx * (int64_t)sizeof(T) % 16 == 0;
    if (!a.A) return vec ? launch_kind<T, true, 0>(a, s) : launch_kind<T, false, 0>(a, s);
    if (a.dga % 8 == 0) return vec ? launch_kind<T, true, 1>(a, s) : launch_kind<T, false, 1>(a, s);
    return launch_kind<T, false, 2>(a, s);
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t s) {
    return a.bf16 ? launch_type<uint16_t>(a, s) : launch_type<float>(a, s);
}

}  // namespace grkan
