// grkan_quantize.hip -- e4m3 codes and power-of-two scales for blocks of 128
// (gfx950).
//
// Bound: memory, one read of x and one byte an element for each layout.
#include "grkan_fp8.h"
#include "grkan_e4m3.h"
#include "grkan_lanes.h"

namespace grkan {
namespace {

// A workgroup takes 128 rows x 128 columns, 8 x 8 values a thread in registers.
// The maxima of rows meet over 16 lanes, those of columns through LDS; the
// transposed codes pass through LDS, so that both layouts leave as whole rows.
template <class T>
__global__ __launch_bounds__(256) void grkan_quantize_tile_kernel(QuantizeArgs a) {
    __shared__ float colmax[16][kBlock8 + 1];
    __shared__ float rowmax[kBlock8];
    __shared__ uint8_t codes[kBlock8][kBlock8 + 8];
    const int t = (int)threadIdx.x, cl = t & 15, rg = t >> 4;
    const int cb = (a.cols + kBlock8 - 1) / kBlock8;
    const int bc = (int)blockIdx.x % cb, br = (int)blockIdx.x / cb;
    const int c0 = bc * kBlock8 + cl * 8, r0 = br * kBlock8 + rg * 8;
    const T *x = static_cast<const T *>(a.x);
    float v[8][8];
    Coefs<5, 4> coef;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[i][e] = r0 + i < a.rows && c0 + e < a.cols ? load1(x + (int64_t)(r0 + i) * a.ldx + c0 + e) : 0.0f;
    if (a.A) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (c0 + e >= a.cols) continue;
            coef = load_coefs<5, 4>(a.A, a.B, (c0 + e) / a.dga);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r0 + i < a.rows) v[i][e] = rational<5, 4>(v[i][e], coef);
        }
    }
    float rm[8], cm[8] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        rm[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float m = finite_size(v[i][e]);
            rm[i] = fmaxf(rm[i], m);
            cm[e] = fmaxf(cm[e], m);
        }
        rm[i] = max16(rm[i]);
        if (cl == 0) rowmax[rg * 8 + i] = rm[i];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) colmax[rg][cl * 8 + e] = cm[e];
    __syncthreads();
    float all = 0.0f;
    if (a.tile) {
        for (int i = 0; i < kBlock8; ++i) all = fmaxf(all, rowmax[i]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cm[e] = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) cm[e] = fmaxf(cm[e], colmax[i][cl * 8 + e]);
        }
    }
    if (a.q) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float s = block_scale(a.tile ? all : rm[i]), inv = inverse_scale(s);
            const int r = r0 + i;
            if (r >= a.rows) continue;
            const u32x2 w = encode8(v[i], inv);
            uint8_t *to = a.q + (int64_t)r * a.ldq + c0;
            if (c0 < (a.cols + 15) / 16 * 16) *reinterpret_cast<u32x2 *>(to) = w;
            if (cl == 0 && !a.tile) a.scale[(int64_t)bc * a.lds + r] = s;
        }
        if (a.tile && t == 0) a.scale[(int64_t)bc * a.lds + br] = block_scale(all);
    }
    if (a.qt) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float s = block_scale(a.tile ? all : cm[e]), inv = inverse_scale(s);
            float u[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = v[i][e];
            *reinterpret_cast<u32x2 *>(&codes[cl * 8 + e][rg * 8]) = encode8(u, inv);
            if (rg == 0 && !a.tile && c0 + e < a.cols) a.scale_t[(int64_t)br * a.ldst + c0 + e] = s;
        }
        if (a.tile && t == 0) a.scale_t[(int64_t)br * a.ldst + bc] = block_scale(all);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = bc * kBlock8 + rg * 8 + i, r = br * kBlock8 + cl * 8;
            if (c < a.cols && r < (a.rows + 15) / 16 * 16)
                *reinterpret_cast<u32x2 *>(a.qt + (int64_t)c * a.ldqt + r) =
                    *reinterpret_cast<const u32x2 *>(&codes[rg * 8 + i][cl * 8]);
        }
    }
}

}  // namespace

hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t s) {
    const unsigned cb = (unsigned)((a.cols + kBlock8 - 1) / kBlock8);
    const unsigned rb = (unsigned)(((int64_t)a.rows + kBlock8 - 1) / kBlock8);
    if (a.bf16)
        hipLaunchKernelGGL((grkan_quantize_tile_kernel<uint16_t>), dim3(cb * rb), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((grkan_quantize_tile_kernel<float>), dim3(cb * rb), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace grkan
