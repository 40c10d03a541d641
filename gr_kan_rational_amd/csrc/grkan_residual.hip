// grkan_residual.hip -- h = x + scale gate post(f), z = norm(h), and the
// backward (gfx950).
//
// Compiled per I/O type (GRKAN_RESIDUAL_BF16) and direction
// (GRKAN_RESIDUAL_BACKWARD).
//
// Bound: memory.  A row is held in registers by one wave (up to 1,024
// channels) or by 2 to 16, so each tensor is read or written once; the sums of
// a row stay inside the wave or meet in LDS.  50,432 x 768 bf16: forward with a gate for
// each sample 53 us (5.9 TB/s); backward 88 us (5.3 TB/s), with norms on both sides and a
// gate for each image and channel 99 and 8.6 for the sums' last step.
#include "grkan_residual.h"

#include "grkan_lanes.h"

#ifndef GRKAN_RESIDUAL_BF16
#error "GRKAN_RESIDUAL_BF16"
#endif

namespace grkan {
namespace {

#if GRKAN_RESIDUAL_BF16
typedef uint16_t io_t;
#else
typedef float io_t;
#endif

// The columns of a lane: 4 from 4 (lane + 64 W k), k < K, over the W waves of a row.
// K is the least that covers them, so only the last k can lie past the end.
template <int W, int K> struct Columns {
    int first, C;
    __device__ inline Columns(int lane_of_row, int C_) : first(4 * lane_of_row), C(C_) {}
    __device__ inline int at(int k) const { return first + 256 * W * k; }
    __device__ inline int nv(int k) const { return k < K - 1 ? 4 : min(C - at(k), 4); }  // at most 0: none
};

// Four values as they lie in memory, so that a row on its way takes few registers.
#if GRKAN_RESIDUAL_BF16
typedef u32x2 raw4;
__device__ static inline f32x4 widen(raw4 w) {
    return f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                 __uint_as_float(w[1] & 0xffff0000u)};
}
#else
typedef f32x4 raw4;
__device__ static inline f32x4 widen(raw4 w) { return w; }
#endif
template <bool VEC> __device__ static inline raw4 load_raw(const io_t *p, int nv) {
    raw4 w = {};
    if constexpr (VEC) {
        if (nv > 0) w = __builtin_nontemporal_load(reinterpret_cast<const raw4 *>(p));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < nv) reinterpret_cast<io_t *>(&w)[e] = p[e];
    }
    return w;
}

// Sums of N values over the W waves of a row, the same bits in every lane.
template <int W, int N> __device__ static inline void row_sum(float (&v)[N], float (*red)[8], int wave) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = sum64(v[i]);
    if constexpr (W > 1) {
        __syncthreads();  // the sums before these have been read
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) red[wave][i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) v[i] += red[w][i];
        }
    }
}

// A vector of one value per channel, or `none` for each; zeros past the end.  With
// the scale zero there (and x, f, dh and dz read as zeros) what a lane forms past the
// end adds nothing to a row's sums.
template <bool VEC> __device__ static inline f32x4 vector4(const float *p, int at, int nv, float none) {
    if (p) return load4<VEC>(p + at, nv);
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = e < nv ? none : 0.0f;
    return v;
}

// How a kernel takes its gate: known when it is compiled, since a branch inside the
// rows' loop keeps their loads from overlapping (2,048 channels, one gate a sample:
// 70 us forward with branches, 50 without).  kAny serves what is rare: rows that are
// not whole accesses, and fp32 gates of bf16 rows.
enum GateMode : int { kAny = -1, kNoGate = 0, kNarrow = 1, kShared = 2, kElement = 3 };

// The gate's row of a row (rows fit 31 bits).
__device__ static inline int64_t gate_row(const ResidualArgs &a, int64_t row) {
    return a.gate_rows == 1 ? row : (int64_t)fastdiv((uint32_t)row, a.gate_div);
}

// The gate of a lane's columns: per row (narrow, or one for each element) as it lies in
// memory, fetched with its row; shared by rows that follow each other, loaded
// where that changes.
template <int W, int K, bool VEC, int GM> struct Gate {
    uint32_t narrow;
    raw4 element[GM == kElement ? K : 1];
    f32x4 held[GM == kShared || GM == kAny ? K : 1];

    // With row `row`, before its data.
    __device__ inline void fetch(const ResidualArgs &a, int64_t row, const Columns<W, K> &c) {
        if constexpr (GM == kNarrow) {
            const int64_t g = gate_row(a, row);
            narrow = a.gate_bf16 ? static_cast<const uint16_t *>(a.gate)[g] : static_cast<const uint32_t *>(a.gate)[g];
        } else if constexpr (GM == kElement) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                element[k] = load_raw<VEC>(static_cast<const io_t *>(a.gate) + row * a.C + c.at(k), c.nv(k));
        }
    }
    // At a row from which it differs.
    __device__ inline void load(const ResidualArgs &a, int64_t row, const Columns<W, K> &c) {
        if constexpr (GM == kShared || GM == kAny) {
            if (GM == kAny && !a.gate) return;
            const int64_t g = gate_row(a, row);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int at = c.at(k), nv = c.nv(k);
                if (GM == kShared) {
                    held[k] = load4<VEC>(static_cast<const io_t *>(a.gate) + g * a.C + at, nv);
                } else if (!a.gate_wide) {
                    const float v = a.gate_bf16 ? load1(static_cast<const uint16_t *>(a.gate) + g) : static_cast<const float *>(a.gate)[g];
                    held[k] = f32x4{v, v, v, v};
                } else if (a.gate_bf16) {
                    held[k] = load4<VEC>(static_cast<const uint16_t *>(a.gate) + g * a.C + at, nv);
                } else {
                    held[k] = load4<VEC>(static_cast<const float *>(a.gate) + g * a.C + at, nv);
                }
            }
        }
    }
    // v gate
    __device__ inline f32x4 times(const ResidualArgs &a, f32x4 v, int k) const {
        if constexpr (GM == kNarrow) return v * __uint_as_float(a.gate_bf16 ? narrow << 16 : narrow);
        if constexpr (GM == kElement) return v * widen(element[k]);
        if constexpr (GM == kShared) return v * held[k];
        if constexpr (GM == kAny) return a.gate ? v * held[k] : v;
        return v;
    }
};

// mean and 1 / sqrt(var + eps) of a row held as v (zeros past its columns).
template <int W, int K>
__device__ static inline void moments(const f32x4 (&v)[K], const Columns<W, K> &c, int kind, float eps, float (*red)[8],
                                      int wave, float &mean, float &rstd) {
    const float inv = 1.0f / (float)c.C;
    float s[1] = {0.0f};
    mean = 0.0f;
    if (kind == GRKAN_NORM_LAYER) {
#pragma unroll
        for (int k = 0; k < K; ++k) s[0] += (v[k][0] + v[k][1]) + (v[k][2] + v[k][3]);
        row_sum<W>(s, red, wave);
        mean = s[0] * inv;
    }
    s[0] = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float d = k < K - 1 || e < c.nv(k) ? v[k][e] - mean : 0.0f;
            s[0] = fmaf(d, d, s[0]);
        }
    row_sum<W>(s, red, wave);
    rstd = 1.0f / sqrtf(fmaf(s[0], inv, eps));
}

#if !GRKAN_RESIDUAL_BACKWARD

// A walker's rows one after another, the vectors of a lane's columns in registers, the
// next row on its way while one is worked on.
template <int W, int K, bool VEC, bool POST, int GM>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void grkan_residual_forward_kernel(ResidualArgs a) {
    __shared__ float red[W][8];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const Columns<W, K> c(W == 1 ? (int)threadIdx.x & 63 : (int)threadIdx.x, a.C);
    const int64_t walker = W == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
    const int64_t r0 = walker * a.p.walk, r1 = min(r0 + a.p.walk, a.rows);
    if (r0 >= r1) return;
    f32x4 weight[K], bias[K], scale[K], pw[POST ? K : 1], pb[POST ? K : 1];
    raw4 nx[K], nf[K];
    Gate<W, K, VEC, GM> ng;
    auto fetch = [&](int64_t row) {
        ng.fetch(a, row, c);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            nx[k] = load_raw<VEC>(static_cast<const io_t *>(a.x) + row * a.ldx + c.at(k), c.nv(k));
            nf[k] = load_raw<VEC>(static_cast<const io_t *>(a.f) + row * a.ldf + c.at(k), c.nv(k));
        }
    };
    fetch(r0);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        weight[k] = vector4<VEC>(a.weight, c.at(k), c.nv(k), 1.0f);
        bias[k] = vector4<VEC>(a.bias, c.at(k), c.nv(k), 0.0f);
        scale[k] = vector4<VEC>(a.scale, c.at(k), c.nv(k), 1.0f);
        if constexpr (POST) {
            pw[k] = vector4<VEC>(a.post_weight, c.at(k), c.nv(k), 1.0f);
            pb[k] = vector4<VEC>(a.post_bias, c.at(k), c.nv(k), 0.0f);
        }
    }
    int64_t changes = r0;  // the next row whose shared gate is another
    for (int64_t r = r0; r < r1; ++r) {
        f32x4 h[K], u[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            h[k] = widen(nx[k]);
            u[k] = widen(nf[k]);
        }
        if ((GM == kShared || GM == kAny) && r == changes) {
            ng.load(a, r, c);
            changes = (gate_row(a, r) + 1) * a.gate_rows;
        }
        const Gate<W, K, VEC, GM> gate = ng;
        if (r + 1 < r1) fetch(r + 1);
        float mean, rstd;
        if constexpr (POST) {
            moments<W, K>(u, c, a.post, a.eps, red, wave, mean, rstd);
#pragma unroll
            for (int k = 0; k < K; ++k) u[k] = (u[k] - mean) * rstd * pw[k] + pb[k];
            if (c.first == 0) {
                a.stats[2 * a.rows + r] = mean;
                a.stats[3 * a.rows + r] = rstd;
            }
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            h[k] += gate.times(a, scale[k], k) * u[k];
            store4<VEC>(static_cast<io_t *>(a.h) + r * a.C + c.at(k), c.nv(k), h[k]);
        }
        moments<W, K>(h, c, a.norm, a.eps, red, wave, mean, rstd);
#pragma unroll
        for (int k = 0; k < K; ++k)
            store4<VEC>(static_cast<io_t *>(a.z) + r * a.C + c.at(k), c.nv(k), (h[k] - mean) * rstd * weight[k] + bias[k]);
        if (c.first == 0) {
            a.stats[r] = mean;
            a.stats[a.rows + r] = rstd;
        }
    }
}
#define GRKAN_RESIDUAL_KERNEL grkan_residual_forward_kernel

#else

// Rows one after another; their column sums stay in registers, meet in LDS where a
// workgroup's waves hold different rows, and leave as one row of partials per
// workgroup: dz xh, dz, and g gate f (dscale) or, with a post norm, P = g gate fh and
// Q = g gate, of which, a column's factors being the same in every row,
// dpost_weight = scale P, dpost_bias = scale Q, dscale = post_weight P + post_bias Q.
template <int W, int K, bool VEC, bool POST, int GM>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W, W <= 8 ? 2 : 1) void grkan_residual_backward_kernel(ResidualArgs a) {
    constexpr int S = POST ? 4 : 3, V = POST ? 3 : 2;
    __shared__ float red[W][8];
    __shared__ f32x4 meet[W == 1 ? 4 : 1][W == 1 ? 64 : 1];
    __shared__ f32x4 vectors[W == 1 ? V * K : 1][W == 1 ? 64 : 1];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = (int)threadIdx.x & 63;
    const Columns<W, K> c(W == 1 ? lane : (int)threadIdx.x, a.C);
    const float inv = 1.0f / (float)a.C;
    const int per = W == 1 ? 4 : 1;
    const bool layer = a.norm == GRKAN_NORM_LAYER, post_layer = a.post == GRKAN_NORM_LAYER;
    const bool narrow = GM == kAny ? a.gate && !a.gate_wide : GM == kNarrow;
    const bool shared = GM == kAny ? a.gate && a.gate_wide && a.gate_rows > 1 : GM == kShared;
    const bool element = GM == kAny ? a.gate && a.gate_wide && a.gate_rows == 1 : GM == kElement;
    // weight, scale x post_weight and scale x post_bias of a lane's columns (with a post
    // norm; else weight and scale): from LDS where a wave holds a row, since every wave
    // needs all of them, else from memory
    auto make = [&](int v, int k) {
        const int at = c.at(k), nv = c.nv(k);
        if (v == 0) return vector4<VEC>(a.weight, at, nv, 1.0f);
        const f32x4 s = vector4<VEC>(a.scale, at, nv, 1.0f);
        if (!POST) return s;
        return s * (v == 1 ? vector4<VEC>(a.post_weight, at, nv, 1.0f) : vector4<VEC>(a.post_bias, at, nv, 0.0f));
    };
    if constexpr (W == 1) {
        for (int i = wave; i < V * K; i += 4) vectors[i][lane] = make(i / K, i % K);
        __syncthreads();
    }
    auto vector = [&](int v, int k) {
        if constexpr (W == 1) return vectors[v * K + k][lane];
        return make(v, k);
    };
    raw4 nh[K], nf[K], ndh[K], ndz[K];
    Gate<W, K, VEC, GM> ng;
    auto fetch = [&](int64_t r) {
        ng.fetch(a, r, c);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            nh[k] = load_raw<VEC>(static_cast<const io_t *>(a.h) + r * a.C + c.at(k), c.nv(k));
            nf[k] = load_raw<VEC>(static_cast<const io_t *>(a.f) + r * a.ldf + c.at(k), c.nv(k));
            ndh[k] = a.dh ? load_raw<VEC>(static_cast<const io_t *>(a.dh) + r * a.lddh + c.at(k), c.nv(k)) : raw4{};
            ndz[k] = a.dz ? load_raw<VEC>(static_cast<const io_t *>(a.dz) + r * a.lddz + c.at(k), c.nv(k)) : raw4{};
        }
    };
    f32x4 sum[S][K], gsum[K];
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k) sum[i][k] = f32x4{};
    // This walker's rows.  Those of a gate row that lie in one walker's leave its sum as
    // dgate; else each walker leaves what it has, in the first of its two places if the
    // gate row began before, else in the second.
    const int64_t walker = (int64_t)blockIdx.x * per + (W == 1 ? wave : 0);
    const int64_t r0 = walker * a.p.walk, r1 = min(r0 + a.p.walk, a.rows);
    int64_t gr = 0, gate_end = 0;
    auto leave = [&]() {
        if (!shared || !a.dgate) return;
        const bool before = gr * a.gate_rows < r0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int at = c.at(k), nv = c.nv(k);
            if (before || gate_end > r1)
                store4<VEC>(a.gate_sums + (2 * walker + !before) * a.C + at, nv, gsum[k]);
            else if (a.gate_bf16)
                store4<VEC>(static_cast<uint16_t *>(a.dgate) + gr * a.C + at, nv, gsum[k]);
            else
                store4<VEC>(static_cast<float *>(a.dgate) + gr * a.C + at, nv, gsum[k]);
            gsum[k] = f32x4{};
        }
    };
#pragma unroll
    for (int k = 0; k < K; ++k) gsum[k] = f32x4{};
    if (r0 < r1) {
        fetch(r0);
        for (int64_t r = r0; r < r1; ++r) {
            if ((GM == kShared || GM == kAny) && (r == gate_end || r == r0)) {
                if (r > r0) leave();
                ng.load(a, r, c);
                gr = gate_row(a, r);
                gate_end = (gr + 1) * a.gate_rows;
            }
            f32x4 g[K], u[K], t[K], xh[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                xh[k] = widen(nh[k]);
                u[k] = widen(nf[k]);
                g[k] = widen(ndh[k]);
                t[k] = widen(ndz[k]);
            }
            const Gate<W, K, VEC, GM> gate = ng;
            if (r + 1 < r1) fetch(r + 1);
            const float mean = a.stats[r], rstd = a.stats[a.rows + r];
            float m[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < K; ++k) {
                xh[k] = (xh[k] - mean) * rstd;
                sum[0][k] += t[k] * xh[k];
                sum[1][k] += t[k];
                t[k] *= vector(0, k);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    m[0] += t[k][e];
                    m[1] = fmaf(t[k][e], xh[k][e], m[1]);
                }
            }
            row_sum<W>(m, red, wave);
            const float m0 = layer ? m[0] * inv : 0.0f, m1 = m[1] * inv;
            float q[3] = {0.0f, 0.0f, 0.0f};
            float pmean = 0.0f, prstd = 0.0f;
            if constexpr (POST) {
                pmean = a.stats[2 * a.rows + r];
                prstd = a.stats[3 * a.rows + r];
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int at = c.at(k), nv = c.nv(k);
                g[k] += rstd * (t[k] - m0 - xh[k] * m1);
                if (a.dx) store4<VEC>(static_cast<io_t *>(a.dx) + r * a.C + at, nv, g[k]);
                f32x4 fh = u[k];
                if constexpr (POST) {
                    fh = (fh - pmean) * prstd;
                }
                const f32x4 s = vector(1, k), gg = gate.times(a, g[k], k);
                if (narrow || shared || element) {
                    const f32x4 gu = g[k] * (POST ? fh * s + vector(V - 1, k) : fh * s);
                    if (narrow)
                        q[2] += (gu[0] + gu[1]) + (gu[2] + gu[3]);
                    else if (shared)
                        gsum[k] += gu;
                    else if (a.dgate && a.gate_bf16)
                        store4<VEC>(static_cast<uint16_t *>(a.dgate) + r * a.C + at, nv, gu);
                    else if (a.dgate)
                        store4<VEC>(static_cast<float *>(a.dgate) + r * a.C + at, nv, gu);
                }
                sum[2][k] += gg * fh;
                if constexpr (POST) sum[3][k] += gg;
                const f32x4 d = gg * s;
                if constexpr (POST) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        q[0] += d[e];
                        q[1] = fmaf(d[e], fh[e], q[1]);
                    }
                    xh[k] = fh;
                    t[k] = d;
                } else if (a.df) {
                    store4<VEC>(static_cast<io_t *>(a.df) + r * a.C + at, nv, d);
                }
            }
            if (POST || narrow) row_sum<W>(q, red, wave);
            if (narrow && a.dgate && c.first == 0) {
                if (a.gate_rows > 1)
                    a.gate_sums[r] = q[2];
                else if (a.gate_bf16)
                    store1(static_cast<uint16_t *>(a.dgate) + r, q[2]);
                else
                    static_cast<float *>(a.dgate)[r] = q[2];
            }
            if constexpr (POST) {
                const float q0 = post_layer ? q[0] * inv : 0.0f, q1 = q[1] * inv;
                if (a.df) {
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        store4<VEC>(static_cast<io_t *>(a.df) + r * a.C + c.at(k), c.nv(k),
                                    prstd * (t[k] - q0 - xh[k] * q1));
                }
            }
        }
        leave();
    }
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float *to = a.sums + ((int64_t)blockIdx.x * S + i) * a.C + c.at(k);
            if constexpr (W == 1) {
                __syncthreads();
                meet[wave][lane] = sum[i][k];
                __syncthreads();
                if (wave == 0) {
                    f32x4 v = sum[i][k];
#pragma unroll
                    for (int w = 1; w < 4; ++w) v += meet[w][lane];
                    store4<VEC>(to, c.nv(k), v);
                }
            } else {
                store4<VEC>(to, c.nv(k), sum[i][k]);
            }
        }
}

// The second step, sums in fp64 and in order: the workgroups' partials of each
// column (32 columns x 32 lanes of workgroups); then, from workgroup `columns` on,
// dgate of each (gate, channel) from what the walkers left, or of each gate from its
// rows.  Bound: latency (505 workgroups' partials of 768 channels: 8.6 us).
__global__ __launch_bounds__(1024) void grkan_residual_sums_kernel(ResidualArgs a, int columns, int64_t gates) {
    __shared__ double red[2][1024];
    const int t = (int)threadIdx.x;
    if ((int)blockIdx.x >= columns) {
        for (int64_t i = (int64_t)((int)blockIdx.x - columns) * 1024 + t; i < gates; i += (int64_t)((int)gridDim.x - columns) * 1024) {
            double s = 0.0;
            if (a.gate_wide && a.gate_rows > 0) {
                const int64_t g = i / a.C, col = i - g * a.C, first = g * a.gate_rows / a.p.walk;
                const int64_t last = ((g + 1) * a.gate_rows - 1) / a.p.walk;
                if (first == last) continue;  // (written by its walker)
                const bool before = g * a.gate_rows < first * a.p.walk;
                s = (double)a.gate_sums[(2 * first + !before) * a.C + col];
#pragma unroll 8
                for (int64_t w = first + 1; w <= last; ++w) s += (double)a.gate_sums[2 * w * a.C + col];
            } else {
                const float *p = a.gate_sums + i * a.gate_rows;
#pragma unroll 8
                for (int64_t k = 0; k < a.gate_rows; ++k) s += (double)p[k];
            }
            if (a.gate_bf16)
                store1(static_cast<uint16_t *>(a.dgate) + i, (float)s);
            else
                static_cast<float *>(a.dgate)[i] = (float)s;
        }
        return;
    }
    const int cb = (a.C + 31) / 32, i = (int)blockIdx.x / cb, col = ((int)blockIdx.x - i * cb) * 32 + (t & 31);
    // (with a post norm the third and fourth columns' sums together: P and Q)
    const bool two = i == 2 && a.post != GRKAN_NORM_NONE;
    double v = 0.0, w = 0.0;
    if (col < a.C) {
        const float *p = a.sums + (int64_t)i * a.C + col;
        const int64_t step = (int64_t)a.p.sums * a.C;
        if (two) {
#pragma unroll 8
            for (int64_t b = t >> 5; b < a.p.blocks; b += 32) {
                v += (double)p[b * step];
                w += (double)p[b * step + a.C];
            }
        } else {
#pragma unroll 16
            for (int64_t b = t >> 5; b < a.p.blocks; b += 32) v += (double)p[b * step];
        }
    }
    red[0][t] = v;
    red[1][t] = w;
    __syncthreads();
    if (t >= 32 || col >= a.C) return;
#pragma unroll
    for (int q = 1; q < 32; ++q) {
        v += red[0][t + 32 * q];
        w += red[1][t + 32 * q];
    }
    if (i < 2) {
        float *out = i == 0 ? a.dweight : a.dbias;
        if (out) out[col] = (float)v;
        return;
    }
    if (!two) {
        if (a.dscale) a.dscale[col] = (float)v;
        return;
    }
    const double scale = a.scale ? a.scale[col] : 1.0f;
    if (a.dpost_weight) a.dpost_weight[col] = (float)(scale * v);
    if (a.dpost_bias) a.dpost_bias[col] = (float)(scale * w);
    if (a.dscale)
        a.dscale[col] = (float)((a.post_weight ? a.post_weight[col] : 1.0f) * v + (a.post_bias ? a.post_bias[col] : 0.0f) * w);
}

#define GRKAN_RESIDUAL_KERNEL grkan_residual_backward_kernel
#endif

template <int W, int K, bool VEC, bool POST> hipError_t launch_gate(const ResidualArgs &a, int mode, hipStream_t s) {
    const dim3 grid((unsigned)a.p.blocks), block(W == 1 ? 256 : 64 * W);
    if constexpr (VEC) {
        // (a wave alone takes no four accesses of these: see residual_plan)
        constexpr bool planned = !(GRKAN_RESIDUAL_BACKWARD && POST && W == 1 && K == 4);
        if constexpr (!planned) {
            if (mode == kShared || mode == kElement) return hipErrorInvalidValue;
        }
        switch (mode) {
            case kNoGate: hipLaunchKernelGGL((GRKAN_RESIDUAL_KERNEL<W, K, true, POST, kNoGate>), grid, block, 0, s, a); return hipGetLastError();
            case kNarrow: hipLaunchKernelGGL((GRKAN_RESIDUAL_KERNEL<W, K, true, POST, kNarrow>), grid, block, 0, s, a); return hipGetLastError();
            case kShared:
                if constexpr (planned) hipLaunchKernelGGL((GRKAN_RESIDUAL_KERNEL<W, K, true, POST, kShared>), grid, block, 0, s, a);
                return hipGetLastError();
            case kElement:
                if constexpr (planned) hipLaunchKernelGGL((GRKAN_RESIDUAL_KERNEL<W, K, true, POST, kElement>), grid, block, 0, s, a);
                return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((GRKAN_RESIDUAL_KERNEL<W, K, VEC, POST, kAny>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int W, int K> hipError_t launch_kernel(const ResidualArgs &a, hipStream_t s) {
    const bool same = a.gate_bf16 == (sizeof(io_t) == 2);
    int mode = kAny;
    if (!a.gate)
        mode = kNoGate;
    else if (!a.gate_wide)
        mode = kNarrow;
    else if (same)
        mode = a.gate_rows > 1 ? kShared : kElement;
    if (a.post != GRKAN_NORM_NONE)
        return a.vec ? launch_gate<W, K, true, true>(a, mode, s) : launch_gate<W, K, false, true>(a, mode, s);
    return a.vec ? launch_gate<W, K, true, false>(a, mode, s) : launch_gate<W, K, false, false>(a, mode, s);
}

// The pairs of (waves, K) that plans have.
hipError_t launch_rows(const ResidualArgs &a, hipStream_t s) {
    switch (a.p.waves * 8 + a.p.K) {
        case 8 + 1: return launch_kernel<1, 1>(a, s);
        case 8 + 2: return launch_kernel<1, 2>(a, s);
        case 8 + 3: return launch_kernel<1, 3>(a, s);
        case 8 + 4: return launch_kernel<1, 4>(a, s);
        case 16 + 2: return launch_kernel<2, 2>(a, s);
        case 16 + 3: return launch_kernel<2, 3>(a, s);
        case 32 + 2: return launch_kernel<4, 2>(a, s);
        case 32 + 3: return launch_kernel<4, 3>(a, s);
        case 64 + 2: return launch_kernel<8, 2>(a, s);
        case 64 + 3: return launch_kernel<8, 3>(a, s);
        case 64 + 4: return launch_kernel<8, 4>(a, s);
        case 128 + 3: return launch_kernel<16, 3>(a, s);
        case 128 + 4: return launch_kernel<16, 4>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

#if !GRKAN_RESIDUAL_BACKWARD
template <> hipError_t launch_residual_forward<io_t>(const ResidualArgs &a, hipStream_t s) { return launch_rows(a, s); }
#else
// (without rows the sums are all that is left, zeros)
template <> hipError_t launch_residual_backward<io_t>(const ResidualArgs &a, hipStream_t s) {
    hipError_t e = a.rows > 0 ? launch_rows(a, s) : hipSuccess;
    if (e != hipSuccess) return e;
    const bool sums = a.dweight || a.dbias || a.dscale || a.dpost_weight || a.dpost_bias;
    const int64_t gates = a.dgate && a.gate_rows != 1 ? a.gates * (a.gate_wide ? a.C : 1) : 0;
    const ResidualSums grid = residual_sums(a.C, sums, gates);
    if (grid.blocks > 0) {
        hipLaunchKernelGGL(grkan_residual_sums_kernel, dim3((unsigned)grid.blocks), dim3(1024), 0, s, a, grid.columns, gates);
        e = hipGetLastError();
    }
    return e;
}
#endif

}  // namespace grkan
