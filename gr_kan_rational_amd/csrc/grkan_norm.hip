// grkan_norm.hip -- group norm with an activation, channels last (gfx950).
// Compiled once per I/O type (GRKAN_NORM_BF16) and direction
// (GRKAN_NORM_BACKWARD).
//
// Forward, for sample n and group g over its positions x D values:
//   mean, rstd;  xh = (x - mean) rstd;  h = xh w + b;  y = act(h).
// Backward, with dh = dy act'(h), t = dh w, <.> the mean over the group:
//   dx = rstd (t - <t> - xh <t xh>);  dw = sum dh xh;  db = sum dh;  dA, dB.
//
// Bound: memory.  The forward cannot do without reading x and writing y, the
// backward without reading x and dy and writing dx; the three ways to cover a
// group (grkan_norm.h) differ in whether the values stay on chip between the
// sums and their use.
//
// Precision.  Sums are fp32 over at most a lane's and a workgroup's values;
// the variance is taken about the mean (two passes over registers), so a mean
// far from zero costs nothing; where the values do not stay on chip the sums
// of x and x^2 are fp64 instead, which leaves var good to 2^-53 (mean / std)^2.
// Column sums (dw, db, dA, dB) are fp32 within a lane's rows and added across
// lanes in fp32, across workgroups in fp64, in a fixed order.
#include "grkan_norm.h"

#include "grkan_act.h"

namespace grkan {

#if GRKAN_NORM_BF16
typedef bf16io NormIo;
#else
typedef float NormIo;
#endif

namespace {

typedef NormIo IO;
constexpr int ES = GRKAN_NORM_BF16 ? 2 : 4;
constexpr int kMaxV = 16 / ES;

// ------------------------------------------------------------ accesses

// V elements as one access of V * ES bytes.  The address is aligned to an
// element only (an odd number of channels, a sliced tensor): gfx950 takes
// global accesses of any alignment, and the compiler is told the alignment so
// that it assumes no more.
template <int V> struct Pack {
    static constexpr int kBytes = V * ES, kWords = kBytes >= 4 ? kBytes / 4 : 1;
    typedef uint32_t vec __attribute__((ext_vector_type(kWords)));
    typedef vec uvec __attribute__((aligned(ES)));
    vec r;

    __device__ static inline Pack load(const char *p) {
        Pack k;
        if constexpr (kBytes == 2)
            k.r[0] = *reinterpret_cast<const uint16_t *>(p);
        else
            k.r = *reinterpret_cast<const uvec *>(p);
        return k;
    }
    // the first nv elements; the rest are zeros
    __device__ static inline Pack load(const char *p, int nv) {
        if (nv == V) return load(p);
        Pack k;
#pragma unroll
        for (int i = 0; i < kWords; ++i) k.r[i] = 0u;
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < nv) {
                if constexpr (ES == 4)
                    k.r[e] = *reinterpret_cast<const uint32_t *>(p + 4 * e);
                else
                    k.r[e / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(p + 2 * e) << (16 * (e & 1));
            }
        return k;
    }
    __device__ inline float get(int e) const {
        if constexpr (ES == 4)
            return __uint_as_float(r[e]);
        else
            return __uint_as_float((e & 1) ? (r[e / 2] & 0xffff0000u) : (r[e / 2] << 16));
    }
    // rounds to nearest even for bf16
    __device__ static inline Pack from(const float (&f)[V]) {
        Pack k;
        if constexpr (ES == 4) {
#pragma unroll
            for (int e = 0; e < V; ++e) k.r[e] = __float_as_uint(f[e]);
        } else if constexpr (V == 1) {
            k.r[0] = __builtin_bit_cast(uint16_t, (__bf16)f[0]);
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                f32x2 q = {f[2 * i], f[2 * i + 1]};
                k.r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(q, bf16x2));
            }
        }
        return k;
    }
    __device__ inline void store(char *p, int nv) const {
        if (nv == V) {
            if constexpr (kBytes == 2)
                *reinterpret_cast<uint16_t *>(p) = (uint16_t)r[0];
            else
                *reinterpret_cast<uvec *>(p) = r;
            return;
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < nv) {
                if constexpr (ES == 4)
                    *reinterpret_cast<uint32_t *>(p + 4 * e) = r[e];
                else
                    *reinterpret_cast<uint16_t *>(p + 2 * e) = (uint16_t)(r[e / 2] >> (16 * (e & 1)));
            }
    }
};

// A lane's columns: weight, bias and (rational) the coefficients of their one
// activation group.  Absent columns get weight 0.
template <int V, bool RAT> struct Cols {
    int col, nv;
    float w[V], b[V];
    Coefs<5, 4> c;

    __device__ inline void init(const NormArgs &a, int col_, int nv_) {
        col = col_;
        nv = nv_;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const bool in = e < nv;
            w[e] = in ? (a.w ? a.w[col + e] : 1.0f) : 0.0f;
            b[e] = in && a.b ? a.b[col + e] : 0.0f;
        }
        if constexpr (RAT) c = load_coefs<5, 4>(a.A, a.B, nv > 0 ? col / a.dga : 0);
    }
};

// y of one access, the statistics folded into one multiplication and addition
// after the subtraction of the mean (which is exact enough only when done
// first).
template <int V, bool RAT>
__device__ static inline Pack<V> apply_forward(const Pack<V> &x, float mean, float rstd, const Cols<V, RAT> &k,
                                               int act) {
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = act_value<RAT>(fmaf((x.get(e) - mean) * rstd, k.w[e], k.b[e]), act, k.c);
    return Pack<V>::from(f);
}

// Sums of column values kept by a lane over its rows.
template <int V, bool RAT> struct ColSums {
    float dw[V], db[V], coef[RAT ? 10 : 1];
    __device__ inline void clear() {
#pragma unroll
        for (int e = 0; e < V; ++e) dw[e] = db[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < (RAT ? 10 : 1); ++i) coef[i] = 0.0f;
    }
    static constexpr int kValues = 2 * V + (RAT ? 10 : 0);
    __device__ inline float get(int i) const {
        return i < V ? dw[i] : (i < 2 * V ? db[i - V] : coef[i - 2 * V]);
    }
};

// dh and xh of element e.
template <int V, bool RAT>
__device__ static inline float slope(float x, float dy, float mean, float rstd, const Cols<V, RAT> &k, int e, int act,
                                     float *coef, float &xh) {
    xh = (x - mean) * rstd;
    const float h = fmaf(xh, k.w[e], k.b[e]);
    if constexpr (RAT) {
        return rational_slope(h, dy, k.c, *reinterpret_cast<float (*)[10]>(coef));
    } else {
        return dy * act_slope(h, act);
    }
}

// ------------------------------------------------------------ reductions

// Sum of v over the T lanes of a slot, in every one of them.  T <= 64: a
// butterfly within the wave.  Larger T is the whole workgroup: one value per
// wave through LDS (`lds` is 2 x 16 floats x NV used alternately, so that one
// barrier per call is enough).
template <int NV>
__device__ static inline void slot_sum(float (&v)[NV], int T, float *lds, int &phase) {
    const int top = T < 64 ? T : 64;
    for (int o = top >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] += __shfl_xor(v[i], o, 64);
    if (T > 64) {
        float *buf = lds + phase * 16 * NV;
        phase ^= 1;
        const int wv = (int)threadIdx.x >> 6, nw = T >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) buf[i * 16 + wv] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float s = 0.0f;
            for (int w = 0; w < nw; ++w) s += buf[i * 16 + w];
            v[i] = s;
        }
    }
}

// Sums of NV values over each group of a column block of TX x TY lanes, in
// every lane of the group.  `lds` holds NV * (threads + groups) values.
template <class R, int NV>
__device__ static inline void group_sum(R (&v)[NV], const NormPlan &p, int vpg, int ngroups, int jg, char *ldsb) {
    R *red = reinterpret_cast<R *>(ldsb);
    R *res = red + NV * p.block;
    const int t = (int)threadIdx.x, l = t & (p.L - 1);
#pragma unroll
    for (int i = 0; i < NV; ++i) red[i * p.block + t] = v[i];
    __syncthreads();
    const int count = vpg * p.TY;
    for (int j = t / p.L; j < ngroups; j += p.block / p.L) {
        R s[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = 0;
        for (int q = l; q < count; q += p.L) {
            const int row = q / vpg, at = row * p.TX + j * vpg + (q - row * vpg);
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] += red[i * p.block + at];
        }
        for (int o = p.L >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] += __shfl_xor(s[i], o, 64);
        if (l == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) res[i * p.gpb + j] = s[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = res[i * p.gpb + jg];
}

// A lane's place in a column block: columns, group within the block, row lane.
struct Place {
    int g0, ngroups, vpg;    // first group of the block, groups in it, accesses per group in it
    int jg, col, nv, ty;
    bool on;
    __device__ inline Place(const NormArgs &a, int cb) {
        const NormPlan &p = a.p;
        const int t = (int)threadIdx.x, tx = t % p.TX;
        ty = t / p.TX;
        int vi;
        if (p.bpg == 1) {
            g0 = cb * p.gpb;
            ngroups = min(p.gpb, a.G - g0);
            vpg = p.vpg;
            jg = tx / vpg;
            vi = tx - jg * vpg;
        } else {
            g0 = cb / p.bpg;
            ngroups = 1;
            vpg = p.TX;
            jg = 0;
            vi = (cb - g0 * p.bpg) * p.TX + tx;
        }
        on = ty < p.TY && jg < ngroups && vi < p.vpg;
        if (jg >= ngroups) jg = 0;
        col = (g0 + jg) * a.D + vi * p.vec;
        nv = on ? min(p.vec, a.D - vi * p.vec) : 0;
    }
    // index of the lane's access in a row of all groups
    __device__ inline int64_t access(const NormArgs &a) const {
        const int g = col / a.D;
        return (int64_t)g * a.p.vpg + (col - g * a.D) / a.p.vec;
    }
};

__device__ static inline const char *at(const void *base, int64_t e) {
    return static_cast<const char *>(base) + e * ES;
}
__device__ static inline char *at(void *base, int64_t e) { return static_cast<char *>(base) + e * ES; }

__device__ static inline float rstd_of(float var, float eps) { return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps); }

// Sample of a (workgroup, column block): with 8 samples or more the column
// blocks of a sample go to one XCD (workgroups are dealt to the 8 XCDs in
// turn), where the cache lines that two blocks share are fetched once.
__device__ static inline void sample_block(int64_t b, int ncb, int64_t N, int64_t &n, int &cb) {
    if (N >= 8) {
        const int64_t q = b >> 3;
        cb = (int)(q % ncb);
        n = q / ncb * 8 + (b & 7);
    } else {
        cb = (int)(b % ncb);
        n = b / ncb;
    }
}

#if !GRKAN_NORM_BACKWARD
// ============================================================ forward

template <int V, bool RAT, int K>
__global__ __launch_bounds__(512) void grkan_norm_token_fwd_kernel(NormArgs a) {
    __shared__ float lds[2 * 16];
    const NormPlan &p = a.p;
    const int t = (int)threadIdx.x, l = t & (p.T - 1);
    const int64_t slot = (int64_t)blockIdx.x * p.spw + t / p.T;
    const int g = (int)(slot % a.G);
    const int64_t step = p.blocks * p.spw / a.G;
    Cols<V, RAT> k[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int vi = l + i * p.T;
        k[i].init(a, g * a.D + min(vi, p.vpg - 1) * V, vi < p.vpg ? min(V, a.D - vi * V) : 0);
    }
    const float inv = 1.0f / (float)a.D;
    int phase = 0;
    // T <= 64: a slot ends when its samples do; larger T: the slot is the
    // workgroup, and n is the same in all its lanes
    for (int64_t n = slot / a.G; n < a.N; n += step) {
        Pack<V> x[K];
#pragma unroll
        for (int i = 0; i < K; ++i) x[i] = Pack<V>::load(at(a.x, n * a.xs + k[i].col), k[i].nv);
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) s[0] += x[i].get(e);
        slot_sum<1>(s, p.T, lds, phase);
        const float mean = s[0] * inv;
        float m2[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = e < k[i].nv ? x[i].get(e) - mean : 0.0f;
                m2[0] = fmaf(d, d, m2[0]);
            }
        slot_sum<1>(m2, p.T, lds, phase);
        const float rstd = rstd_of(m2[0] * inv, a.eps);
        if (l == 0) {
            a.mean[n * a.G + g] = mean;
            a.rstd[n * a.G + g] = rstd;
        }
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (k[i].nv > 0) apply_forward<V, RAT>(x[i], mean, rstd, k[i], a.act).store(at(a.y, n * a.C + k[i].col), k[i].nv);
    }
}

template <int V, bool RAT, int R>
__global__ __launch_bounds__(1024) void grkan_norm_slab_fwd_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const NormPlan &p = a.p;
    const int64_t total = p.blocks;
    const float inv = 1.0f / ((float)a.D * (float)a.S);
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        int64_t n;
        int cb;
        sample_block(b, p.ncb, a.N, n, cb);
        if (n >= a.N) continue;  // the same for the whole workgroup
        const Place q(a, cb);
        Cols<V, RAT> k;
        k.init(a, q.col, q.nv);
        const int S = (int)a.S;
        Pack<V> x[R];
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = q.ty + i * p.TY;
            x[i] = Pack<V>::load(at(a.x, n * a.xs + (r < S ? r : 0) * a.xr + k.col), r < S ? k.nv : 0);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) s[0] += x[i].get(e);
        group_sum<float, 1>(s, p, q.vpg, q.ngroups, q.jg, lds);
        const float mean = s[0] * inv;
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int nv = q.ty + i * p.TY < S ? k.nv : 0;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = e < nv ? x[i].get(e) - mean : 0.0f;
                s[0] = fmaf(d, d, s[0]);
            }
        }
        group_sum<float, 1>(s, p, q.vpg, q.ngroups, q.jg, lds);
        const float rstd = rstd_of(s[0] * inv, a.eps);
        if (q.on && q.ty == 0 && q.col % a.D == 0) {
            a.mean[n * a.G + q.g0 + q.jg] = mean;
            a.rstd[n * a.G + q.g0 + q.jg] = rstd;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = q.ty + i * p.TY;
            if (r < S && k.nv > 0)
                apply_forward<V, RAT>(x[i], mean, rstd, k, a.act).store(at(a.y, (n * a.S + r) * a.C + k.col), k.nv);
        }
    }
}

// Split, first pass: fp64 sums of x and x^2 of a row chunk of a column block.
template <int V>
__global__ __launch_bounds__(256) void grkan_norm_sums_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const NormPlan &p = a.p;
    const int64_t total = a.N * p.chunks * p.ncb;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int cb = (int)(b % p.ncb);
        const int64_t nc = b / p.ncb, n = nc / p.chunks, c = nc % p.chunks;
        const Place q(a, cb);
        const int64_t r1 = min(a.S, (c + 1) * p.chunk_rows);
        double s[2] = {0.0, 0.0};
        if (q.nv > 0) {
            const char *src = at(a.x, n * a.xs + q.col);
#pragma unroll 4
            for (int64_t r = c * p.chunk_rows + q.ty; r < r1; r += p.TY) {
                const Pack<V> x = Pack<V>::load(src + r * a.xr * ES, q.nv);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const double f = (double)x.get(e);
                    s[0] += f;
                    s[1] = fma(f, f, s[1]);
                }
            }
        }
        group_sum<double, 2>(s, p, q.vpg, q.ngroups, q.jg, lds);
        const int first = p.bpg == 1 ? q.jg * p.vpg : 0;
        if (q.ty == 0 && (int)threadIdx.x % p.TX == first && (int)threadIdx.x < p.TX && q.jg < q.ngroups) {
            const int part = p.bpg == 1 ? 0 : cb % p.bpg;
            double *o = a.stats + 2 * (((n * a.G + q.g0 + q.jg) * p.chunks + c) * p.bpg + part);
            o[0] = s[0];
            o[1] = s[1];
        }
    }
}

// Split, second step: one wave per (sample, group) adds the chunks' sums.
__global__ __launch_bounds__(256) void grkan_norm_stats_kernel(NormArgs a) {
    const int64_t ng = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (ng >= a.N * a.G) return;
    const int lane = (int)threadIdx.x & 63;
    const int64_t count = a.p.chunks * a.p.bpg;
    double s0 = 0.0, s1 = 0.0;
    for (int64_t i = lane; i < count; i += 64) {
        const double *o = a.stats + 2 * (ng * count + i);
        s0 += o[0];
        s1 += o[1];
    }
    for (int o = 32; o > 0; o >>= 1) {
        s0 += __shfl_xor(s0, o, 64);
        s1 += __shfl_xor(s1, o, 64);
    }
    if (lane == 0) {
        const double m = (double)a.D * (double)a.S, mean = s0 / m;
        a.mean[ng] = (float)mean;
        a.rstd[ng] = rstd_of((float)(s1 / m - mean * mean), a.eps);
    }
}

// Split, third step: y over a row chunk of a column block.
template <int V, bool RAT>
__global__ __launch_bounds__(256) void grkan_norm_apply_fwd_kernel(NormArgs a) {
    const NormPlan &p = a.p;
    const int64_t total = a.N * p.chunks * p.ncb;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int cb = (int)(b % p.ncb);
        const int64_t nc = b / p.ncb, n = nc / p.chunks, c = nc % p.chunks;
        const Place q(a, cb);
        if (q.nv == 0) continue;
        Cols<V, RAT> k;
        k.init(a, q.col, q.nv);
        const float mean = a.mean[n * a.G + q.g0 + q.jg], rstd = a.rstd[n * a.G + q.g0 + q.jg];
        const int64_t r1 = min(a.S, (c + 1) * p.chunk_rows);
#pragma unroll 4
        for (int64_t r = c * p.chunk_rows + q.ty; r < r1; r += p.TY)
            apply_forward<V, RAT>(Pack<V>::load(at(a.x, n * a.xs + r * a.xr + k.col), k.nv), mean, rstd, k, a.act)
                .store(at(a.y, (n * a.S + r) * a.C + k.col), k.nv);
    }
}

template <int V, bool RAT>
hipError_t forward_vec(const NormArgs &a, hipStream_t s) {
    const NormPlan &p = a.p;
    const dim3 grid((unsigned)(p.blocks < (1 << 20) ? p.blocks : (1 << 20))), block((unsigned)p.block);
    if (p.kind == kNormToken) {
        const dim3 tgrid((unsigned)p.blocks);
        switch (p.K) {
            case 1: hipLaunchKernelGGL((grkan_norm_token_fwd_kernel<V, RAT, 1>), tgrid, block, 0, s, a); break;
            case 2: hipLaunchKernelGGL((grkan_norm_token_fwd_kernel<V, RAT, 2>), tgrid, block, 0, s, a); break;
            case 3: hipLaunchKernelGGL((grkan_norm_token_fwd_kernel<V, RAT, 3>), tgrid, block, 0, s, a); break;
            default: hipLaunchKernelGGL((grkan_norm_token_fwd_kernel<V, RAT, 4>), tgrid, block, 0, s, a); break;
        }
        return hipGetLastError();
    }
    if (p.kind == kNormSlab) {
        if (p.regs <= 4)
            hipLaunchKernelGGL((grkan_norm_slab_fwd_kernel<V, RAT, 4>), grid, block, p.lds, s, a);
        else
            hipLaunchKernelGGL((grkan_norm_slab_fwd_kernel<V, RAT, 16>), grid, block, p.lds, s, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((grkan_norm_sums_kernel<V>), grid, block, p.lds, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(grkan_norm_stats_kernel, dim3((unsigned)((a.N * a.G + 3) / 4)), dim3(256), 0, s, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((grkan_norm_apply_fwd_kernel<V, RAT>), grid, block, 0, s, a);
    return hipGetLastError();
}

#else
// ============================================================ backward

// Writes a lane's column sums, added over the row lanes of the workgroup (and,
// for token plans, over its slots of one group), to row `prow` of the
// partials.  `lds` holds block * min(values, kBatch) floats.
constexpr int kBatch = 13;

template <int V, bool RAT>
__device__ static inline void store_col_sums(const NormArgs &a, const ColSums<V, RAT> &cs, int width, int depth,
                                             int lane, int64_t prow, int col, int nv, int64_t access, float *lds) {
    constexpr int NVAL = ColSums<V, RAT>::kValues;
    const int t = (int)threadIdx.x, block = a.p.block;
    const bool writer = lane == 0;
    float *out = a.partials + prow * norm_partial_row(a.p, a.C, RAT);
#pragma unroll
    for (int i0 = 0; i0 < NVAL; i0 += kBatch) {
        __syncthreads();
#pragma unroll
        for (int i = i0; i < NVAL && i < i0 + kBatch; ++i) lds[(i - i0) * block + t] = nv > 0 ? cs.get(i) : 0.0f;
        __syncthreads();
        if (writer && nv > 0) {
#pragma unroll
            for (int i = i0; i < NVAL && i < i0 + kBatch; ++i) {
                float s = 0.0f;
                for (int q = 0; q < depth; ++q) s += lds[(i - i0) * block + t + q * width];
                if (i < V) {
                    if (i < nv) out[col + i] = s;
                } else if (i < 2 * V) {
                    if (i - V < nv) out[a.C + col + i - V] = s;
                } else {
                    out[2 * (int64_t)a.C + (int64_t)(i - 2 * V) * a.p.cv + access] = s;
                }
            }
        }
    }
}

template <int V, bool RAT, int K>
__global__ __launch_bounds__(512) void grkan_norm_token_bwd_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char ldsb[];
    float *lds = reinterpret_cast<float *>(ldsb);
    const NormPlan &p = a.p;
    const int t = (int)threadIdx.x, l = t & (p.T - 1), sl = t / p.T;
    const int64_t slot = (int64_t)blockIdx.x * p.spw + sl;
    const int g = (int)(slot % a.G);
    const int64_t step = p.blocks * p.spw / a.G;
    Cols<V, RAT> k[K];
    ColSums<V, RAT> cs[K];
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int vi = l + i * p.T;
        k[i].init(a, g * a.D + min(vi, p.vpg - 1) * V, vi < p.vpg ? min(V, a.D - vi * V) : 0);
        cs[i].clear();
    }
    const float inv = 1.0f / (float)a.D;
    int phase = 0;
    for (int64_t n = slot / a.G; n < a.N; n += step) {
        const float mean = a.mean[n * a.G + g], rstd = a.rstd[n * a.G + g];
        Pack<V> x[K], dy[K];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            x[i] = Pack<V>::load(at(a.x, n * a.xs + k[i].col), k[i].nv);
            dy[i] = Pack<V>::load(at(a.dy, n * a.ds + k[i].col), k[i].nv);
        }
        float m[2] = {0.0f, 0.0f};
        float tt[K][V], xh[K][V];
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const bool in = e < k[i].nv;
                const float dh = slope<V, RAT>(in ? x[i].get(e) : mean, in ? dy[i].get(e) : 0.0f, mean, rstd, k[i], e,
                                               a.act, cs[i].coef, xh[i][e]);
                cs[i].db[e] += dh;
                cs[i].dw[e] = fmaf(dh, xh[i][e], cs[i].dw[e]);
                tt[i][e] = dh * k[i].w[e];
                m[0] += tt[i][e];
                m[1] = fmaf(tt[i][e], xh[i][e], m[1]);
            }
        slot_sum<2>(m, p.T, lds, phase);
        const float m1 = m[0] * inv, m2 = m[1] * inv;
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (k[i].nv > 0) {
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] = rstd * (tt[i][e] - m1 - xh[i][e] * m2);
                Pack<V>::from(f).store(at(a.y, n * a.C + k[i].col), k[i].nv);
            }
    }
    // slots of one group in this workgroup: spw / G of them, G slots apart
    // (slot = workgroup * spw + sl, spw a multiple of G), or each its own
    const int depth = p.spw > a.G ? p.spw / a.G : 1;
    const int64_t prow = p.spw > a.G ? (int64_t)blockIdx.x : slot / a.G;
    const int first = p.spw > a.G ? (sl < a.G ? 0 : 1) : 0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        const int vi = l + i * p.T;
        store_col_sums<V, RAT>(a, cs[i], a.G * p.T, depth, first, prow, k[i].col, k[i].nv,
                               (int64_t)g * p.vpg + vi, lds);
    }
}

template <int V, bool RAT, int R>
__global__ __launch_bounds__(512) void grkan_norm_slab_bwd_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const NormPlan &p = a.p;
    const float inv = 1.0f / ((float)a.D * (float)a.S);
    int64_t n0;
    int cb;
    sample_block(blockIdx.x, p.ncb, p.chunks, n0, cb);
    if (n0 >= p.chunks) return;  // the whole workgroup
    const Place q(a, cb);
    Cols<V, RAT> k;
    k.init(a, q.col, q.nv);
    ColSums<V, RAT> cs;
    cs.clear();
    const int S = (int)a.S;
    for (int64_t n = n0; n < a.N; n += p.chunks) {
        const float mean = a.mean[n * a.G + q.g0 + q.jg], rstd = a.rstd[n * a.G + q.g0 + q.jg];
        Pack<V> x[R], dy[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = q.ty + i * p.TY;
            const int nv = r < S ? k.nv : 0;
            const int64_t rr = r < S ? r : 0;
            x[i] = Pack<V>::load(at(a.x, n * a.xs + rr * a.xr + k.col), nv);
            dy[i] = Pack<V>::load(at(a.dy, n * a.ds + rr * a.dr + k.col), nv);
        }
        float m[2] = {0.0f, 0.0f};
        float tt[R][V];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int nv = q.ty + i * p.TY < S ? k.nv : 0;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const bool in = e < nv;
                float xh;
                const float dh = slope<V, RAT>(in ? x[i].get(e) : mean, in ? dy[i].get(e) : 0.0f, mean, rstd, k, e,
                                               a.act, cs.coef, xh);
                cs.db[e] += dh;
                cs.dw[e] = fmaf(dh, xh, cs.dw[e]);
                tt[i][e] = dh * k.w[e];
                m[0] += tt[i][e];
                m[1] = fmaf(tt[i][e], xh, m[1]);
            }
        }
        group_sum<float, 2>(m, p, q.vpg, q.ngroups, q.jg, lds);
        const float m1 = m[0] * inv, m2 = m[1] * inv;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = q.ty + i * p.TY;
            if (r < S && k.nv > 0) {
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] = rstd * (tt[i][e] - m1 - (x[i].get(e) - mean) * rstd * m2);
                Pack<V>::from(f).store(at(a.y, (n * a.S + r) * a.C + k.col), k.nv);
            }
        }
    }
    store_col_sums<V, RAT>(a, cs, p.TX, p.TY, q.ty, n0, k.col, k.nv, q.access(a), reinterpret_cast<float *>(lds));
}

// Split, first pass: sums of t and t xh and the column sums of a row chunk.
template <int V, bool RAT>
__global__ __launch_bounds__(256) void grkan_norm_sums_bwd_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const NormPlan &p = a.p;
    const int64_t total = a.N * p.chunks * p.ncb;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int cb = (int)(b % p.ncb);
        const int64_t nc = b / p.ncb, n = nc / p.chunks, c = nc % p.chunks;
        const Place q(a, cb);
        Cols<V, RAT> k;
        k.init(a, q.col, q.nv);
        ColSums<V, RAT> cs;
        cs.clear();
        const int64_t r1 = min(a.S, (c + 1) * p.chunk_rows);
        double s[2] = {0.0, 0.0};
        if (q.nv > 0) {
            const float mean = a.mean[n * a.G + q.g0 + q.jg], rstd = a.rstd[n * a.G + q.g0 + q.jg];
#pragma unroll 2
            for (int64_t r = c * p.chunk_rows + q.ty; r < r1; r += p.TY) {
                const Pack<V> x = Pack<V>::load(at(a.x, n * a.xs + r * a.xr + k.col), k.nv);
                const Pack<V> dy = Pack<V>::load(at(a.dy, n * a.ds + r * a.dr + k.col), k.nv);
                float m1 = 0.0f, m2 = 0.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const bool in = e < k.nv;
                    float xh;
                    const float dh = slope<V, RAT>(in ? x.get(e) : mean, in ? dy.get(e) : 0.0f, mean, rstd, k, e,
                                                   a.act, cs.coef, xh);
                    cs.db[e] += dh;
                    cs.dw[e] = fmaf(dh, xh, cs.dw[e]);
                    const float t = dh * k.w[e];
                    m1 += t;
                    m2 = fmaf(t, xh, m2);
                }
                s[0] += (double)m1;
                s[1] += (double)m2;
            }
        }
        group_sum<double, 2>(s, p, q.vpg, q.ngroups, q.jg, lds);
        const int first = p.bpg == 1 ? q.jg * p.vpg : 0;
        if (q.ty == 0 && (int)threadIdx.x % p.TX == first && (int)threadIdx.x < p.TX && q.jg < q.ngroups) {
            const int part = p.bpg == 1 ? 0 : cb % p.bpg;
            double *o = a.stats + 2 * (((n * a.G + q.g0 + q.jg) * p.chunks + c) * p.bpg + part);
            o[0] = s[0];
            o[1] = s[1];
        }
        store_col_sums<V, RAT>(a, cs, p.TX, p.TY, q.ty, n * p.chunks + c, k.col, k.nv, q.access(a),
                               reinterpret_cast<float *>(lds));
        __syncthreads();
    }
}

// Split, second step: <t> and <t xh>, one wave per (sample, group).
__global__ __launch_bounds__(256) void grkan_norm_means_kernel(NormArgs a) {
    const int64_t ng = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (ng >= a.N * a.G) return;
    const int lane = (int)threadIdx.x & 63;
    const int64_t count = a.p.chunks * a.p.bpg;
    double s0 = 0.0, s1 = 0.0;
    for (int64_t i = lane; i < count; i += 64) {
        const double *o = a.stats + 2 * (ng * count + i);
        s0 += o[0];
        s1 += o[1];
    }
    for (int o = 32; o > 0; o >>= 1) {
        s0 += __shfl_xor(s0, o, 64);
        s1 += __shfl_xor(s1, o, 64);
    }
    if (lane == 0) {
        const double m = (double)a.D * (double)a.S;
        a.means[2 * ng] = (float)(s0 / m);
        a.means[2 * ng + 1] = (float)(s1 / m);
    }
}

// Split, third step: dx over a row chunk.  The slope is formed again: keeping
// it would cost a write and a read of a tensor.
template <int V, bool RAT>
__global__ __launch_bounds__(256) void grkan_norm_apply_bwd_kernel(NormArgs a) {
    const NormPlan &p = a.p;
    const int64_t total = a.N * p.chunks * p.ncb;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int cb = (int)(b % p.ncb);
        const int64_t nc = b / p.ncb, n = nc / p.chunks, c = nc % p.chunks;
        const Place q(a, cb);
        if (q.nv == 0) continue;
        Cols<V, RAT> k;
        k.init(a, q.col, q.nv);
        const int64_t ng = n * a.G + q.g0 + q.jg;
        const float mean = a.mean[ng], rstd = a.rstd[ng], m1 = a.means[2 * ng], m2 = a.means[2 * ng + 1];
        const int64_t r1 = min(a.S, (c + 1) * p.chunk_rows);
        float unused[10] = {};
#pragma unroll 2
        for (int64_t r = c * p.chunk_rows + q.ty; r < r1; r += p.TY) {
            const Pack<V> x = Pack<V>::load(at(a.x, n * a.xs + r * a.xr + k.col), k.nv);
            const Pack<V> dy = Pack<V>::load(at(a.dy, n * a.ds + r * a.dr + k.col), k.nv);
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float xh;
                const float dh = slope<V, RAT>(x.get(e), dy.get(e), mean, rstd, k, e, a.act, unused, xh);
                f[e] = rstd * (dh * k.w[e] - m1 - xh * m2);
            }
            Pack<V>::from(f).store(at(a.y, (n * a.S + r) * a.C + k.col), k.nv);
        }
    }
}

// The column partials added over their rows in fp64: workgroups of 64 columns
// x 16 row lanes for dw and db, then one workgroup per (activation group,
// coefficient), whose accesses are a contiguous range.
template <bool RAT>
__global__ __launch_bounds__(1024) void grkan_norm_columns_kernel(NormArgs a) {
    __shared__ double red[1024];
    const int t = (int)threadIdx.x;
    const int64_t row = norm_partial_row(a.p, a.C, RAT), P = a.p.prows;
    const int64_t colblocks = (2 * (int64_t)a.C + 63) / 64;
    if ((int64_t)blockIdx.x < colblocks) {
        const int64_t c = (int64_t)blockIdx.x * 64 + (t & 63);
        double s = 0.0;
        if (c < 2 * (int64_t)a.C) {
#pragma unroll 8
            for (int64_t r = t >> 6; r < P; r += 16) s += (double)a.partials[r * row + c];
        }
        red[t] = s;
        __syncthreads();
        if (t < 64 && c < 2 * (int64_t)a.C) {
            for (int q = 1; q < 16; ++q) s += red[t + 64 * q];
            if (c < a.C) {
                if (a.dw) a.dw[c] = (float)s;
            } else if (a.db) {
                a.db[c - a.C] = (float)s;
            }
        }
        return;
    }
    if constexpr (RAT) {
        const int64_t gk = blockIdx.x - colblocks;
        const int g = (int)(gk / 10), k = (int)(gk % 10);
        // accesses of columns [g dga, (g + 1) dga): they never straddle a boundary
        const int64_t c0 = (int64_t)g * a.dga, c1 = c0 + a.dga;
        const int64_t v0 = c0 / a.D * a.p.vpg + (c0 % a.D + a.p.vec - 1) / a.p.vec;
        const int64_t v1 = c1 / a.D * a.p.vpg + (c1 % a.D + a.p.vec - 1) / a.p.vec;
        const int64_t w = v1 - v0;
        double s = 0.0;
#pragma unroll 8
        for (int64_t i = t; i < P * w; i += 1024) {
            const int64_t r = i / w;
            s += (double)a.partials[r * row + 2 * (int64_t)a.C + k * a.p.cv + v0 + (i - r * w)];
        }
        red[t] = s;
        __syncthreads();
        for (int o = 512; o > 0; o >>= 1) {
            if (t < o) red[t] += red[t + o];
            __syncthreads();
        }
        if (t == 0) {
            if (k < 6)
                a.dA[g * 6 + k] = (float)red[0];
            else
                a.dB[g * 4 + k - 6] = (float)red[0];
        }
    }
}

template <int V, bool RAT>
hipError_t backward_vec(const NormArgs &a, hipStream_t s) {
    const NormPlan &p = a.p;
    const dim3 block((unsigned)p.block);
    hipError_t e;
    if (p.kind == kNormToken) {
        const dim3 grid((unsigned)p.blocks);
        switch (p.K) {
            case 1: hipLaunchKernelGGL((grkan_norm_token_bwd_kernel<V, RAT, 1>), grid, block, p.lds, s, a); break;
            case 2: hipLaunchKernelGGL((grkan_norm_token_bwd_kernel<V, RAT, 2>), grid, block, p.lds, s, a); break;
            case 3: hipLaunchKernelGGL((grkan_norm_token_bwd_kernel<V, RAT, 3>), grid, block, p.lds, s, a); break;
            default: hipLaunchKernelGGL((grkan_norm_token_bwd_kernel<V, RAT, 4>), grid, block, p.lds, s, a); break;
        }
    } else if (p.kind == kNormSlab) {
        const dim3 grid((unsigned)p.blocks);
        if (p.regs <= 2)
            hipLaunchKernelGGL((grkan_norm_slab_bwd_kernel<V, RAT, 2>), grid, block, p.lds, s, a);
        else
            hipLaunchKernelGGL((grkan_norm_slab_bwd_kernel<V, RAT, 8>), grid, block, p.lds, s, a);
    } else {
        const dim3 grid((unsigned)(p.blocks < (1 << 20) ? p.blocks : (1 << 20)));
        hipLaunchKernelGGL((grkan_norm_sums_bwd_kernel<V, RAT>), grid, block, p.lds, s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL(grkan_norm_means_kernel, dim3((unsigned)((a.N * a.G + 3) / 4)), dim3(256), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL((grkan_norm_apply_bwd_kernel<V, RAT>), grid, block, 0, s, a);
    }
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t groups = RAT ? (int64_t)a.ng * 10 : 0;
    if (!a.dw && !a.db && !RAT) return hipSuccess;
    const dim3 rgrid((unsigned)((2 * (int64_t)a.C + 63) / 64 + groups));
    hipLaunchKernelGGL((grkan_norm_columns_kernel<RAT>), rgrid, dim3(1024), 0, s, a);
    return hipGetLastError();
}
#endif

template <int V>
hipError_t launch_vec(const NormArgs &a, hipStream_t s) {
#if GRKAN_NORM_BACKWARD
    return a.act == GRKAN_ACT_RATIONAL ? backward_vec<V, true>(a, s) : backward_vec<V, false>(a, s);
#else
    return a.act == GRKAN_ACT_RATIONAL ? forward_vec<V, true>(a, s) : forward_vec<V, false>(a, s);
#endif
}

}  // namespace

#if GRKAN_NORM_BACKWARD
template <> hipError_t launch_norm_backward<NormIo>(const NormArgs &a, hipStream_t s) {
#else
template <> hipError_t launch_norm_forward<NormIo>(const NormArgs &a, hipStream_t s) {
#endif
    switch (a.p.vec) {
        case 8:
            if constexpr (kMaxV >= 8) return launch_vec<8>(a, s);
            return hipErrorInvalidValue;
        case 4: return launch_vec<4>(a, s);
        case 2: return launch_vec<2>(a, s);
        case 1: return launch_vec<1>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace grkan
