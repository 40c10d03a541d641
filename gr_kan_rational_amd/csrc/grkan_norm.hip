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
// of x and x^2 are fp64 instead, from fp32 differences of at most 32 rows to the
// first of them, which leaves var good to 2^-53 (mean / std)^2 and, where such
// first rows alone make up a group's variance, to 2^-16 (a lane's sum of squares,
// worst of 400 such columns; a large first position in whole tensors stayed
// within 64 2^-24).
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
    // Keeps the compiler from holding the unpacked values from one use to the
    // next: unpacking again costs an instruction an element, holding them up to
    // twice the registers.
    __device__ inline void repack() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            uint32_t w = r[i];
            asm volatile("" : "+v"(w));
            r[i] = w;
        }
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

// n <= V fp32 parameters at p (absent pointers give `none`), the rest zeros.
template <int V> __device__ static inline void load_params(const float *p, int n, float none, float (&f)[V]) {
    typedef float fvec __attribute__((ext_vector_type(V)));
    typedef fvec any __attribute__((aligned(4)));
    if (p && n == V) {
        if constexpr (V > 1) {
            const fvec v = *reinterpret_cast<const any *>(p);
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = v[e];
        } else {
            f[0] = p[0];
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = e < n ? (p ? p[e] : none) : 0.0f;
}

// A lane's columns: weight, bias and (rational) the coefficients of their one
// activation group.  Absent columns get weight 0.
template <int V, bool RAT> struct Cols {
    int col, nv;
    float w[V], b[V];
    Coefs<5, 4> c;

    __device__ inline void init(const NormArgs &a, int col_, int nv_) {
        col = col_;
        nv = nv_;
        load_params<V>(a.w ? a.w + col : nullptr, nv, 1.0f, w);
        load_params<V>(a.b ? a.b + col : nullptr, nv, 0.0f, b);
        if constexpr (RAT) c = load_coefs<5, 4>(a.A, a.B, nv > 0 ? col / a.dga : 0);
    }
};

// Statistics of a lane's elements: one pair, or one per element where accesses
// straddle groups.
template <int V, bool MIXED> struct Stats {
    static constexpr int N = MIXED ? V : 1;
    float mean[N], rstd[N];
    __device__ inline float m(int e) const { return mean[MIXED ? e : 0]; }
    __device__ inline float r(int e) const { return rstd[MIXED ? e : 0]; }
};

// y of one access.  The mean is subtracted first, which is exact for values
// near it; rstd w is one factor.
template <int V, bool RAT, bool MIXED>
__device__ static inline Pack<V> apply_forward(const Pack<V> &x, const Stats<V, MIXED> &s, const Cols<V, RAT> &k,
                                               int act) {
    float f[V];
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = act_value<RAT>(fmaf(x.get(e) - s.m(e), s.r(e) * k.w[e], k.b[e]), act, k.c);
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
};

// dh at xh of element e.
template <int V, bool RAT>
__device__ static inline float slope(float xh, float dy, const Cols<V, RAT> &k, const SlopeCoefs &sc, int e, int act,
                                     float *coef) {
    const float h = fmaf(xh, k.w[e], k.b[e]);
    if constexpr (RAT)
        return rational_slope(h, dy, sc, *reinterpret_cast<float (*)[10]>(coef));
    else
        return dy * act_slope(h, act);
}

// A token lane's K accesses: columns, weights, biases and the rational's
// coefficients.  The accesses of a group's lanes interleave (access l + i T),
// which coalesces, and each has a set of coefficients (RAT 1).  RUN: a lane
// takes K V consecutive columns instead, so that one set, or two where runs
// straddle activation groups (RAT 2: the second from element `split` of the run
// on), serves them all.  The backward of the rational, which also sums per
// set, is bound by its arithmetic and takes runs (at 48 bytes a lane the forward
// spent its time in the address units instead: 65 us against 44 at 50,432 x
// 768).
template <int V, int RAT, int K, bool RUN> struct TokenCols {
    static constexpr int kSets = RAT == 0 ? 1 : (RUN ? RAT : K);
    int col[K], nv[K], split;
    float w[K][V], b[K][V];
    Coefs<5, 4> c[kSets];

    __device__ inline void init(const NormArgs &a, int g, int l) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int first = (RUN ? l * K + i : l + i * a.p.T) * V;
            nv[i] = min(max(a.D - first, 0), V);
            col[i] = g * a.D + (nv[i] > 0 ? first : 0);
            load_params<V>(a.w ? a.w + col[i] : nullptr, nv[i], 1.0f, w[i]);
            load_params<V>(a.b ? a.b + col[i] : nullptr, nv[i], 0.0f, b[i]);
        }
        split = K * V;
        if constexpr (RAT != 0 && !RUN) {
#pragma unroll
            for (int i = 0; i < K; ++i) c[i] = load_coefs<5, 4>(a.A, a.B, col[i] / a.dga);
        } else if constexpr (RAT != 0) {
            const int group = col[0] / a.dga;
            c[0] = load_coefs<5, 4>(a.A, a.B, group);
            if constexpr (RAT == 2) {
                split = (group + 1) * a.dga - col[0];
                c[1] = load_coefs<5, 4>(a.A, a.B, min(group + 1, a.ng - 1));
            }
        }
    }
    // the coefficients of element j = i V + e
    __device__ inline Coefs<5, 4> coefs(int j) const {
        if constexpr (!RUN) {
            return c[RAT ? j / V : 0];
        } else if constexpr (RAT == 2) {
            Coefs<5, 4> k;
#pragma unroll
            for (int i = 0; i < 6; ++i) k.a[i] = j < split ? c[0].a[i] : c[1].a[i];
#pragma unroll
            for (int i = 0; i < 4; ++i) k.b[i] = j < split ? c[0].b[i] : c[1].b[i];
            return k;
        } else {
            return c[0];
        }
    }
};

// ------------------------------------------------------------ reductions

__device__ static inline float rstd_of(float var, float eps) { return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps); }

// v of the lane that the DPP control names (all lanes are named by some lane).
template <int CTRL> __device__ static inline float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// Sum of v over aligned runs of T <= 64 lanes (T a power of two), in each of
// them: within 16 lanes by DPP (quads by permutation, then the mirrored half and
// the mirrored row, whose lanes already agree), beyond by swapping rows.
__device__ static inline float lane_sum(float v, int T) {
    if (T > 1) v += dpp<0xb1>(v);
    if (T > 2) v += dpp<0x4e>(v);
    if (T > 4) v += dpp<0x141>(v);
    if (T > 8) v += dpp<0x140>(v);
    if (T > 16) {
        const auto w = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(w[0]) + __uint_as_float(w[1]);
    }
    if (T > 32) {
        const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(w[0]) + __uint_as_float(w[1]);
    }
    return v;
}

// Sum of v over the T lanes of a slot, in every one of them.  T > 64 is the
// whole workgroup: one value per wave through LDS (two buffers of 16 NV floats
// used in turn, so that one barrier per call is enough).
template <int NV>
__device__ static inline void slot_sum(float (&v)[NV], int T, float *lds, int &phase) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = lane_sum(v[i], T);
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

// A lane's place in a column block.
struct Place {
    int c0, width;           // the block's columns
    int g0, ngroups;         // its groups (the first and last may reach outside it)
    int col, nv, tx, ty;
    int first, edge;         // the lane's first element's group, counted from g0, and where the next begins
    __device__ inline Place(const NormArgs &a, int cb) {
        const NormPlan &p = a.p;
        const int t = (int)threadIdx.x;
        ty = t / p.TX;
        tx = t - ty * p.TX;
        c0 = cb * p.width;
        width = min(p.width, a.C - c0);
        g0 = c0 / a.D;
        ngroups = (c0 + width - 1) / a.D - g0 + 1;
        col = c0 + tx * p.vec;
        nv = ty < p.TY ? min(max(width - tx * p.vec, 0), p.vec) : 0;
        const int g = min(col, c0 + width - 1) / a.D;
        first = g - g0;
        edge = (g + 1) * a.D - col;
    }
    // group of element e, counted from g0 (clamped for absent elements); an
    // access lies in at most two groups unless groups are shorter than it
    __device__ inline int group(const NormArgs &a, int e) const {
        if (a.D >= a.p.vec) return min(first + (e < edge ? 0 : 1), ngroups - 1);
        return min(col + e, c0 + width - 1) / a.D - g0;
    }
};

// Sums over each group of a column block: v[i][e] is value i of element e (of
// the whole access unless MIXED) in this lane; afterwards the sum over the
// element's group, of its columns in this block.  First over the row lanes of
// each column (p.P lanes a column), then over the columns of each group (p.L
// lanes a group).  `lds` holds NV * (E * (threads + TX) + groups) values, E = V
// if MIXED else 1.
template <class R, int NV, int V, bool MIXED>
__device__ static inline void group_sum(R (&v)[NV][MIXED ? V : 1], const NormArgs &a, const Place &q, char *ldsb) {
    constexpr int E = MIXED ? V : 1;
    const NormPlan &p = a.p;
    R *red = reinterpret_cast<R *>(ldsb);
    R *sums = red + NV * E * p.block;
    R *res = sums + NV * E * p.TX;
    const int t = (int)threadIdx.x, ncols = E * p.TX;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) red[(i * E + e) * p.block + t] = v[i][e];
    __syncthreads();
    for (int c = t / p.P; c < ncols; c += p.block / p.P) {
        const int l = t & (p.P - 1), at = (c % E) * p.block + c / E;
        R s[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = 0;
        for (int r = l; r < p.TY; r += p.P)
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] += red[i * E * p.block + at + r * p.TX];
        for (int o = p.P >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] += __shfl_xor(s[i], o, 64);
        if (l == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) sums[i * ncols + c] = s[i];
        }
    }
    __syncthreads();
    for (int j = t / p.L; j < q.ngroups; j += p.block / p.L) {
        // the group's columns in this block; accesses unless MIXED
        int lo = max((q.g0 + j) * a.D - q.c0, 0), hi = min((q.g0 + j + 1) * a.D - q.c0, q.width);
        if constexpr (!MIXED) lo /= V, hi /= V;
        R s[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = 0;
        for (int c = lo + (t & (p.L - 1)); c < hi; c += p.L)
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] += sums[i * ncols + c];
        for (int o = p.L >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < NV; ++i) s[i] += __shfl_xor(s[i], o, 64);
        if ((t & (p.L - 1)) == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) res[i * p.groups + j] = s[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int j = q.group(a, e);
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i][e] = res[i * p.groups + j];
    }
}

// The groups' sums of a block as group_sum left them in LDS.
template <class R, int NV, int E>
__device__ static inline const R *group_results(const NormPlan &p, const char *ldsb) {
    return reinterpret_cast<const R *>(ldsb) + NV * E * (p.block + p.TX);
}

__device__ static inline const char *at(const void *base, int64_t e) {
    return static_cast<const char *>(base) + e * ES;
}
__device__ static inline char *at(void *base, int64_t e) { return static_cast<char *>(base) + e * ES; }

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

// Split: the block's group sums (pairs in LDS after group_sum) as this chunk's
// and block's part of each group.
template <int E>
__device__ static inline void store_parts(const NormArgs &a, const Place &q, int64_t n, int64_t c, int cb,
                                          const char *lds) {
    const NormPlan &p = a.p;
    const double *res = group_results<double, 2, E>(p, lds);
    for (int j = (int)threadIdx.x; j < q.ngroups; j += p.block) {
        const int g = q.g0 + j, part = cb - g * a.D / p.width;
        double *o = a.stats + 2 * (((n * a.G + g) * p.chunks + c) * p.parts + part);
        o[0] = res[j];
        o[1] = res[p.groups + j];
    }
}

// Blocks that group g lies in.
__device__ static inline int group_parts(const NormArgs &a, int g) {
    return ((g + 1) * a.D - 1) / a.p.width - g * a.D / a.p.width + 1;
}

// A group's statistics from the sums of x and x^2 (forward), or <t> and <t xh>
// from theirs (backward).
__device__ static inline float2 of_sums(const NormArgs &a, double s0, double s1) {
    const double m = (double)a.D * (double)a.S;
#if GRKAN_NORM_BACKWARD
    return float2{(float)(s0 / m), (float)(s1 / m)};
#else
    const double mean = s0 / m;
    return float2{(float)mean, rstd_of((float)(s1 / m - mean * mean), a.eps)};
#endif
}

// Split: the sum of a group's parts, by a workgroup of 256; in thread 0.
__device__ static inline void add_parts(const NormArgs &a, int64_t ng, double &s0, double &s1) {
    __shared__ double red[2][4];
    const NormPlan &p = a.p;
    const int g = (int)(ng % a.G), t = (int)threadIdx.x, parts = group_parts(a, g);
    const int64_t count = p.chunks * p.parts;
    s0 = s1 = 0.0;
#pragma unroll 4
    for (int64_t i = t; i < count; i += 256) {
        if ((int)(i % p.parts) >= parts) continue;
        const double *o = a.stats + 2 * (ng * count + i);
        s0 += o[0];
        s1 += o[1];
    }
    for (int o = 32; o > 0; o >>= 1) {
        s0 += __shfl_xor(s0, o, 64);
        s1 += __shfl_xor(s1, o, 64);
    }
    if ((t & 63) == 0) red[0][t >> 6] = s0, red[1][t >> 6] = s1;
    __syncthreads();
    if (t == 0) {
        s0 = red[0][0] + red[0][1] + red[0][2] + red[0][3];
        s1 = red[1][0] + red[1][1] + red[1][2] + red[1][3];
    }
    __syncthreads();  // the sums in LDS have been read
}

// Split, few parts: each workgroup of the second pass adds the parts of its
// groups itself (p.L lanes a group, the same order in every workgroup) and
// leaves the statistics in LDS.
__device__ static inline void own_parts(const NormArgs &a, const Place &q, int64_t n, float2 *stats) {
    const NormPlan &p = a.p;
    const int t = (int)threadIdx.x, l = t & (p.L - 1);
    const int count = (int)(p.chunks * p.parts);
    for (int j = t / p.L; j < q.ngroups; j += p.block / p.L) {
        const int parts = group_parts(a, q.g0 + j);
        const double *o = a.stats + 2 * (n * a.G + q.g0 + j) * (int64_t)count;
        double s0 = 0.0, s1 = 0.0;
#pragma unroll 4
        for (int i = l; i < count; i += p.L) {
            if (p.parts > 1 && i % p.parts >= parts) continue;
            s0 += o[2 * i];
            s1 += o[2 * i + 1];
        }
        for (int u = p.L >> 1; u > 0; u >>= 1) {
            s0 += __shfl_xor(s0, u, 64);
            s1 += __shfl_xor(s1, u, 64);
        }
        if (l == 0) stats[j] = of_sums(a, s0, s1);
    }
    __syncthreads();
}

// Workgroups of a launch that has one for each (sample, group) while they are
// not too many.
unsigned group_blocks(const NormArgs &a) { return (unsigned)(a.N * a.G < kMaxBlocks ? a.N * a.G : kMaxBlocks); }

// Launches KERN with `lds` bytes of dynamic LDS, which may pass the 64 KB a kernel
// has without asking.
template <auto KERN>
hipError_t start(const NormArgs &a, dim3 grid, dim3 block, size_t lds, hipStream_t s) {
    if (lds > (64u << 10)) {
        static const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(KERN),
                                                        hipFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxLds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(KERN, grid, block, lds, s, a);
    return hipGetLastError();
}

#if !GRKAN_NORM_BACKWARD
// ============================================================ forward

// Token: a group of one position lies in T lanes' registers; sums by lane
// exchanges (LDS beyond a wave), mean first, then the variance about it.  The
// next sample's values are on their way while this one's are worked on.
// 50,432 x 768, bf16, the rational: 44 us, 3.5 TB/s of 5.0; the vector units are
// busy 0.93 of the CUs' time, which bounds it.  1 x 768: 5.3 us, latency.
template <int V, int RAT, int K>
__global__ __launch_bounds__(K * V == 1 ? 1024 : 256) void grkan_norm_token_fwd_kernel(NormArgs a) {
    __shared__ float lds[2 * 16];
    const NormPlan &p = a.p;
    const int t = (int)threadIdx.x, l = t & (p.T - 1);
    const int64_t slot = (int64_t)blockIdx.x * p.spw + t / p.T;
    const int g = (int)(slot % a.G);
    const int64_t step = p.blocks * p.spw / a.G;
    const float inv = 1.0f / (float)a.D;
    int phase = 0;
    TokenCols<V, RAT, K, RAT == 2> k;
    k.init(a, g, l);
    // T <= 64: a slot ends when its samples do; larger T: the slot is the
    // workgroup, and n is the same in all its lanes.  The next sample's values
    // are on their way while this one's are reduced.
    int64_t n = slot / a.G;
    Pack<V> next[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
        next[i] = Pack<V>::load(at(a.x, (n < a.N ? n : 0) * a.xs + k.col[i]), n < a.N ? k.nv[i] : 0);
    for (; n < a.N; n += step) {
        Pack<V> x[K];
        const int64_t nn = n + step < a.N ? n + step : n;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            x[i] = next[i];
            next[i] = Pack<V>::load(at(a.x, nn * a.xs + k.col[i]), k.nv[i]);
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) s[0] += x[i].get(e);
        slot_sum<1>(s, p.T, lds, phase);
        const float mean = s[0] * inv;
        float m2[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < K; ++i) {
            x[i].repack();
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = e < k.nv[i] ? x[i].get(e) - mean : 0.0f;
                m2[0] = fmaf(d, d, m2[0]);
            }
        }
        slot_sum<1>(m2, p.T, lds, phase);
        const float rstd = rstd_of(m2[0] * inv, a.eps);
        if (l == 0) {
            a.mean[n * a.G + g] = mean;
            a.rstd[n * a.G + g] = rstd;
        }
#pragma unroll
        for (int i = 0; i < K; ++i) {
            x[i].repack();
            if (k.nv[i] > 0) {
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    f[e] = act_value<RAT != 0>(fmaf((x[i].get(e) - mean) * rstd, k.w[i][e], k.b[i][e]), a.act,
                                               k.coefs(i * V + e));
                Pack<V>::from(f).store(at(a.y, n * a.C + k.col[i]), k.nv[i]);
            }
        }
    }
}

// Slab: whole groups of a sample, all positions, in a workgroup's registers;
// one read of x, the variance about the mean.  Rows are cut into pieces of 64
// bytes or more: with 20- and 40-byte pieces (8 x 4,096 x 320, bf16, 32 groups,
// held in registers all the same) it ran 58 and 42 us against the split's 28.
template <int V, bool RAT, bool MIXED, int R>
__global__ __launch_bounds__(1024) void grkan_norm_slab_fwd_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int E = MIXED ? V : 1;
    const NormPlan &p = a.p;
    const float inv = 1.0f / ((float)a.D * (float)a.S);
    for (int64_t b = blockIdx.x; b < p.blocks; b += gridDim.x) {
        int64_t n;
        int cb;
        sample_block(b, p.ncb, a.N, n, cb);
        if (n >= a.N) continue;  // the same for the whole workgroup
        const Place q(a, cb);
        const int S = (int)a.S;
        Pack<V> x[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = q.ty + i * p.TY;
            x[i] = Pack<V>::load(at(a.x, n * a.xs + (r < S ? r : 0) * a.xr + q.col), r < S ? q.nv : 0);
        }
        Cols<V, RAT> k;
        k.init(a, q.col, q.nv);
        // absent elements are zeros, and absent rows
        float s[1][E] = {};
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) s[0][MIXED ? e : 0] += x[i].get(e);
        group_sum<float, 1, V, MIXED>(s, a, q, lds);
        Stats<V, MIXED> st;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            st.mean[e] = s[0][e] * inv;
            s[0][e] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            x[i].repack();
            const int nv = q.ty + i * p.TY < S ? k.nv : 0;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = e < nv ? x[i].get(e) - st.m(e) : 0.0f;
                s[0][MIXED ? e : 0] = fmaf(d, d, s[0][MIXED ? e : 0]);
            }
        }
        group_sum<float, 1, V, MIXED>(s, a, q, lds);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            st.rstd[e] = rstd_of(s[0][e] * inv, a.eps);
            if (q.ty == 0 && e < q.nv && (q.col + e) % a.D == 0) {
                const int64_t ng = n * a.G + (q.col + e) / a.D;
                a.mean[ng] = st.mean[e];
                a.rstd[ng] = st.rstd[e];
            }
        }
        // (the asm keeps the stores' rows and addresses from being formed, and held
        // in registers, before the sums)
        int row = q.ty;
        asm volatile("" : "+v"(row));
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = row + i * p.TY;
            x[i].repack();
            if (r < S && k.nv > 0)
                apply_forward<V, RAT, MIXED>(x[i], st, k, a.act).store(at(a.y, (n * a.S + r) * a.C + k.col), k.nv);
        }
    }
}

// Split, first pass: sums of x and x^2 of a row chunk of a column block.  A
// lane sums the differences from its first row (and their squares) in fp32,
// column by column, over at most 32 rows, and turns them into fp64 sums of x
// and x^2 about zero at the end: three fp32 operations an element, with the
// digits of a mean far from zero kept out of them.  8 x 4,096 x 320, bf16: 12.9 us
// for 21 MB, 1 x 65,536 x 128, fp32: 11.3 us for 34 MB: ramp and latency, a
// workgroup or four a CU with 4 to 32 rows a lane.
template <int V, bool MIXED>
__global__ __launch_bounds__(1024) void grkan_norm_sums_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int E = MIXED ? V : 1;
    const NormPlan &p = a.p;
    const int64_t total = a.N * p.chunks * p.ncb;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int cb = (int)(b % p.ncb);
        const int64_t nc = b / p.ncb, n = nc / p.chunks, c = nc % p.chunks;
        const Place q(a, cb);
        const int64_t r0 = c * p.chunk_rows + q.ty, r1 = min(a.S, (c + 1) * p.chunk_rows);
        double s[2][E] = {};
        if (q.nv > 0 && r0 < r1) {
            const char *src = at(a.x, n * a.xs + q.col);
            const Pack<V> first = Pack<V>::load(src + r0 * a.xr * ES, q.nv);
            float s1[V] = {}, s2[V] = {};
#pragma unroll 4
            for (int64_t r = r0 + p.TY; r < r1; r += p.TY) {
                const Pack<V> x = Pack<V>::load(src + r * a.xr * ES, q.nv);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = x.get(e) - first.get(e);
                    s1[e] += d;
                    s2[e] = fmaf(d, d, s2[e]);
                }
            }
            const double m = (double)((r1 - r0 + p.TY - 1) / p.TY);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const double f = (double)first.get(e), d = (double)s1[e];
                s[0][MIXED ? e : 0] += fma(m, f, d);
                s[1][MIXED ? e : 0] += fma(f, fma(m, f, 2.0 * d), (double)s2[e]);
            }
        }
        group_sum<double, 2, V, MIXED>(s, a, q, lds);
        store_parts<E>(a, q, n, c, cb, lds);
    }
}

// Split, many parts: a workgroup per (sample, group) adds them (4.1 us for 32
// groups of 1,024 parts; latency).
__global__ __launch_bounds__(256) void grkan_norm_stats_kernel(NormArgs a) {
    for (int64_t ng = blockIdx.x; ng < a.N * a.G; ng += gridDim.x) {
        double s0, s1;
        add_parts(a, ng, s0, s1);
        if (threadIdx.x == 0) {
            const float2 st = of_sums(a, s0, s1);
            a.mean[ng] = st.x;
            a.rstd[ng] = st.y;
        }
    }
}

// Split, second pass: y over a row chunk of a column block, x most likely from
// the Infinity Cache.  8 x 4,096 x 320, bf16, silu: 17.5 us; 1 x 65,536 x 128,
// fp32: 13.4 us for 67 MB, 5.0 TB/s.  Reading four rows ahead moved the one by
// +2% and the other by -5%.
template <int V, bool RAT, bool MIXED>
__global__ __launch_bounds__(1024) void grkan_norm_apply_fwd_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    float2 *stats = reinterpret_cast<float2 *>(lds);
    constexpr int B = 4;  // rows on their way at a time
    const NormPlan &p = a.p;
    const int64_t total = a.N * p.chunks * p.ncb;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int cb = (int)(b % p.ncb);
        const int64_t nc = b / p.ncb, n = nc / p.chunks, c = nc % p.chunks;
        const Place q(a, cb);
        // the first rows are on their way while the statistics are formed
        const int64_t r0 = c * p.chunk_rows + q.ty, r1 = min(a.S, (c + 1) * p.chunk_rows);
        Pack<V> next[B];
        auto fetch = [&](int64_t r) {
#pragma unroll
            for (int i = 0; i < B; ++i) {
                const int64_t row = r + i * p.TY;
                next[i] = Pack<V>::load(at(a.x, n * a.xs + (row < r1 ? row : 0) * a.xr + q.col), row < r1 ? q.nv : 0);
            }
        };
        fetch(r0);
        if (p.fused) own_parts(a, q, n, stats);
        Cols<V, RAT> k;
        k.init(a, q.col, q.nv);
        Stats<V, MIXED> st;
#pragma unroll
        for (int e = 0; e < Stats<V, MIXED>::N; ++e) {
            const int j = q.group(a, e);
            const int64_t ng = n * a.G + q.g0 + j;
            st.mean[e] = p.fused ? stats[j].x : a.mean[ng];
            st.rstd[e] = p.fused ? stats[j].y : a.rstd[ng];
        }
        if (p.fused && c == 0)  // the first chunk's workgroups store the statistics of groups that begin in them
            for (int j = (int)threadIdx.x; j < q.ngroups; j += p.block)
                if ((q.g0 + j) * a.D >= q.c0) {
                    a.mean[n * a.G + q.g0 + j] = stats[j].x;
                    a.rstd[n * a.G + q.g0 + j] = stats[j].y;
                }
        for (int64_t r = r0; r < r1; r += B * p.TY) {
            Pack<V> x[B];
#pragma unroll
            for (int i = 0; i < B; ++i) x[i] = next[i];
            fetch(r + B * p.TY);
#pragma unroll
            for (int i = 0; i < B; ++i)
                if (r + i * p.TY < r1 && k.nv > 0)
                    apply_forward<V, RAT, MIXED>(x[i], st, k, a.act)
                        .store(at(a.y, (n * a.S + r + i * p.TY) * a.C + k.col), k.nv);
        }
        __syncthreads();  // the statistics in LDS have been read
    }
}

template <int V, int RAT, int K> hipError_t launch_token_k(const NormArgs &a, hipStream_t s) {
    if constexpr (RAT == 2 && K * V < 4) {  // the plan straddles with runs of 4 or more only
        return hipErrorInvalidValue;
    } else {
        return start<&grkan_norm_token_fwd_kernel<V, RAT, K>>(a, dim3((unsigned)a.p.blocks), dim3((unsigned)a.p.block), 0,
                                                              s);
    }
}

template <int V, int RAT> hipError_t launch_token(const NormArgs &a, hipStream_t s) {
    switch (a.p.K) {
        case 1: return launch_token_k<V, RAT, 1>(a, s);
        case 2: return launch_token_k<V, RAT, 2>(a, s);
        case 3: return launch_token_k<V, RAT, 3>(a, s);
        default: return launch_token_k<V, RAT, 4>(a, s);
    }
}

template <int V, bool RAT, bool MIXED>
hipError_t launch_blocks(const NormArgs &a, hipStream_t s) {
    const NormPlan &p = a.p;
    const dim3 grid((unsigned)(p.blocks < kMaxBlocks ? p.blocks : kMaxBlocks)), block((unsigned)p.block);
    if (p.kind == kNormSlab) {
        if (p.regs <= 4) return start<&grkan_norm_slab_fwd_kernel<V, RAT, MIXED, 4>>(a, grid, block, p.lds, s);
        if (p.regs <= 8) return start<&grkan_norm_slab_fwd_kernel<V, RAT, MIXED, 8>>(a, grid, block, p.lds, s);
        return start<&grkan_norm_slab_fwd_kernel<V, RAT, MIXED, 16>>(a, grid, block, p.lds, s);
    }
    hipError_t e = start<&grkan_norm_sums_kernel<V, MIXED>>(a, grid, block, p.lds, s);
    if (e == hipSuccess && !p.fused)
        e = start<&grkan_norm_stats_kernel>(a, dim3(group_blocks(a)), dim3(256), 0, s);
    if (e != hipSuccess) return e;
    return start<&grkan_norm_apply_fwd_kernel<V, RAT, MIXED>>(a, grid, block, p.groups * sizeof(float2), s);
}

#else
// ============================================================ backward

// Adds NVAL sums of a lane over `depth` lanes `width` apart (row lanes, or a
// token plan's slots of one group) and writes the first n of them to row
// `prow` of the partials, value i of lane x < width at its at + i * pitch.  All
// threads share the additions.  `lds` holds block * (NVAL + 3) floats.
template <int NVAL>
__device__ static inline void store_sums(const NormArgs &a, const float (&v)[NVAL], int width, int depth, int64_t prow,
                                         int64_t at, int n, int64_t pitch, float *lds) {
    const int t = (int)threadIdx.x, block = a.p.block;
    int *where = reinterpret_cast<int *>(lds + NVAL * block);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NVAL; ++i) lds[i * block + t] = v[i];
    where[t] = n;
    where[block + t] = (int)(uint32_t)at;
    where[2 * block + t] = (int)(uint32_t)((uint64_t)at >> 32);
    __syncthreads();
    float *out = a.partials + prow * a.p.row;
    for (int u = t; u < NVAL * width; u += block) {
        const int i = u / width, x = u - i * width;
        if (i >= where[x]) continue;
        float s = 0.0f;
        for (int q = 0; q < depth; ++q) s += lds[i * block + x + q * width];
        const int64_t o = (int64_t)((uint64_t)(uint32_t)where[block + x] | (uint64_t)(uint32_t)where[2 * block + x] << 32);
        out[o + i * pitch] = s;
    }
}

template <int V, bool RAT>
__device__ static inline void store_col_sums(const NormArgs &a, const ColSums<V, RAT> &cs, const Place &q, int cb,
                                             int64_t prow, char *ldsb) {
    float *lds = reinterpret_cast<float *>(ldsb);
    const NormPlan &p = a.p;
    store_sums<V>(a, cs.dw, p.TX, p.TY, prow, q.col, q.nv, 1, lds);
    store_sums<V>(a, cs.db, p.TX, p.TY, prow, a.C + (int64_t)q.col, q.nv, 1, lds);
    if constexpr (RAT)
        store_sums<10>(a, cs.coef, p.TX, p.TY, prow, 2 * (int64_t)a.C + (int64_t)cb * p.TX + q.tx, q.nv > 0 ? 10 : 0,
                       p.cv, lds);
}

// Token backward: dh and xh of a lane's run in registers, two sums over the
// group, dx; column and coefficient sums stay in registers over all the
// samples a workgroup walks over.  201,728 x 768, bf16, the rational: 306 us a
// call in a long series, 10 of them the columns', 3.1 TB/s (ten calls from idle,
// traced: 322 us the fastest, 379 the median); its 64 instructions an element keep
// the vector units busy 0.94 of the time, which bounds it.
// The second bound keeps two or three waves on a SIMD: left alone, the compiler
// evaluates all of a lane's elements side by side, in 270 registers for 12.  (The
// 20 bytes of scratch at K V = 12 are two values put away before the walk and
// taken back after it; the walk itself touches none.)
template <int V, int RAT, int K>
__global__ __launch_bounds__(K * V == 1 ? 1024 : 256, K * V == 1 ? 1 : (RAT == 2 || K * V > 12 ? 2 : 3)) void
grkan_norm_token_bwd_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char ldsb[];
    float *lds = reinterpret_cast<float *>(ldsb);
    constexpr int kSets = RAT == 2 ? 2 : 1;
    const NormPlan &p = a.p;
    const int t = (int)threadIdx.x, l = t & (p.T - 1), sl = t / p.T;
    const int64_t slot = (int64_t)blockIdx.x * p.spw + sl;
    const int g = (int)(slot % a.G);
    const int64_t step = p.blocks * p.spw / a.G;
    const float inv = 1.0f / (float)a.D;
    int phase = 0;
    TokenCols<V, RAT, K, RAT != 0> k;
    k.init(a, g, l);
    SlopeCoefs sc;
    if constexpr (RAT == 1) sc.init(k.c[0]);
    float dw[K][V] = {}, db[K][V] = {}, coef[kSets][RAT ? 10 : 1] = {};
    int64_t n = slot / a.G;
    Pack<V> nx[K], ndy[K];
    float nmean = 0.0f, nrstd = 0.0f;
    auto fetch = [&](int64_t m, bool any) {
        nmean = any ? a.mean[m * a.G + g] : 0.0f;
        nrstd = any ? a.rstd[m * a.G + g] : 0.0f;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            nx[i] = Pack<V>::load(at(a.x, m * a.xs + k.col[i]), any ? k.nv[i] : 0);
            ndy[i] = Pack<V>::load(at(a.dy, m * a.ds + k.col[i]), any ? k.nv[i] : 0);
        }
    };
    fetch(n < a.N ? n : 0, n < a.N);
    for (; n < a.N; n += step) {
        const float mean = nmean, rstd = nrstd;
        Pack<V> x[K], dy[K];
#pragma unroll
        for (int i = 0; i < K; ++i) x[i] = nx[i], dy[i] = ndy[i];
        fetch(n + step < a.N ? n + step : n, true);
        float m[2] = {0.0f, 0.0f};
        float tt[K][V], xh[K][V];
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                // absent elements: dy = 0, and xh = 0 in place of -mean rstd
                xh[i][e] = e < k.nv[i] ? (x[i].get(e) - mean) * rstd : 0.0f;
                float h = fmaf(xh[i][e], k.w[i][e], k.b[i][e]), dh;
                const float gr = dy[i].get(e);
                if constexpr (RAT == 0) {
                    dh = gr * act_slope(h, a.act);
                } else if constexpr (RAT == 1) {
                    dh = rational_slope(h, gr, sc, *reinterpret_cast<float (*)[10]>(coef[0]));
                } else {
                    const int j = i * V + e;
                    // (one element after another, as in rational_slope)
                    asm volatile("" : "+v"(h) : "v"(coef[0][0]), "v"(coef[0][1]), "v"(coef[0][2]), "v"(coef[0][3]),
                                 "v"(coef[0][4]), "v"(coef[0][5]), "v"(coef[0][6]), "v"(coef[0][7]), "v"(coef[0][8]),
                                 "v"(coef[0][9]), "v"(coef[1][0]), "v"(coef[1][1]), "v"(coef[1][2]), "v"(coef[1][3]),
                                 "v"(coef[1][4]), "v"(coef[1][5]), "v"(coef[1][6]), "v"(coef[1][7]), "v"(coef[1][8]),
                                 "v"(coef[1][9]));
                    sc.init(k.coefs(j));
                    float term[10] = {};
                    dh = rational_slope(h, gr, sc, term);
#pragma unroll
                    for (int q = 0; q < 10; ++q) {
                        coef[0][q] += j < k.split ? term[q] : 0.0f;
                        coef[1][q] += j < k.split ? 0.0f : term[q];
                    }
                }
                db[i][e] += dh;
                dw[i][e] = fmaf(dh, xh[i][e], dw[i][e]);
                tt[i][e] = dh * k.w[i][e];
                m[0] += tt[i][e];
                m[1] = fmaf(tt[i][e], xh[i][e], m[1]);
            }
        slot_sum<2>(m, p.T, lds, phase);
        const float m1 = m[0] * inv, m2 = m[1] * inv;
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (k.nv[i] > 0) {
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] = rstd * (tt[i][e] - fmaf(xh[i][e], m2, m1));
                Pack<V>::from(f).store(at(a.y, n * a.C + k.col[i]), k.nv[i]);
            }
    }
    // slots of one group in this workgroup: spw / G of them, G slots apart
    // (slot = workgroup * spw + sl, spw a multiple of G), or each its own;
    // either way the workgroup's sums lie in one row of the partials
    const bool shared = p.spw > a.G;
    const int width = shared ? a.G * p.T : p.spw * p.T, depth = shared ? p.spw / a.G : 1;
    const int64_t prow = shared ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * p.spw / a.G;
    const int64_t coefs0 = 2 * (int64_t)a.C;
#pragma unroll
    for (int i = 0; i < K; ++i) {
        store_sums<V>(a, dw[i], width, depth, prow, k.col[i], k.nv[i], 1, lds);
        store_sums<V>(a, db[i], width, depth, prow, a.C + k.col[i], k.nv[i], 1, lds);
    }
    if constexpr (RAT != 0) {
#pragma unroll
        for (int q = 0; q < kSets; ++q)
            store_sums<10>(a, coef[q], width, depth, prow, coefs0 + 10 * q * p.cv + (int64_t)g * p.vpg + l,
                           k.nv[0] > 0 ? 10 : 0, p.cv, lds);
    }
}

// Slab backward: x, dy and dh of a sample's groups in registers, so that x and
// dy are read once.  128 x 197 x 192 in 8 groups, fp32, gelu: 23.6 us for 58 MB (2.5
// TB/s; two samples a workgroup, the loads and the sums of the first exposed);
// 1,024 samples: 132 us, 3.5 TB/s.
template <int V, bool RAT, bool MIXED, int R>
__global__ __launch_bounds__(512) void grkan_norm_slab_bwd_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int E = MIXED ? V : 1;
    const NormPlan &p = a.p;
    const float inv = 1.0f / ((float)a.D * (float)a.S);
    int64_t n0;
    int cb;
    sample_block(blockIdx.x, p.ncb, p.chunks, n0, cb);
    if (n0 >= p.chunks) return;  // the whole workgroup
    const Place q(a, cb);
    Cols<V, RAT> k;
    k.init(a, q.col, q.nv);
    SlopeCoefs sc;
    if constexpr (RAT) sc.init(k.c);
    ColSums<V, RAT> cs;
    cs.clear();
    const int S = (int)a.S;
    // A sample's values; AHEAD: while one is worked on, the next one's are on
    // their way.
    constexpr bool AHEAD = R * V <= 24;
    Pack<V> nx[R], ndy[R];
    Stats<V, MIXED> nst;
    auto fetch = [&](int64_t n, Pack<V>(&x)[R], Pack<V>(&dy)[R], Stats<V, MIXED> &st) {
        const bool any = n < a.N;
        const int64_t m = any ? n : 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = q.ty + i * p.TY;
            const int nv = any && r < S ? k.nv : 0;
            const int64_t rr = r < S ? r : 0;
            x[i] = Pack<V>::load(at(a.x, m * a.xs + rr * a.xr + k.col), nv);
            dy[i] = Pack<V>::load(at(a.dy, m * a.ds + rr * a.dr + k.col), nv);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int64_t ng = m * a.G + q.g0 + q.group(a, e);
            st.mean[e] = a.mean[ng];
            st.rstd[e] = a.rstd[ng];
        }
    };
    if constexpr (AHEAD) fetch(n0, nx, ndy, nst);
    for (int64_t n = n0; n < a.N; n += p.chunks) {
        Pack<V> x[R], dy[R];
        Stats<V, MIXED> st;
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                x[i] = nx[i];
                dy[i] = ndy[i];
            }
            st = nst;
            fetch(n + p.chunks, nx, ndy, nst);
        } else {
            fetch(n, x, dy, st);
        }
        float dh[R][V], sdh[V] = {}, sdx[V] = {};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (q.ty + i * p.TY < S) {  // rows past the end add nothing
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = e < k.nv ? (x[i].get(e) - st.m(e)) * st.r(e) : 0.0f;
                    dh[i][e] = slope<V, RAT>(xh, dy[i].get(e), k, sc, e, a.act, cs.coef);
                    sdh[e] += dh[i][e];
                    sdx[e] = fmaf(dh[i][e], xh, sdx[e]);
                }
            }
        }
        float m[2][E] = {};
#pragma unroll
        for (int e = 0; e < V; ++e) {
            cs.db[e] += sdh[e];
            cs.dw[e] += sdx[e];
            m[0][MIXED ? e : 0] = fmaf(sdh[e], k.w[e], m[0][MIXED ? e : 0]);
            m[1][MIXED ? e : 0] = fmaf(sdx[e], k.w[e], m[1][MIXED ? e : 0]);
        }
        group_sum<float, 2, V, MIXED>(m, a, q, lds);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = q.ty + i * p.TY;
            x[i].repack();
            if (r < S && k.nv > 0) {
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = (x[i].get(e) - st.m(e)) * st.r(e);
                    f[e] = st.r(e) * (dh[i][e] * k.w[e] - fmaf(xh, m[1][MIXED ? e : 0] * inv, m[0][MIXED ? e : 0] * inv));
                }
                Pack<V>::from(f).store(at(a.y, (n * a.S + r) * a.C + k.col), k.nv);
            }
        }
    }
    store_col_sums<V, RAT>(a, cs, q, cb, n0, lds);
}

// Split, first pass: sums of t and t xh and the column sums of a row chunk (one
// read of x and dy; for groups too long for registers).
template <int V, bool RAT, bool MIXED>
__global__ __launch_bounds__(512) void grkan_norm_sums_bwd_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int E = MIXED ? V : 1;
    const NormPlan &p = a.p;
    const int64_t total = a.N * p.chunks * p.ncb;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int cb = (int)(b % p.ncb);
        const int64_t nc = b / p.ncb, n = nc / p.chunks, c = nc % p.chunks;
        const Place q(a, cb);
        Cols<V, RAT> k;
        k.init(a, q.col, q.nv);
        SlopeCoefs sc;
        if constexpr (RAT) sc.init(k.c);
        ColSums<V, RAT> cs;
        cs.clear();
        const int64_t r1 = min(a.S, (c + 1) * p.chunk_rows);
        if (q.nv > 0) {
            Stats<V, MIXED> st;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int64_t ng = n * a.G + q.g0 + q.group(a, e);
                st.mean[e] = a.mean[ng];
                st.rstd[e] = a.rstd[ng];
            }
#pragma unroll RAT ? 1 : 2
            for (int64_t r = c * p.chunk_rows + q.ty; r < r1; r += p.TY) {
                const Pack<V> x = Pack<V>::load(at(a.x, n * a.xs + r * a.xr + k.col), k.nv);
                const Pack<V> dy = Pack<V>::load(at(a.dy, n * a.ds + r * a.dr + k.col), k.nv);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = e < k.nv ? (x.get(e) - st.m(e)) * st.r(e) : 0.0f;
                    const float dh = slope<V, RAT>(xh, dy.get(e), k, sc, e, a.act, cs.coef);
                    cs.db[e] += dh;
                    cs.dw[e] = fmaf(dh, xh, cs.dw[e]);
                }
            }
        }
        double s[2][E] = {};
#pragma unroll
        for (int e = 0; e < V; ++e) {
            s[0][MIXED ? e : 0] += (double)cs.db[e] * (double)k.w[e];
            s[1][MIXED ? e : 0] += (double)cs.dw[e] * (double)k.w[e];
        }
        group_sum<double, 2, V, MIXED>(s, a, q, lds);
        store_parts<E>(a, q, n, c, cb, lds);
        store_col_sums<V, RAT>(a, cs, q, cb, n * p.chunks + c, lds);
        __syncthreads();
    }
}

// Split, many parts: <t> and <t xh>, a workgroup per (sample, group).
__global__ __launch_bounds__(256) void grkan_norm_means_kernel(NormArgs a) {
    for (int64_t ng = blockIdx.x; ng < a.N * a.G; ng += gridDim.x) {
        double s0, s1;
        add_parts(a, ng, s0, s1);
        if (threadIdx.x == 0) reinterpret_cast<float2 *>(a.means)[ng] = of_sums(a, s0, s1);
    }
}

// Split, second pass: dx over a row chunk.  The slope is formed again: keeping
// it would cost a write and a read of a tensor.
template <int V, bool RAT, bool MIXED>
__global__ __launch_bounds__(512) void grkan_norm_apply_bwd_kernel(NormArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    float2 *means = reinterpret_cast<float2 *>(lds);
    const NormPlan &p = a.p;
    const int64_t total = a.N * p.chunks * p.ncb;
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        const int cb = (int)(b % p.ncb);
        const int64_t nc = b / p.ncb, n = nc / p.chunks, c = nc % p.chunks;
        const Place q(a, cb);
        if (p.fused) own_parts(a, q, n, means);
        Cols<V, RAT> k;
        k.init(a, q.col, q.nv);
        SlopeCoefs sc;
        if constexpr (RAT) sc.init(k.c);
        Stats<V, MIXED> st, mm;  // mm: <t> and <t xh>
#pragma unroll
        for (int e = 0; e < Stats<V, MIXED>::N; ++e) {
            const int j = q.group(a, e);
            const int64_t ng = n * a.G + q.g0 + j;
            const float2 m = p.fused ? means[j] : reinterpret_cast<const float2 *>(a.means)[ng];
            st.mean[e] = a.mean[ng];
            st.rstd[e] = a.rstd[ng];
            mm.mean[e] = m.x;
            mm.rstd[e] = m.y;
        }
        const int64_t r1 = min(a.S, (c + 1) * p.chunk_rows);
        float unused[10] = {};
        if (q.nv > 0) {
#pragma unroll RAT ? 1 : 2
            for (int64_t r = c * p.chunk_rows + q.ty; r < r1; r += p.TY) {
                const Pack<V> x = Pack<V>::load(at(a.x, n * a.xs + r * a.xr + k.col), k.nv);
                const Pack<V> dy = Pack<V>::load(at(a.dy, n * a.ds + r * a.dr + k.col), k.nv);
                float f[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float xh = (x.get(e) - st.m(e)) * st.r(e);
                    const float dh = slope<V, RAT>(xh, dy.get(e), k, sc, e, a.act, unused);
                    f[e] = st.r(e) * (dh * k.w[e] - fmaf(xh, mm.r(e), mm.m(e)));
                }
                Pack<V>::from(f).store(at(a.y, (n * a.S + r) * a.C + k.col), k.nv);
            }
        }
        __syncthreads();  // the means in LDS have been read
    }
}

// The column partials added over their rows in fp64: workgroups of 64 columns
// x 16 row lanes for dw and db, then one workgroup per (activation group,
// coefficient), whose accesses are a contiguous range.  3.9 us for 64 rows of 384
// columns, 10.5 us for 1,009 rows of 1,536 and 8 x 10 coefficients: latency.
template <bool RAT>
__device__ static inline void add_columns(const NormArgs &a, int64_t b, double *red) {
    const int t = (int)threadIdx.x;
    const NormPlan &p = a.p;
    const int64_t row = p.row, P = p.prows;
    const int64_t colblocks = (2 * (int64_t)a.C + 63) / 64;
    if (b < colblocks) {
        const int64_t c = b * 64 + (t & 63);
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
        const int64_t gk = b - colblocks;
        const int g = (int)(gk / 10), k = (int)(gk % 10);
        // The lanes whose first column lies in this group, counted over a row
        // (token: runs of K V columns from each norm group on; else accesses
        // from each block's first column on); where runs straddle groups also
        // the second sums of the lanes of the group before.
        const bool token = p.kind == kNormToken;
        const int per = token ? a.D : p.width, lanes = token ? p.vpg : p.TX, len = token ? p.K * p.vec : p.vec;
        auto lane = [&](int64_t c) { return c / per * lanes + (c % per + len - 1) / len; };
        double s = 0.0;
        for (int set = 0; set <= (p.straddle ? 1 : 0); ++set) {
            const int64_t g0 = (int64_t)g - set;
            if (g0 < 0) continue;
            const int64_t v0 = lane(g0 * a.dga), w = lane((g0 + 1) * a.dga) - v0;
            const float *src = a.partials + 2 * (int64_t)a.C + (10 * set + k) * p.cv + v0;
#pragma unroll 8
            for (int64_t i = t; i < P * w; i += 1024) {
                const int64_t r = i / w;
                s += (double)src[r * row + (i - r * w)];
            }
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

template <bool RAT>
__global__ __launch_bounds__(1024) void grkan_norm_columns_kernel(NormArgs a, int64_t total) {
    __shared__ double red[1024];
    for (int64_t b = blockIdx.x; b < total; b += gridDim.x) {
        add_columns<RAT>(a, b, red);
        __syncthreads();  // the sums in LDS have been read
    }
}

template <bool RAT> hipError_t launch_columns(const NormArgs &a, hipStream_t s) {
    if (!a.dw && !a.db && !RAT) return hipSuccess;
    const int64_t total = (2 * (int64_t)a.C + 63) / 64 + (RAT ? (int64_t)a.ng * 10 : 0);
    hipLaunchKernelGGL(grkan_norm_columns_kernel<RAT>, dim3((unsigned)(total < kMaxBlocks ? total : kMaxBlocks)), dim3(1024),
                       0, s, a, total);
    return hipGetLastError();
}

template <int V, int RAT, int K> hipError_t launch_token_k(const NormArgs &a, hipStream_t s) {
    // the plan gives a lane 16 elements at most, and straddles with runs of 4 or more only
    if constexpr ((K > 1 && K * V > 16) || (RAT == 2 && K * V < 4)) {
        return hipErrorInvalidValue;
    } else {
        const hipError_t e = start<&grkan_norm_token_bwd_kernel<V, RAT, K>>(a, dim3((unsigned)a.p.blocks),
                                                                            dim3((unsigned)a.p.block), a.p.lds, s);
        return e != hipSuccess ? e : launch_columns<RAT != 0>(a, s);
    }
}

template <int V, int RAT> hipError_t launch_token(const NormArgs &a, hipStream_t s) {
    switch (a.p.K) {
        case 1: return launch_token_k<V, RAT, 1>(a, s);
        case 2: return launch_token_k<V, RAT, 2>(a, s);
        case 3: return launch_token_k<V, RAT, 3>(a, s);
        default: return launch_token_k<V, RAT, 4>(a, s);
    }
}

template <int V, bool RAT, bool MIXED>
hipError_t launch_blocks(const NormArgs &a, hipStream_t s) {
    const NormPlan &p = a.p;
    const dim3 grid((unsigned)(p.blocks < kMaxBlocks ? p.blocks : kMaxBlocks)), block((unsigned)p.block);
    hipError_t e;
    if (p.kind == kNormSlab) {
        if (p.regs <= 3)
            e = start<&grkan_norm_slab_bwd_kernel<V, RAT, MIXED, 3>>(a, dim3((unsigned)p.blocks), block, p.lds, s);
        else if (p.regs <= 5)
            e = start<&grkan_norm_slab_bwd_kernel<V, RAT, MIXED, 5>>(a, dim3((unsigned)p.blocks), block, p.lds, s);
        else
            e = start<&grkan_norm_slab_bwd_kernel<V, RAT, MIXED, 8>>(a, dim3((unsigned)p.blocks), block, p.lds, s);
    } else {
        e = start<&grkan_norm_sums_bwd_kernel<V, RAT, MIXED>>(a, grid, block, p.lds, s);
        if (e == hipSuccess && !p.fused)
            e = start<&grkan_norm_means_kernel>(a, dim3(group_blocks(a)), dim3(256), 0, s);
        if (e == hipSuccess)
            e = start<&grkan_norm_apply_bwd_kernel<V, RAT, MIXED>>(a, grid, block, p.groups * sizeof(float2), s);
    }
    return e != hipSuccess ? e : launch_columns<RAT>(a, s);
}
#endif

template <int V, bool RAT> hipError_t launch_vec(const NormArgs &a, hipStream_t s) {
    if (a.p.kind == kNormToken) {
        if constexpr (RAT) return a.p.straddle ? launch_token<V, 2>(a, s) : launch_token<V, 1>(a, s);
        return launch_token<V, 0>(a, s);
    }
    if constexpr (V > 1) {
        if (a.p.mixed) return launch_blocks<V, RAT, true>(a, s);
    }
    return launch_blocks<V, RAT, false>(a, s);
}

}  // namespace

#if GRKAN_NORM_BACKWARD
template <> hipError_t launch_norm_backward<NormIo>(const NormArgs &a, hipStream_t s) {
#else
template <> hipError_t launch_norm_forward<NormIo>(const NormArgs &a, hipStream_t s) {
#endif
    const bool rational = a.act == GRKAN_ACT_RATIONAL;
    if (!rational) {
        if (a.p.vec == kMaxV) return launch_vec<kMaxV, false>(a, s);
        if (a.p.vec == kMaxV / 2 && a.p.kind == kNormToken) return launch_token<kMaxV / 2, 0>(a, s);
        return hipErrorInvalidValue;
    }
    switch (a.p.vec) {
        case 8:
            if constexpr (kMaxV >= 8) return launch_vec<8, true>(a, s);
            return hipErrorInvalidValue;
        case 4: return launch_vec<4, true>(a, s);
        case 2: return launch_vec<2, true>(a, s);
        case 1: return launch_vec<1, true>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace grkan
