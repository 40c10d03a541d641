// grkan_linear.hip -- the linear map z = act(x W^T + b) + r and its gradients
// on the matrix cores (gfx950): bf16 operands, fp32 sums.
//
// Compiled twice: GRKAN_LINEAR_ALIGNED 1 (every 16-byte chunk of the operands
// aligned and whole) and 0 (any widths, strides and alignment).
//
// Bound: many rows, the matrix cores; few rows, the bytes of W.
//
// The tile kernel.  A workgroup of 4 waves (2 x 2; 8 waves, 2 x 4, for the
// 256 x 256 tile) forms a BM x BN tile of the result; a wave a part of it in
// 32 x 32 blocks of v_mfma_f32_32x32x16_bf16.  The instruction's row operand is
// P (columns of the result) and its column operand Q (rows of the result), so a
// lane's accumulators run along n within one row of the result, and exchanging
// them with the lane 32 away leaves 8 consecutive columns in a lane, which take
// bias, activation and residual together and leave through LDS as whole rows.
// k advances BK at a time through two or three LDS stages.  While step t is
// multiplied, the chunks of the step after (or two after) travel from memory
// straight into LDS (no registers); one barrier a step, before the step's last
// group of matrix instructions, whose fragments are already in registers,
// covers both the arrival of step t + 1 and the release of step t's stage.  The
// launch has as many workgroups as the CUs hold at once (one of 8 waves, three
// of 4); each walks over its tiles, and the fetches run on into the next tile
// while a result leaves.
//
// Measured on MI355X, products alone: 1,180-1,240 TFLOP/s at 8,192 x 8,192 from
// 8,192 (the library's 1,358), 286-324 us at 50,432 x 3,072 from 768 and 280 us at
// 50,432 x 768 from 3,072 (238 GFLOP; the library's 230-300 us).  What bounds them
// is the way into LDS and the power it takes: with every fetch left out the
// same loop ran at 1,700-1,800 TFLOP/s, with all fetches from one place in L2
// as fast as without the change, and more steps in flight, wave priorities and
// fixed orders of reads and products changed 0-3%.  So the largest tile counts, since it
// fetches least: 256 x 256 in 8 waves and two stages of 64 against 256 x 128
// in 4 waves, two workgroups a CU, three stages of 32 (the products above 1.1 to
// 1.3 times as long) and against three or four stages of 32 (1.05 to 1.1 times).
// 256 x 256 in 4 waves needs 352 registers: 376 TFLOP/s with one wave a SIMD.
//
// LDS layouts.  Chunks are 16 bytes and land in the order of the lanes, so
// bank conflicts are avoided by choosing which chunk a lane fetches:
//   K contiguous   [row][BK]: chunk c of row r sits at c ^ f(r), with f(r) = r mod
//                  8 for BK = 64 and (r / 2) mod 4 for BK = 32, bit 0 flipped in
//                  every other 8 rows: 8 consecutive rows of one chunk column
//                  cover 128 bytes of banks and 16 cover 256
//   K strided      [k][rows]: chunk c of row k sits at c ^ s(k), s = 2 (j + 4 (j
//                  mod 2)), j = k mod 4 (2 j for 64 rows, whose k rows are half
//                  as long); fragments are read with the transposing
//                  ds_read_b64_tr_b16, whose 16 lanes touch rows k..k+3 of 32
//                  bytes: four different 32-byte banks, and the two groups of
//                  16 side by side eight different ones
#include "grkan_linear.h"

#include <type_traits>

#include "grkan_act.h"

namespace grkan {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

constexpr bool kAligned = GRKAN_LINEAR_ALIGNED != 0;

// nv (0..8) elements at p, the rest zeros; p is aligned to an element.
__device__ static inline u32x4 load8(const uint16_t *p, int nv) {
    if (nv >= 8) return *reinterpret_cast<const u32x4_any *>(p);
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < nv) v[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
    return v;
}
__device__ static inline void store8(uint16_t *p, int nv, u32x4 v) {
    if (nv >= 8) {
        *reinterpret_cast<u32x4_any *>(p) = v;
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < nv) p[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
}

// store8 for results larger than the caches: non-temporal, so that they do not
// drive the operands out (50,432 x 3,072 from 768: 355 us with ordinary stores,
// 323 with these).
__device__ static inline void stream8(uint16_t *p, int nv, u32x4 v) {
    if (nv >= 8)
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any *>(p));
    else
        store8(p, nv, v);
}

// ------------------------------------------------------------ epilogue

// RAT: 0 an activation without coefficients, 1 the rational with 8-column
// chunks inside one activation group, 2 the rational with any groups.
template <int RAT> struct ChunkParams {
    float bias[8];
    Coefs<5, 4> c;
    int n, nv;
    __device__ inline void init(const Epilogue &e, int n_, int N) {
        n = n_;
        nv = N - n < 8 ? N - n : 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) bias[i] = e.bias && i < nv ? e.bias[n + i] : 0.0f;
        if constexpr (RAT == 1) c = load_coefs<5, 4>(e.A, e.B, nv > 0 ? n / e.dga : 0);
    }
};

// act(h) of 8 columns, in place.
template <int RAT>
__device__ static inline void activate8(float (&h)[8], const Epilogue &e, const ChunkParams<RAT> &k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (RAT == 2) {
            if (i < k.nv) h[i] = rational<5, 4>(h[i], load_coefs<5, 4>(e.A, e.B, (k.n + i) / e.dga));
        } else {
            h[i] = act_value<RAT == 1>(h[i], e.act, k.c);
        }
    }
}

// 8 sums of row m, columns n.. -> pre, z.
template <int RAT>
__device__ static inline void finish8(float (&h)[8], const Epilogue &e, const ChunkParams<RAT> &k, int64_t m, int N) {
    if (k.nv <= 0) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += k.bias[i];
    const int64_t at = m * N + k.n;
    if (e.pre) store8(static_cast<uint16_t *>(e.pre) + at, k.nv, Io<bf16io>::pack(h));
    activate8<RAT>(h, e, k);
    if (e.residual) {
        float r[8];
        Io<bf16io>::unpack(load8(static_cast<const uint16_t *>(e.residual) + m * e.ldr + k.n, k.nv), r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] += r[i];
    }
    store8(static_cast<uint16_t *>(e.z) + at, k.nv, Io<bf16io>::pack(h));
}

// ------------------------------------------------------------ staging

constexpr uint32_t kNowhere = 0x80000000u;  // past every buffer: reads zeros

// 16 bytes per lane from offset `off` of the buffer to LDS, lane after lane
// from `to` (the same in all lanes; the instruction takes it from M0).  Written
// as an instruction because it has no result: the compiler, which cannot tell
// the stages apart, would wait for every such load before each transposing LDS
// read (the products with a strided operand took 1.5 times as long); arrival is
// waited for by count (wait_loads).  Loads that the compiler does know of only
// wait longer for the ones it does not.  M0 is the compiler's to use nowhere
// else in these kernels.
__device__ static inline void fetch_chunk(u32x4 rsrc, uint32_t off, const char *to) {
    const uint32_t lds = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char *)to);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(rsrc)
                 : "memory");
}

// The swizzles f and s of the LDS layouts above.
template <int BK> __device__ static inline int chunk_of_row(int row) {
    return ((BK == 64 ? row : row >> 1) & (BK / 8 - 1)) ^ ((row >> 3) & 1);
}
template <int ROWS> __device__ static inline int chunk_of_k(int k) {
    return ROWS >= 128 ? 2 * ((k & 3) + 4 * (k & 1)) : 2 * (k & 3);
}

// One operand's tile of ROWS x BK, as this thread's chunks: chunk id i * T +
// thread, at byte 16 id of its stage.
template <int ROWS, int BK, bool STRIDED, int T> struct Stager {
    static constexpr int kChunks = ROWS * BK / 8 / T;
    static constexpr int kBytes = ROWS * BK * 2;
    static constexpr int kPerRow = STRIDED ? ROWS / 8 : BK / 8;  // chunks per LDS row
    static_assert(ROWS * BK / 8 % T == 0 && T % kPerRow == 0, "whole chunks");

    const char *base;    // first row of the tile at its first k
    int64_t step;        // bytes from one k step to the next
    int64_t ld;
    uint32_t off[kChunks];   // byte offset of the chunk from base, or kNowhere
    int k0;              // K contiguous: k of the chunks; strided: k of chunk 0
    int valid;           // strided: elements of a chunk inside the operand's own range
    bool inside;         // the tile lies inside the operand: unaligned chunks of a whole step need no checks
    u32x4 r[2][kAligned ? 1 : kChunks];  // unaligned: chunks on their way, of two steps

    __device__ inline void init(const Operand &o, int row0, int rows, int kstart) {
        const int t = (int)threadIdx.x;
        ld = o.ld;
        const int slot = t % kPerRow, r0 = t / kPerRow;
        if constexpr (STRIDED) {
            base = static_cast<const char *>(o.p) + ((int64_t)kstart * ld + row0) * 2;
            step = (int64_t)BK * ld * 2;
            k0 = r0;
            // the rows of a thread's chunks are a multiple of 4 apart, so chunk_of_k is one value
            static_assert(T / kPerRow % 4 == 0, "one swizzle per thread");
            const int c = slot ^ chunk_of_k<ROWS>(r0);
            valid = min(max(rows - row0 - c * 8, 0), 8);
            inside = row0 + ROWS <= rows;
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                off[i] = valid > 0 ? (uint32_t)((r0 + i * (T / kPerRow)) * ld * 2 + c * 16) : kNowhere;
        } else {
            base = static_cast<const char *>(o.p) + ((int64_t)row0 * ld + kstart) * 2;
            step = BK * 2;
            static_assert(T / kPerRow % 16 == 0, "one swizzle per thread");
            const int c = slot ^ chunk_of_row<BK>(r0);
            k0 = c * 8;
            valid = 8;
            inside = true;
            // rows past the end: zeros, or (unaligned) the last row once more; what
            // they form is not stored
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                int row = r0 + i * (T / kPerRow);
                if (!kAligned) row = min(row, rows - 1 - row0);
                off[i] = row0 + row < rows ? (uint32_t)(row * ld * 2 + c * 16) : kNowhere;
            }
        }
    }

    // Chunks of step t, `left` values of k before its end: aligned into the stage
    // at LDS byte offset `stage`, else into register set SET; past the end zeros.
    template <int SET> __device__ inline void fetch(char *lds, int stage, int t, int left) {
        const char *src = base + t * step;
        if constexpr (kAligned) {
            const uint64_t addr = reinterpret_cast<uint64_t>(src);
            const u32x4 rsrc = {(uint32_t)__builtin_amdgcn_readfirstlane((int)addr), (uint32_t)__builtin_amdgcn_readfirstlane((int)(addr >> 32)) & 0xffffu,
                                0x7ffffff0u, 0x00020000u};
            const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int k = STRIDED ? k0 + i * (T / kPerRow) : k0;
                fetch_chunk(rsrc, k < left ? off[i] : kNowhere, lds + stage + (i * T + wave * 64) * 16);
            }
        } else if (left >= BK && inside) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i) r[SET][i] = *reinterpret_cast<const u32x4_any *>(src + off[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                const int k = STRIDED ? k0 + i * (T / kPerRow) : k0;
                const int nv = STRIDED ? (k < left ? valid : 0) : min(max(left - k, 0), 8);
                r[SET][i] = load8(reinterpret_cast<const uint16_t *>(src + (nv ? off[i] : 0)), nv);
            }
        }
    }
    // Unaligned: the chunks of a register set into their stage.
    template <int SET> __device__ inline void put(char *lds, int stage) {
        if constexpr (!kAligned) {
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                *reinterpret_cast<u32x4 *>(lds + stage + (i * T + (int)threadIdx.x) * 16) = r[SET][i];
        }
    }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Fragments of NB blocks of 32 rows from row `row0` of the tile, k from 16 ks.
template <int ROWS, int BK, bool STRIDED, int NB> struct Reader {
    int at[STRIDED ? NB : BK / 16];
    __device__ inline void init(int row0) {
        const int lane = (int)threadIdx.x & 63;
        if constexpr (STRIDED) {
            const int k = 8 * (lane >> 5) + ((lane & 15) >> 2);
            const int col = row0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int c = (col + 32 * i) >> 3;
                at[i] = k * ROWS * 2 + ((c ^ chunk_of_k<ROWS>(k)) << 4) + (col & 4) * 2;
            }
        } else {
            const int row = row0 + (lane & 31);
#pragma unroll
            for (int ks = 0; ks < BK / 16; ++ks)
                at[ks] = row * BK * 2 + (((2 * ks + (lane >> 5)) ^ chunk_of_row<BK>(row)) << 4);
        }
    }
    __device__ inline void read(const char *stage, int ks, bf16x8 (&f)[NB]) const {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            if constexpr (STRIDED) {
                typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
                const char *p = stage + at[i] + ks * 16 * ROWS * 2;
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * ROWS * 2));
                f[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            } else {
                f[i] = *reinterpret_cast<const bf16x8 *>(stage + at[ks] + i * 32 * BK * 2);
            }
        }
    }
};

// s_waitcnt vmcnt(n), lgkmcnt(0).
template <int N> __device__ static inline void wait_loads() {
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
}
__device__ static inline void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// ------------------------------------------------------------ tile kernel

template <int BM, int BN, int BK> struct TileShape {
    static constexpr int kWavesN = BN == 256 ? 4 : 2, kThreads = 2 * kWavesN * 64;
    static constexpr int kStages = BN == 256 ? 2 : 3;
    static constexpr int kStage = (BM + BN) * BK * 2;
    static constexpr size_t kLds = kStages * (size_t)kStage + BN * 4 + BN / 8 * 12 * 4;
};

// The epilogue's parameters of a tile's BN columns in LDS: bias, then for each
// 8-column chunk the rational's coefficients (a_0..a_5, b_1..b_4, two unused).
template <int RAT, int BN, int T>
__device__ static inline void load_params(float *params, const Epilogue &e, int n0, int N) {
    const int t = (int)threadIdx.x;
    if (t < BN) params[t] = e.bias && n0 + t < N ? e.bias[n0 + t] : 0.0f;
    if constexpr (RAT == 1) {
        for (int i = t; i < BN / 8 * 12; i += T) {
            const int c = i / 12, k = i - 12 * c, n = n0 + 8 * c, g = n < N ? n / e.dga : 0;
            params[BN + i] = k < 6 ? e.A[g * 6 + k] : (k < 10 ? e.B[g * 4 + k - 6] : 0.0f);
        }
    }
}
template <int BN> __device__ static inline void add_bias(float (&h)[8], const float *params, int chunk) {
    const f32x4 u = *reinterpret_cast<const f32x4 *>(params + 8 * chunk);
    const f32x4 v = *reinterpret_cast<const f32x4 *>(params + 8 * chunk + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] += u[i];
        h[4 + i] += v[i];
    }
}
template <int RAT, int BN>
__device__ static inline void activate_tile(float (&h)[8], const float *params, int chunk, int act) {
    Coefs<5, 4> c;
    if constexpr (RAT == 1) {
        const f32x4 *p = reinterpret_cast<const f32x4 *>(params + BN + 12 * chunk);
        const f32x4 u = p[0], v = p[1], w = p[2];
        c = Coefs<5, 4>{{u[0], u[1], u[2], u[3], v[0], v[1]}, {v[2], v[3], w[0], w[1]}};
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = act_value<RAT == 1>(h[i], act, c);
}

// FORM as in ProductForm; PARTIAL: fp32 sums of a split to memory.
template <int BM, int BN, int BK, int FORM, bool PARTIAL, int RAT>
__global__ __launch_bounds__((TileShape<BM, BN, BK>::kThreads), 2) void grkan_linear_tile_kernel(ProductArgs a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    using Shape = TileShape<BM, BN, BK>;
    constexpr int T = Shape::kThreads, S = Shape::kStages;
    float *params = reinterpret_cast<float *>(lds + S * Shape::kStage);
    constexpr bool QS = FORM == kFormDw, PS = FORM != kFormForward;
    constexpr int WM = BM / 2, WN = BN / Shape::kWavesN, NM = WM / 32, NN = WN / 32;  // 32 x 32 blocks of a wave
    constexpr int kStage = Shape::kStage, kQ = BM * BK * 2;
    constexpr int KS = BK / 16;

    const int nb = (a.N + BN - 1) / BN, mb = (a.M + BM - 1) / BM, tiles = mb * nb;
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int mrow = wave / Shape::kWavesN * WM, ncol = wave % Shape::kWavesN * WN;

    // Tile b of the launch.  Workgroups go to the 8 XCDs in turn, and what an
    // XCD's workgroups share should stay in its L2, so each XCD takes an eighth
    // of the tiles: of all splits, those of a split together, its column tiles of a panel of
    // BM rows one after another.
    const int all = tiles * (PARTIAL ? a.splits : 1), per = (all + 7) / 8, count = per * 8;
    int m0, n0, split = 0, kb = 0, len = a.K;
    auto place = [&](int b) {
        const int t = (b & 7) * per + (b >> 3), i = PARTIAL ? t % tiles : t;
        if constexpr (PARTIAL) {
            split = t / tiles;
            kb = split * a.k_split;
            len = min(a.K - kb, a.k_split);
        }
        m0 = i / nb * BM;
        n0 = i % nb * BN;
    };
    // The next tile of this workgroup from b on, or `count` or more.
    auto next = [&](int b) {
        while (b < count && (b & 7) * per + (b >> 3) >= all) b += (int)gridDim.x;
        return b;
    };

    Stager<BM, BK, QS, T> sq;
    Stager<BN, BK, PS, T> sp;
    Reader<BM, BK, QS, NM> rq;
    Reader<BN, BK, PS, NN> rp;
    rq.init(mrow);
    rp.init(ncol);
    constexpr int kInFlight = Stager<BM, BK, QS, T>::kChunks + Stager<BN, BK, PS, T>::kChunks;

    f32x16 acc[NN][NM];
    bf16x8 fq[2][NM], fp[2][NN];
    auto multiply = [&](int set) {
#pragma unroll
        for (int j = 0; j < NN; ++j)
#pragma unroll
            for (int i = 0; i < NM; ++i)
                acc[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp[set][j], fq[set][i], acc[j][i], 0, 0, 0);
    };

    // The fetches run two steps ahead of the products, on through the tiles
    // of this workgroup: fetch_tile, fetch_step say what comes next.  Past
    // the last tile they read zeros, so the count in flight is fixed.
    int fetch_tile = next((int)blockIdx.x), fetch_step = 0, fetch_len = 0;
    if (fetch_tile >= count) return;
    auto start_tile = [&]() {
        if (fetch_tile < count) {
            place(fetch_tile);
            sq.init(a.q, m0, a.M, kb);
            sp.init(a.p, n0, a.N, kb);
            fetch_len = len;
        } else {
            fetch_len = 0;
        }
        fetch_step = 0;
    };
    auto fetch = [&](int stage, auto set) {
        const int left = fetch_len - fetch_step * BK;
        sq.template fetch<set()>(lds, stage, fetch_step, left);
        sp.template fetch<set()>(lds, stage + kQ, fetch_step, left);
        ++fetch_step;
        if (fetch_step * BK >= fetch_len && fetch_tile < count) {
            fetch_tile = next(fetch_tile + (int)gridDim.x);
            start_tile();
        }
    };
    auto put = [&](int stage, auto set) {
        sq.template put<set()>(lds, stage);
        sp.template put<set()>(lds, stage + kQ);
    };
    // The step whose chunks put has stored, or that was fetched into LDS before
    // the last kInFlight fetches (and `later` operations after it), has arrived.
    auto arrived = [&](auto later) {
        if constexpr (kAligned)
            wait_loads<(S - 2) * kInFlight + later()>();
        else
            __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    };
    constexpr std::integral_constant<int, 0> zero;
    constexpr std::integral_constant<int, 1> one;

    // Stages of steps t, t + 1, t + 2.
    int at[S];
#pragma unroll
    for (int i = 0; i < S; ++i) at[i] = i * kStage;
    int tile = fetch_tile;
    bool whole = false;  // the last tile stored by this workgroup had no edge
    bool odd = true;     // the register set of the next step
    constexpr int kStores = WM * WN / 512;
    start_tile();
    fetch(at[0], zero);
    put(at[0], zero);
#pragma unroll
    for (int i = 1; i < S - 1; ++i) fetch(at[i], one);
    arrived(zero);
    barrier();
    rq.read(lds + at[0], 0, fq[0]);
    rp.read(lds + at[0] + kQ, 0, fp[0]);
    static_assert(KS % 2 == 0, "the first fragments of a step are always set 0");
    for (; tile < count; tile = next(tile + (int)gridDim.x)) {
        place(tile);
        const int steps = (len + BK - 1) / BK;
        const int tm0 = m0, tn0 = n0, tsplit = split;
        if constexpr (!PARTIAL) load_params<RAT, BN, T>(params, a.e, tn0, a.N);
#pragma unroll
        for (int j = 0; j < NN; ++j)
#pragma unroll
            for (int i = 0; i < NM; ++i) acc[j][i] = f32x16{};
        // SET: the register set that holds (unaligned) step t + 1
        auto step = [&](int t, auto SET) {
            fetch(at[S - 1], std::integral_constant<int, 1 - SET()>{});
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int set = ks & 1;
                if (ks + 1 < KS) {
                    rq.read(lds + at[0], ks + 1, fq[set ^ 1]);
                    rp.read(lds + at[0] + kQ, ks + 1, fp[set ^ 1]);
                } else {
                    // step t + 1 has arrived, and every wave holds its last
                    // fragments of step t in registers
                    put(at[1], SET);
                    // memory operations end in the order of their issue: after a
                    // whole tile its kStores stores stand between step 1's fetch
                    // and step 2's, and need not be waited for
                    if (!PARTIAL && S > 2 && t == 0 && whole)
                        arrived(std::integral_constant<int, kStores>{});
                    else
                        arrived(zero);
                    barrier();
                    rq.read(lds + at[1], 0, fq[set ^ 1]);
                    rp.read(lds + at[1] + kQ, 0, fp[set ^ 1]);
                }
                multiply(set);
            }
            const int first = at[0];
#pragma unroll
            for (int i = 0; i + 1 < S; ++i) at[i] = at[i + 1];
            at[S - 1] = first;
        };
        if constexpr (kAligned) {
            for (int t = 0; t < steps; ++t) step(t, one);
        } else {
            for (int t = 0; t < steps; ++t, odd = !odd) {
                if (odd)
                    step(t, one);
                else
                    step(t, zero);
            }
        }
        // Here the first stage holds the next tile's first step (its first
        // fragments are in registers) and the last stage is free.

        // A lane's 16 accumulators of a block: row of the result lane mod 32,
        // columns 8 (v / 4) + 4 (lane / 32) + v mod 4.  Swapping the upper lanes of
        // quad 2 p with the lower lanes of quad 2 p + 1 leaves the lower lanes
        // columns 16 p + 0..7 and the upper ones 16 p + 8..15 of the same rows.
        const int mw = tm0 + mrow, nw = tn0 + ncol;
        auto take8 = [&](int j, int p, int i, float (&h)[8]) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[j][i][8 * p + v]),
                                                                __float_as_uint(acc[j][i][8 * p + 4 + v]), false, false);
                h[v] = __uint_as_float(w[0]);
                h[4 + v] = __uint_as_float(w[1]);
            }
        };
        if constexpr (PARTIAL) {
#pragma unroll
            for (int j = 0; j < NN; ++j)
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int i = 0; i < NM; ++i) {
                        float h[8];
                        take8(j, p, i, h);
                        const int m = mw + 32 * i + (lane & 31), n = nw + 32 * j + 16 * p + 8 * (lane >> 5);
                        if (m >= a.M) continue;
                        float *o = a.partials + ((int64_t)tsplit * a.M + m) * a.N + n;
                        if (n + 8 <= a.N) {
                            *reinterpret_cast<f32x4_any *>(o) = f32x4{h[0], h[1], h[2], h[3]};
                            *reinterpret_cast<f32x4_any *>(o + 4) = f32x4{h[4], h[5], h[6], h[7]};
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (n + e < a.N) o[e] = h[e];
                        }
                    }
        } else {
            // bf16 results pass through the wave's own corner of the free stage, 32 rows
            // of WN columns at a time, so that memory sees whole rows: from the
            // accumulators a lane holds 8 columns of 32 different rows (32-byte
            // pieces; storing those took 110 us of 420 at 50,432 x 3,072 from
            // 768).  Chunk c of row r sits at c ^ g(r), conflict-free both
            // ways.  The residual comes the same way, into the slot its result
            // will take.
            constexpr int CP = WN / 8, RP = 64 / CP;
            static_assert(T / 64 * 32 * WN * 2 <= kStage, "staging fits");
            char *own = lds + at[S - 1] + wave * (32 * WN * 2);
            auto slot = [&](int r, int c) {
                const int g = ((CP == 8 ? r : r >> 1) & (CP - 1)) ^ ((r >> 3) & 1);
                return reinterpret_cast<u32x4 *>(own + r * (WN * 2) + ((c ^ g) << 4));
            };
            const int row = lane / CP, chunk = lane % CP;
            const int cn = nw + chunk * 8, cnv = min(max(a.N - cn, 0), 8);
            auto fence = [] { asm volatile("" ::: "memory"); };  // LDS serves a wave in order
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                const int mh = mw + 32 * i;
                auto store_rows = [&](void *out) {
                    fence();
#pragma unroll
                    for (int it = 0; it < 32 / RP; ++it) {
                        const int r = it * RP + row;
                        if (mh + r < a.M && cnv > 0)
                            stream8(static_cast<uint16_t *>(out) + (int64_t)(mh + r) * a.N + cn, cnv, *slot(r, chunk));
                    }
                    fence();
                };
                // sums + bias, back in the accumulators in their new order
#pragma unroll
                for (int j = 0; j < NN; ++j)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const int c = 4 * j + 2 * p + (lane >> 5);
                        float h[8];
                        take8(j, p, i, h);
                        add_bias<BN>(h, params, ncol / 8 + c);
                        if (a.e.pre) *slot(lane & 31, c) = Io<bf16io>::pack(h);
#pragma unroll
                        for (int v = 0; v < 8; ++v) acc[j][i][8 * p + v] = h[v];
                    }
                if (a.e.pre) store_rows(a.e.pre);
                if (a.e.residual) {
#pragma unroll
                    for (int it = 0; it < 32 / RP; ++it) {
                        const int r = it * RP + row;
                        const int nv = mh + r < a.M ? cnv : 0;
                        *slot(r, chunk) = load8(
                            static_cast<const uint16_t *>(a.e.residual) + (nv ? (int64_t)(mh + r) * a.e.ldr + cn : 0), nv);
                    }
                    fence();
                }
#pragma unroll
                for (int j = 0; j < NN; ++j)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const int c = 4 * j + 2 * p + (lane >> 5);
                        float h[8];
#pragma unroll
                        for (int v = 0; v < 8; ++v) h[v] = acc[j][i][8 * p + v];
                        activate_tile<RAT, BN>(h, params, ncol / 8 + c, a.e.act);
                        u32x4 *to = slot(lane & 31, c);
                        if (a.e.residual) {
                            float r[8];
                            Io<bf16io>::unpack(*to, r);
#pragma unroll
                            for (int e = 0; e < 8; ++e) h[e] += r[e];
                        }
                        *to = Io<bf16io>::pack(h);
                    }
                store_rows(a.e.z);
            }
            whole = tm0 + BM <= a.M && tn0 + BN <= a.N;
            // the stage goes back to the fetches, the parameters to the next tile
            __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
            barrier();
        }
    }
    wait_loads<0>();  // nothing may still be on its way into LDS when the workgroup ends
}

// ------------------------------------------------------------ skinny kernel

// Few rows of x: a workgroup takes 16 columns of the result (16 rows of W)
// and 16 MT rows; its waves share the k range in turns of 64, each lane
// reading 32 consecutive bytes of a row of W (a line per row and turn) and of
// x, straight into the operand registers of v_mfma_f32_16x16x32_bf16: the
// order of k inside a turn is the lanes' own, the same for both operands.  The
// loads of up to kTurns turns are on their way at once.  The waves' sums meet in LDS,
// where one thread finishes 8 columns of a row.  Bound: W's bytes for many
// columns, latency below: 1 x 3,072 from 768 (4.7 MB) 4.4 us.
constexpr int kSkinnyWaves = 8;

template <int MT, int RAT>
__global__ __launch_bounds__(kSkinnyWaves * 64) void grkan_linear_skinny_kernel(ProductArgs a) {
    constexpr int kTurns = MT == 1 ? 4 : 2;
    __shared__ float red[kSkinnyWaves][MT * 16][17];
    const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6;
    const int n0 = (int)blockIdx.x * 16, m0 = (int)blockIdx.y * 16 * MT;
    // rows past the end are clamped (their results are not stored)
    const int kl = (lane >> 4) * 16;
    const uint16_t *W = static_cast<const uint16_t *>(a.p.p) + (int64_t)min(n0 + (lane & 15), a.N - 1) * a.p.ld + kl;
    const uint16_t *x[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
        x[i] = static_cast<const uint16_t *>(a.q.p) + (int64_t)min(m0 + 16 * i + (lane & 15), a.M - 1) * a.q.ld + kl;
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f32x4{};
    // k0 of this wave's turns: 64 wave, then every 64 kSkinnyWaves
    constexpr int kNext = 64 * kSkinnyWaves;
    int k0 = wave * 64;
    auto turns = [&](auto count, auto whole) {
        constexpr int U = count();
        u32x4 w[U][2], q[U][MT][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // whole: every chunk of these turns lies before K; else each lane
                // takes what does, and zeros past it for both operands
                const int k = k0 + u * kNext + 8 * h;
                const int nv = whole() ? 8 : min(max(a.K - k - kl, 0), 8);
                w[u][h] = load8(W + (nv ? k : 0), nv);
#pragma unroll
                for (int i = 0; i < MT; ++i) q[u][i][h] = load8(x[i] + (nv ? k : 0), nv);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w[u][h]),
                                                                     __builtin_bit_cast(bf16x8, q[u][i][h]), acc[i], 0, 0, 0);
        k0 += U * kNext;
    };
    while (k0 + (kTurns - 1) * kNext + 64 <= a.K) turns(std::integral_constant<int, kTurns>{}, std::true_type{});
    if (kTurns > 2 && k0 + kNext + 64 <= a.K) turns(std::integral_constant<int, 2>{}, std::true_type{});
    if (k0 + 64 <= a.K) turns(std::integral_constant<int, 1>{}, std::true_type{});
    if (k0 < a.K) turns(std::integral_constant<int, 1>{}, std::false_type{});
    // lane: row lane mod 16, columns 4 (lane / 16) + v
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[wave][16 * i + (lane & 15)][4 * (lane >> 4) + v] = acc[i][v];
    __syncthreads();
    for (int q = t; q < MT * 32; q += kSkinnyWaves * 64) {
        const int m = q >> 1, c = (q & 1) * 8;
        if (m0 + m >= a.M) continue;
        ChunkParams<RAT> k;
        k.init(a.e, n0 + c, a.N);
        float h[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kSkinnyWaves; ++w) s += red[w][m][c + e];
            h[e] = s;
        }
        finish8<RAT>(h, a.e, k, m0 + m, a.N);
    }
}

// ------------------------------------------------------------ second step

// The splits' sums added, then the epilogue.  SL lanes share the splits of 8
// columns (each adds every SL-th in order, the lanes' sums then in order through
// LDS), so that a small result with many splits still fills the GPU: 768 x 192
// is 18,432 columns of 8 (4.2 us with 16 splits); 768 x 3,072 in 7 splits, 66 MB
// from the Infinity Cache: 13 us, one lane per 8.
template <int RAT, int SL>
__global__ __launch_bounds__(256) void grkan_linear_finish_kernel(ProductArgs a) {
    constexpr int kItems = 256 / SL;
    __shared__ f32x4 red[SL > 1 ? SL : 1][SL > 1 ? 2 * kItems : 1];
    const int chunks = (a.N + 7) / 8, t = (int)threadIdx.x, x = t % kItems, sl = t / kItems;
    const int64_t total = (int64_t)chunks * a.M, plane = (int64_t)a.M * a.N;
    const int64_t i = (int64_t)blockIdx.x * kItems + x;
    const bool on = i < total;
    const int64_t m = on ? i / chunks : 0;
    const int n = on ? (int)(i - m * chunks) * 8 : 0;
    const int nv = min(a.N - n, 8);
    const float *p = a.partials + m * a.N + n + sl * plane;
    f32x4 u = {}, v = {};
#pragma unroll 4
    for (int s = sl; s < a.splits; s += SL, p += SL * plane) {
        if (nv == 8) {
            u += *reinterpret_cast<const f32x4_any *>(p);
            v += *reinterpret_cast<const f32x4_any *>(p + 4);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e < nv) u[e] += p[e];
                if (4 + e < nv) v[e] += p[4 + e];
            }
        }
    }
    if constexpr (SL > 1) {
        red[sl][2 * x] = u;
        red[sl][2 * x + 1] = v;
        __syncthreads();
        if (sl > 0) return;
#pragma unroll
        for (int q = 1; q < SL; ++q) {
            u += red[q][2 * x];
            v += red[q][2 * x + 1];
        }
    }
    if (!on) return;
    ChunkParams<RAT> k;
    k.init(a.e, n, a.N);
    float h[8] = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
    finish8<RAT>(h, a.e, k, m, a.N);
}

// ------------------------------------------------------------ dispatch

template <int BM, int BN, int BK, int FORM, bool PARTIAL, int RAT>
hipError_t launch_tile(const ProductArgs &a, hipStream_t s) {
    auto kern = grkan_linear_tile_kernel<BM, BN, BK, FORM, PARTIAL, RAT>;
    constexpr size_t lds = TileShape<BM, BN, BK>::kLds;
    static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (attr != hipSuccess) return attr;
    const int64_t mb = (a.M + BM - 1) / BM, nb = (a.N + BN - 1) / BN;
    int64_t grid = (mb * nb * (PARTIAL ? a.splits : 1) + 7) / 8 * 8;
    // as many workgroups as fit on the 256 CUs at once; each walks over its tiles
    constexpr int64_t resident = BN == 256 ? 256 : 768;
    if (grid > resident) grid = resident;
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3((TileShape<BM, BN, BK>::kThreads)), lds, s, a);
    return hipGetLastError();
}

template <int BM, int BN, int BK>
hipError_t launch_shape(int form, bool partial, bool rational, const ProductArgs &a, hipStream_t s) {
    if (form == kFormDw)
        return partial ? launch_tile<BM, BN, BK, kFormDw, true, 0>(a, s) : launch_tile<BM, BN, BK, kFormDw, false, 0>(a, s);
    if (form == kFormDx)
        return partial ? launch_tile<BM, BN, BK, kFormDx, true, 0>(a, s) : launch_tile<BM, BN, BK, kFormDx, false, 0>(a, s);
    if (partial) return launch_tile<BM, BN, BK, kFormForward, true, 0>(a, s);
    return rational ? launch_tile<BM, BN, BK, kFormForward, false, 1>(a, s)
                    : launch_tile<BM, BN, BK, kFormForward, false, 0>(a, s);
}

}  // namespace

// The tile kernels of this translation unit's alignment.
#if GRKAN_LINEAR_ALIGNED
#define GRKAN_LAUNCH_TILES launch_tiles_aligned
#else
#define GRKAN_LAUNCH_TILES launch_tiles_any
#endif
hipError_t GRKAN_LAUNCH_TILES(int tile, int form, bool partial, bool rational, const ProductArgs &a, hipStream_t s) {
    switch (tile) {
#if GRKAN_LINEAR_ALIGNED
        case 0: return launch_shape<256, 256, 64>(form, partial, rational, a, s);
#endif
        case 1: return launch_shape<128, 128, 32>(form, partial, rational, a, s);
        case 2: return launch_shape<64, 64, 64>(form, partial, rational, a, s);
        default: return hipErrorInvalidValue;
    }
}

#if !GRKAN_LINEAR_ALIGNED
hipError_t launch_tiles_aligned(int tile, int form, bool partial, bool rational, const ProductArgs &a, hipStream_t s);

namespace {
template <int RAT> hipError_t launch_skinny(int mt, const ProductArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.M + 16 * mt - 1) / (16 * mt))), block(kSkinnyWaves * 64);
    switch (mt) {
        case 1: hipLaunchKernelGGL((grkan_linear_skinny_kernel<1, RAT>), grid, block, 0, s, a); break;
        case 2: hipLaunchKernelGGL((grkan_linear_skinny_kernel<2, RAT>), grid, block, 0, s, a); break;
        default: hipLaunchKernelGGL((grkan_linear_skinny_kernel<4, RAT>), grid, block, 0, s, a); break;
    }
    return hipGetLastError();
}
}  // namespace

namespace {
template <int RAT> hipError_t launch_finish(const ProductArgs &a, hipStream_t s) {
    const int64_t work = (int64_t)((a.N + 7) / 8) * a.M;
    // lanes that share the splits, while a thread per 8 columns leaves CUs idle
    if (a.splits >= 4 && work < 64 * 1024)
        hipLaunchKernelGGL((grkan_linear_finish_kernel<RAT, 4>), dim3((unsigned)((work + 63) / 64)), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((grkan_linear_finish_kernel<RAT, 1>), dim3((unsigned)((work + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_product(int form, const ProductPlan &p, const ProductArgs &args, hipStream_t s) {
    if (!plan_has_kernel(p)) return hipErrorInvalidValue;
    ProductArgs a = args;
    a.splits = p.splits;
    a.k_split = p.k_split;
    const int rat = a.e.act != GRKAN_ACT_RATIONAL ? 0 : (a.e.dga % 8 == 0 ? 1 : 2);
    if (p.kind == kSkinny)
        return rat == 0 ? launch_skinny<0>(p.mt, a, s) : (rat == 1 ? launch_skinny<1>(p.mt, a, s) : launch_skinny<2>(p.mt, a, s));
    hipError_t e;
    if (p.rows > 0) {
        ProductArgs top = a, rest = a;
        top.M = (int32_t)p.rows;
        rest.M = a.M - top.M;
        rest.q.p = static_cast<const uint16_t *>(a.q.p) + p.rows * a.q.ld;
        if (a.e.residual) rest.e.residual = static_cast<const uint16_t *>(a.e.residual) + p.rows * a.e.ldr;
        if (a.e.pre) rest.e.pre = static_cast<uint16_t *>(a.e.pre) + p.rows * a.N;
        rest.e.z = static_cast<uint16_t *>(a.e.z) + p.rows * a.N;
        e = launch_tiles_aligned(p.tile, form, false, rat == 1, top, s);
        return e != hipSuccess ? e : launch_tiles_aligned(p.rest_tile, form, false, rat == 1, rest, s);
    }
    e = p.aligned ? launch_tiles_aligned(p.tile, form, p.two_steps, rat == 1, a, s)
                  : launch_tiles_any(p.tile, form, p.two_steps, rat == 1, a, s);
    if (e != hipSuccess || !p.two_steps) return e;
    return rat == 0 ? launch_finish<0>(a, s) : (rat == 1 ? launch_finish<1>(a, s) : launch_finish<2>(a, s));
}

// ------------------------------------------------------------ dpre, dbias

namespace {

// dpre = dz act'(pre) with its column sums (dbias) and the rational's coefficient
// sums: one pass, two rows of a lane on their way while one is worked on; column
// sums stay in registers over a workgroup's rows.  dpre is rounded to bf16, the
// matrix cores' operand type for dx and dW (their relative error 0.0023 in place
// of 0.0017 with fp32 dpre); dbias, dA and dB are summed from the fp32 values.
// 50,432 x 768, silu: 48 us (43 the fastest), 4.8 TB/s, memory.  25,216 x 768, the
// rational: 35.5 us, 3.3 TB/s, its 58 instructions an element.
template <int V, bool RAT>
__global__ __launch_bounds__(kSlopeTx * kSlopeTy) void grkan_linear_slope_kernel(SlopeArgs a) {
    __shared__ float red[kSlopeTy][kSlopeTx * V + 1];
    __shared__ float redc[RAT ? kSlopeTy : 1][RAT ? 10 * kSlopeTx : 1];
    const int t = (int)threadIdx.x, tx = t % kSlopeTx, ty = t / kSlopeTx;
    const int vi = (int)blockIdx.x * kSlopeTx + tx, n = vi * V, nv = min(max(a.N - n, 0), V);
    const int64_t r0 = (int64_t)blockIdx.y * a.chunk_rows, r1 = min(a.rows, r0 + a.chunk_rows);
    const uint16_t *dz = static_cast<const uint16_t *>(a.dz) + n, *pre = static_cast<const uint16_t *>(a.pre) + n;
    uint16_t *out = static_cast<uint16_t *>(a.dpre) + n;
    float sum[V], coef[RAT ? 10 : 1] = {};
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.0f;
    ExactSlopeCoefs sc;
    if constexpr (RAT) sc.init(load_coefs<5, 4>(a.A, a.B, nv > 0 ? n / a.dga : 0));
    auto value = [](u32x4 v, int e) { return __uint_as_float((e & 1) ? (v[e / 2] & 0xffff0000u) : (v[e / 2] << 16)); };
    // the next row's values are on their way while this one's are worked on
    auto fetch = [&](int64_t r, u32x4 &g, u32x4 &h) {
        if (r >= r1) return;
        g = V == 8 ? load8(dz + r * a.lddz, nv) : u32x4{dz[r * a.lddz], 0u, 0u, 0u};
        if (a.act != GRKAN_ACT_NONE) h = V == 8 ? load8(pre + r * a.N, nv) : u32x4{pre[r * a.N], 0u, 0u, 0u};
    };
    if (nv > 0) {
        u32x4 ng[2] = {}, nh[2] = {};
        fetch(r0 + ty, ng[0], nh[0]);
        fetch(r0 + ty + kSlopeTy, ng[1], nh[1]);
        for (int64_t r = r0 + ty; r < r1; r += kSlopeTy) {
            const u32x4 g = ng[0], h = nh[0];
            ng[0] = ng[1];
            nh[0] = nh[1];
            fetch(r + 2 * kSlopeTy, ng[1], nh[1]);
            float d[8] = {};
            if (a.act == GRKAN_ACT_NONE) {
#pragma unroll
                for (int e = 0; e < V; ++e) sum[e] += value(g, e);
                continue;
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float he = value(h, e), ge = value(g, e);
                if constexpr (RAT) {
                    // pre is what the forward kept, an exact input: Q and its sign are
                    // formed as by the activation's own backward
                    d[e] = rational_slope(he, ge, sc, *reinterpret_cast<float (*)[10]>(coef));
                } else {
                    d[e] = ge * act_slope(he, a.act);
                }
                sum[e] += d[e];
            }
            if constexpr (V == 8)
                store8(out + r * a.ldp, nv, Io<bf16io>::pack(d));
            else
                out[r * a.ldp] = __builtin_bit_cast(uint16_t, (__bf16)d[0]);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) red[ty][tx * V + e] = sum[e];
    if constexpr (RAT) {
#pragma unroll
        for (int k = 0; k < 10; ++k) redc[ty][k * kSlopeTx + tx] = coef[k];
    }
    __syncthreads();
    float *p = a.partials + (int64_t)blockIdx.y * (a.N + (RAT ? 10 * (int64_t)a.vpr : 0));
    for (int i = t; i < kSlopeTx * V; i += kSlopeTx * kSlopeTy) {
        const int c = (int)blockIdx.x * kSlopeTx * V + i;
        if (c >= a.N) continue;
        float s = 0.0f;
        for (int q = 0; q < kSlopeTy; ++q) s += red[q][i];
        p[c] = s;
    }
    if constexpr (RAT) {
        for (int i = t; i < 10 * kSlopeTx; i += kSlopeTx * kSlopeTy) {
            const int v = (int)blockIdx.x * kSlopeTx + i % kSlopeTx, k = i / kSlopeTx;
            if (v >= a.vpr) continue;
            float s = 0.0f;
            for (int q = 0; q < kSlopeTy; ++q) s += redc[q][i];
            p[a.N + (int64_t)k * a.vpr + v] = s;
        }
    }
}

// Column partials over their rows in fp64: 64 columns x 16 row lanes a
// workgroup, then one workgroup per (activation group, coefficient).  5.6 us for
// 512 rows of 768 columns and 960 coefficient sums: latency.
template <bool RAT>
__device__ static inline void add_columns(const SlopeArgs &a, int b, double *red) {
    const int t = (int)threadIdx.x;
    const int64_t row = a.N + (RAT ? 10 * (int64_t)a.vpr : 0);
    const int colblocks = (a.N + 63) / 64;
    double s = 0.0;
    if (b < colblocks) {
        const int c = b * 64 + (t & 63);
        if (c < a.N) {
#pragma unroll 8
            for (int r = t >> 6; r < a.chunks; r += 16) s += (double)a.partials[r * row + c];
        }
        red[t] = s;
        __syncthreads();
        if (t < 64 && c < a.N && a.dbias) {
            for (int q = 1; q < 16; ++q) s += red[t + 64 * q];
            a.dbias[c] = (float)s;
        }
        return;
    }
    if constexpr (RAT) {
        const int gk = b - colblocks, g = gk / 10, k = gk % 10;
        const int v0 = g * a.dga / a.vec, w = a.dga / a.vec;
#pragma unroll 8
        for (int64_t i = t; i < (int64_t)a.chunks * w; i += 1024) {
            const int64_t r = i / w;
            s += (double)a.partials[r * row + a.N + (int64_t)k * a.vpr + v0 + (i - r * w)];
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
__global__ __launch_bounds__(1024) void grkan_linear_columns_kernel(SlopeArgs a, int total) {
    __shared__ double red[1024];
    for (int b = (int)blockIdx.x; b < total; b += (int)gridDim.x) {
        add_columns<RAT>(a, b, red);
        __syncthreads();  // the sums in LDS have been read
    }
}

}  // namespace

hipError_t launch_slope(const SlopeArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)((a.vpr + kSlopeTx - 1) / kSlopeTx), (unsigned)a.chunks), block(kSlopeTx * kSlopeTy);
    const bool rational = a.act == GRKAN_ACT_RATIONAL;
    if (!rational)
        hipLaunchKernelGGL((grkan_linear_slope_kernel<8, false>), grid, block, 0, s, a);
    else if (a.vec == 8)
        hipLaunchKernelGGL((grkan_linear_slope_kernel<8, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((grkan_linear_slope_kernel<1, true>), grid, block, 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || (!a.dbias && !rational)) return e;
    const int total = (a.N + 63) / 64 + (rational ? a.ng * 10 : 0);
    const dim3 rgrid((unsigned)(total < kMaxBlocks ? total : kMaxBlocks));
    if (rational)
        hipLaunchKernelGGL((grkan_linear_columns_kernel<true>), rgrid, dim3(1024), 0, s, a, total);
    else
        hipLaunchKernelGGL((grkan_linear_columns_kernel<false>), rgrid, dim3(1024), 0, s, a, total);
    return hipGetLastError();
}
#endif

}  // namespace grkan
