// grkan_product8.hip -- c = a b^T of e4m3 operands with a scale for each block
// of 128 values of k, on the matrix cores (gfx950).
//
// A block's products are summed from zero; its sum times both scales is added
// to the accumulators in fp32.  Two ways to sum a block (the kernels' CUT):
//
// the values widened to bf16, exactly, and four v_mfma_f32_16x16x32_bf16, whose sums
// are fp32's (1e-7);
//
// where the caller of a bf16 result asks for it, one v_mfma_f32_16x16x128_f8f6f4, at twice the
// rate.  It cuts the products of each 8 values of k off at 2^-13 of the largest one's power
// of two before adding them (measured; the groups of 8 are added in fp32;
// v_mfma_f32_16x16x32_fp8_fp8 does the same).  Results are 1.5e-5 to 5e-5 of their norm
// off, a fortieth of the rounding to bf16 in the mean; a value whose large products cancel may
// be off by more than its own rounding.  50,432 x 3,072 from 768: 150 us against 248; 4,096 x
// 768 from 3,072: 21.5 and 34; 1,003 x 1,501 from 777: 9.1 and 10.9.
//
// Bound, large products, cut sums: LDS (of a 256 x 256 tile's step 192 KB are read and 64 KB written,
// 2,048 cycles of a CU) and the matrix cores (2,048 cycles) side by side, with the
// additions (1,360 cycles of a SIMD) between them, at the clock that the power allows
// (1.95 GHz).  8,192 x 8,192 from 8,192: 460 us, 2,390 TFLOP/s (a library product with
// one scale for all: 3,307).  At short k the results' way out joins them: of 171 us for
// 50,432 x 3,072 from 768 (154 since) 26 went with the stores left out and 21 more with
// what comes before them.
#include "grkan_fp8.h"
#include "grkan_lanes.h"

#include <type_traits>

namespace grkan {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// 16 bytes at p of which the first nv (0..16) exist; the others read as zeros.
__device__ static inline u32x4 chunk16(const uint8_t *p, int nv) {
    if (nv <= 0) return u32x4{0u, 0u, 0u, 0u};
    u32x4 v = *reinterpret_cast<const u32x4 *>(p);
    if (nv < 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int left = nv - 4 * i;
            v[i] = left <= 0 ? 0u : (left >= 4 ? v[i] : v[i] & ((1u << (8 * left)) - 1u));
        }
    }
    return v;
}

__device__ static inline f32x4 mfma8(i32x8 a, i32x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

// 8 e4m3 values as bf16.
__device__ static inline bf16x8 widen(uint32_t lo, uint32_t hi) {
    const bf16x2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A block's sum of products, cut as above or fp32's own.
template <bool CUT> __device__ static inline f32x4 block_product(i32x8 a, i32x8 b) {
    if constexpr (CUT) return mfma8(a, b, f32x4{});
    f32x4 c = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(a[2 * i], a[2 * i + 1]), widen(b[2 * i], b[2 * i + 1]), c, 0, 0, 0);
    return c;
}

// ------------------------------------------------------------ tile kernel

typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

constexpr uint32_t kNowhere = 0x80000000u;  // past every buffer: reads zeros

// 16 (or 4) bytes per lane from offset `off` of the buffer to LDS, lane after
// lane from address `to` (the same in all lanes; taken from M0).  Written as
// instructions because they have no result; arrival is waited for by count.  M0 is
// the compiler's to use nowhere else in these kernels.
__device__ static inline uint32_t lds_address(const char *p) {
    return (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char *)p);
}
__device__ static inline uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
__device__ static inline void fetch16(u32x4 rsrc, uint32_t off, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" : : "s"(uniform(to)), "v"(off), "s"(rsrc) : "memory");
}
__device__ static inline void fetch4(u32x4 rsrc, uint32_t off, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" : : "s"(uniform(to)), "v"(off), "s"(rsrc) : "memory");
}
__device__ static inline u32x4 resource(const void *p, uint32_t bytes) {
    const uint64_t addr = reinterpret_cast<uint64_t>(p);
    return u32x4{uniform((uint32_t)addr), uniform((uint32_t)(addr >> 32)) & 0xffffu, uniform(bytes), 0x00020000u};
}
// s_waitcnt vmcnt(n), lgkmcnt(0), and lgkmcnt(0) alone.
template <int N> __device__ static inline void wait_loads() {
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
}
__device__ static inline void wait_lds() { __builtin_amdgcn_s_waitcnt(0xc07f); }
__device__ static inline void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Nothing moves across: the compiler would gather the fragments' reads early, in
// registers that there are not.
__device__ static inline void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// The chunk (16 bytes) c of a row of 128 bytes sits at c ^ swizzle(row): 8
// consecutive rows of one chunk column cover 128 bytes of banks and 16 cover 256.
__device__ static inline int swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// An operand's rows of a tile: ROWS x 128 codes by threads of 16 bytes.  Rows past
// the end lie past the buffer's (they read zeros).
template <int ROWS, int T> struct Codes {
    static constexpr int kChunks = ROWS * 8 / T;
    static_assert(ROWS * 8 % T == 0 && T / 8 % 16 == 0, "whole chunks, one swizzle a thread");
    const uint8_t *base;
    uint32_t bytes;      // from base to the end of the last row
    uint32_t off;        // of this thread's first chunk; the next lie `step` apart
    int step;
    __device__ inline void init(const Operand8 &o, int row0, int rows, int kstart) {
        const int r0 = (int)threadIdx.x / 8;
        base = o.p + (int64_t)row0 * o.ld + kstart;
        bytes = (uint32_t)(min(rows - row0, ROWS) * o.ld - kstart);
        off = (uint32_t)(r0 * o.ld + first());
        step = (int)(T / 8 * o.ld);
    }
    // k of this thread's chunks
    __device__ static inline int first() { return (((int)threadIdx.x & 7) ^ swizzle((int)threadIdx.x / 8)) * 16; }
    // The chunks of step t, `left` values of k before its end: begin, then each chunk
    // into its place of a stage.
    u32x4 rsrc;
    uint32_t from;
    __device__ inline void begin(int t, int left) {
        rsrc = resource(base + (int64_t)t * kBlock8, left > 0 ? bytes - (uint32_t)t * kBlock8 : 0u);
        from = left >= kBlock8 || first() < left ? off : kNowhere;
    }
    __device__ inline void fetch(uint32_t stage, int wave, int i) const {
        fetch16(rsrc, from + (uint32_t)(i * step), stage + (i * T + wave * 64) * 16);
    }
};

template <int BM, int BN> struct Tile8 {
    static constexpr int kWavesM = 2, kWavesN = BN == 256 ? 4 : 2, kThreads = kWavesM * kWavesN * 64;
    static constexpr int WM = BM / kWavesM, WN = BN / kWavesN, NM = WM / 16, NN = WN / 16;
    // codes of a, of b, then a scale a thread: BM of a's, BN of b's
    static constexpr int kScales = (BM + BN) * kBlock8;
    static constexpr int kStage = kScales + kThreads * 4;
    // two stages, a corner for each wave's 16 rows of bf16 results, the bias of two tiles'
    // columns
    static constexpr int kCorner = 16 * WN * 2, kCorners = 2 * kStage;
    static constexpr int kBias = kCorners + kThreads / 64 * kCorner;
    static constexpr size_t kLds = kBias + 2 * (size_t)BN * 4;
    static_assert(BM + BN <= kThreads && BM % 64 == 0, "a scale a thread, one operand's a wave");
};

// A block of k at a time through two LDS stages.  T: the result's type.  A 256 x 256
// tile in 8 waves of 128 x 64 leaves each byte of LDS the most products that the
// accumulators' registers allow (128 of 256); 128 x 128 and 64 x 64, 4 waves, give two and
// four workgroups to a CU where there are fewer tiles.  The 256 x 256 tile spills 21 vector and 69 scalar
// registers (88 bytes a lane).  fp32 sums: a step of a wave is 128 conversions, 64 matrix
// instructions and 64 to 128 additions, which follow one another more than they overlap: matrix cores
// busy 0.46 (3,072 x 768 from 50,432 in 7 splits: 256 us, 930 TFLOP/s).  Not the
// conversions alone: a form of it with every conversion between two matrix instructions took 249,
// and one with 32 x 32 x 16 instructions and codes read a step ahead 255, of which 208 were left
// without the additions, 221 without the fetches and no less without the conversions.
//
// In the middle of a step every wave holds what is left of it in registers: a barrier
// there covers both that and the arrival of the next step, and the fetches of the
// step after that go into the stage just freed, a whole step ahead of their use.
template <int BM, int BN, class T, bool CUT, bool BTILE, bool PARTIAL>
__global__ __launch_bounds__((Tile8<BM, BN>::kThreads), 2) void grkan_product8_tile_kernel(Product8Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    using Shape = Tile8<BM, BN>;
    constexpr int TH = Shape::kThreads, WM = Shape::WM, WN = Shape::WN, NM = Shape::NM, NN = Shape::NN;
    constexpr int kStage = Shape::kStage, kB = BM * kBlock8, kScales = Shape::kScales;
    const int nb = (a.N + BN - 1) / BN, mb = (a.M + BM - 1) / BM, tiles = mb * nb;
    const int t = (int)threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int mrow = wave / Shape::kWavesN * WM, ncol = wave % Shape::kWavesN * WN;

    // Tile b of the launch.  Workgroups go to the 8 XCDs in turn, and what an
    // XCD's workgroups share should stay in its L2, so each XCD takes an eighth
    // of the tiles (of all splits, those of a split together), its column tiles of
    // a panel of BM rows one after another.
    const int all = tiles * (PARTIAL ? a.splits : 1), per = (all + 7) / 8, count = per * 8;
    int m0, n0, split = 0, kb = 0, len = a.K;
    auto place = [&](int b) {
        const int i = (b & 7) * per + (b >> 3), tile = PARTIAL ? i % tiles : i;
        if constexpr (PARTIAL) {
            split = i / tiles;
            kb = split * a.k_split;
            len = min(a.K - kb, a.k_split);
        }
        m0 = tile / nb * BM;
        n0 = tile % nb * BN;
    };
    auto next = [&](int b) {
        while (b < count && (b & 7) * per + (b >> 3) >= all) b += (int)gridDim.x;
        return b;
    };

    // The fetches run two steps ahead of the products, on through the tiles of this
    // workgroup; past the last they read zeros, so the number in flight is fixed.
    constexpr int kInFlight = Codes<BM, TH>::kChunks + Codes<BN, TH>::kChunks + 1;
    Codes<BM, TH> ca;
    Codes<BN, TH> cb;
    const float *scale_base;
    uint32_t scale_off;
    int64_t scale_step;
    int fetch_tile = next((int)blockIdx.x), fetch_step = 0, fetch_len = 0;
    if (fetch_tile >= count) return;
    auto start_tile = [&]() {
        if (fetch_tile < count) {
            place(fetch_tile);
            ca.init(a.a, m0, a.M, kb);
            cb.init(a.b, n0, a.N, kb);
            const bool of_a = wave * 64 < BM;   // a wave's scales are one operand's
            const Operand8 &o = of_a ? a.a : a.b;
            const int first = of_a ? m0 : n0, i = of_a ? t : t - BM;
            const bool there = i < (of_a ? BM : BN) && first + i < (of_a ? a.M : a.N);
            const bool tiled = BTILE && !of_a;
            const int at = tiled ? (first + i) / kBlock8 - first / kBlock8 : i;
            scale_base = o.scale + (tiled ? first / kBlock8 : first) * o.srow + kb / kBlock8 * o.sblock;
            scale_off = there ? (uint32_t)(at * o.srow * 4) : kNowhere;
            scale_step = o.sblock;
            fetch_len = len;
        } else {
            fetch_len = 0;
        }
        fetch_step = 0;
    };
    u32x4 scale_rsrc;
    auto fetch_begin = [&]() {
        const int left = fetch_len - fetch_step * kBlock8;
        ca.begin(fetch_step, left);
        cb.begin(fetch_step, left);
        scale_rsrc = resource(scale_base + fetch_step * scale_step, left > 0 ? 0x7ffffff0u : 0u);
    };
    const uint32_t base = lds_address(lds);
    auto fetch_part = [&](int stage, int i) {
        if (i < ca.kChunks)
            ca.fetch(base + stage, wave, i);
        else if (i < ca.kChunks + cb.kChunks)
            cb.fetch(base + stage + kB, wave, i - ca.kChunks);
        else
            fetch4(scale_rsrc, scale_off, base + stage + kScales + wave * 256);
    };
    auto fetch_end = [&]() {
        ++fetch_step;
        if (fetch_step * kBlock8 >= fetch_len && fetch_tile < count) {
            fetch_tile = next(fetch_tile + (int)gridDim.x);
            start_tile();
        }
    };
    auto fetch = [&](int stage) {
        fetch_begin();
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) fetch_part(stage, i);
        fetch_end();
    };
    // A chunk that reaches past K: what lies there is the caller's, and cleared here.
    const int ragged = a.K & 15;
    auto clear_past = [&](int stage) {
        const int c = (a.K & 127) >> 4;
        for (int row = t; row < BM + BN; row += TH) {
            const int r = row < BM ? row : row - BM;
            u32x4 *p = reinterpret_cast<u32x4 *>(lds + stage + row * kBlock8 + ((c ^ swizzle(r)) << 4));
            u32x4 v = *p;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int left = ragged - 4 * i;
                v[i] = left <= 0 ? 0u : (left >= 4 ? v[i] : v[i] & ((1u << (8 * (left & 3))) - 1u));
            }
            *p = v;
        }
        wait_lds();
        barrier();
    };

    // Fragments: 32 of the 128 codes of row lane mod 16 to a lane; which 32 does not
    // matter as long as both operands' lanes hold the same.
    const int frow = lane & 15, fc = 2 * (lane >> 4);
    const int f0 = frow * kBlock8 + ((fc ^ swizzle(frow)) << 4), f1 = frow * kBlock8 + (((fc + 1) ^ swizzle(frow)) << 4);
    auto read = [&](int at) {
        const i32x4 lo = *reinterpret_cast<const i32x4 *>(lds + at + f0), hi = *reinterpret_cast<const i32x4 *>(lds + at + f1);
        return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    auto read_a = [&](int stage, int i) { return read(stage + (mrow + 16 * i) * kBlock8); };
    auto read_b = [&](int stage, int j) { return read(stage + kB + (ncol + 16 * j) * kBlock8); };

    f32x4 acc[NM][NN];
    // The rows' fragments of a step, in the order that they are multiplied: X, read during
    // the step before; Y and Z, read at its start; W, read into X's registers once those
    // are through.  Z and W are multiplied after the barrier, while the next step's X and
    // columns are read, X into Y's registers: the two change places from step to step.
    constexpr int Y = NM == 8 ? 2 : 0, W = Y, X = (NM - 2 * Y) / 2, Z = X;
    static_assert(X + Y + Z + W == NM && (Y == 0 || Y == X), "all rows");
    i32x8 fr[2][X], fz[Z], fb[NN];
    float as[NM];
    // The wave's results to memory: rows m0 .., columns n0 ...  WHOLE: all of the tile's
    // exist.
    int turn = 0;  // which half of the bias
    auto finish = [&](auto all_there, int m0, int n0, int split) {
        constexpr bool WHOLE = all_there();
        const int mw = m0 + (lane & 15), nw = n0 + 4 * (lane >> 4);
        const float *bias = reinterpret_cast<const float *>(lds + Shape::kBias) + turn * BN + ncol + 4 * (lane >> 4);
        if constexpr (PARTIAL || sizeof(T) == 4) {
            // 16 bytes a lane, 64 side by side of a row
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                const int m = mw + 16 * i;
                if (!WHOLE && m >= a.M) continue;
#pragma unroll
                for (int j = 0; j < NN; ++j) {
                    const int n = nw + 16 * j, nv = WHOLE ? 4 : min(a.N - n, 4);
                    if (nv <= 0) continue;
                    f32x4 h = acc[i][j];
                    float *o;
                    if constexpr (PARTIAL) {
                        o = a.partials + ((int64_t)split * a.M + m) * a.N + n;
                    } else {
                        o = static_cast<float *>(a.c) + (int64_t)m * a.N + n;
                        h += *reinterpret_cast<const f32x4 *>(bias + 16 * j);
                        if (a.residual) {
                            const float *r = static_cast<const float *>(a.residual) + m * a.ldr + n;
                            h += nv == 4 ? f32x4(*reinterpret_cast<const f32x4_any *>(r)) : load4<false>(r, nv);
                        }
                    }
                    if (nv == 4)
                        *reinterpret_cast<f32x4_any *>(o) = h;
                    else
                        store4<false>(o, nv, h);
                }
            }
        } else {
            // bf16 results pass through the wave's own corner of LDS, 16 rows of WN columns at a
            // time, so that memory sees whole rows.  Chunk c (8 columns) of row r sits at
            // c ^ (r mod CP).  A residual comes the same way, into the place of its result.
            constexpr int CP = WN / 8, RP = 64 / CP;
            char *own = lds + Shape::kCorners + wave * Shape::kCorner;
            auto slot = [&](int r, int c) { return own + r * (WN * 2) + ((c ^ (r & (CP - 1))) << 4); };
            const int row = lane / CP, chunk = lane % CP;
            const int cn = n0 + chunk * 8, cnv = WHOLE ? 8 : min(max(a.N - cn, 0), 8);
            auto fence = [] { asm volatile("" ::: "memory"); };  // LDS serves a wave in order
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                const int mh = m0 + 16 * i;
                if (a.residual) {
#pragma unroll
                    for (int it = 0; it < 16 / RP; ++it) {
                        const int r = it * RP + row;
                        const uint16_t *from = static_cast<const uint16_t *>(a.residual) + (int64_t)(mh + r) * a.ldr + cn;
                        u32x4 v = {0u, 0u, 0u, 0u};
                        if (WHOLE || mh + r < a.M) {
                            if (WHOLE || cnv == 8) {
                                v = *reinterpret_cast<const u32x4_any *>(from);
                            } else {
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    if (e < cnv) v[e / 2] |= (uint32_t)from[e] << (16 * (e & 1));
                            }
                        }
                        *reinterpret_cast<u32x4 *>(slot(r, chunk)) = v;
                    }
                    fence();
                }
#pragma unroll
                for (int j = 0; j < NN; ++j) {
                    f32x4 h = acc[i][j] + *reinterpret_cast<const f32x4 *>(bias + 16 * j);
                    char *to = slot(lane & 15, 2 * j + (lane >> 5)) + ((lane >> 4) & 1) * 8;
                    if (a.residual) {
                        const u32x2 r = *reinterpret_cast<const u32x2 *>(to);
                        h += f32x4{__uint_as_float(r[0] << 16), __uint_as_float(r[0] & 0xffff0000u),
                                   __uint_as_float(r[1] << 16), __uint_as_float(r[1] & 0xffff0000u)};
                    }
                    *reinterpret_cast<u32x2 *>(to) = pack4(h);
                }
                fence();
#pragma unroll
                for (int it = 0; it < 16 / RP; ++it) {
                    const int r = it * RP + row;
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(slot(r, chunk));
                    if (!WHOLE && (mh + r >= a.M || cnv <= 0)) continue;
                    uint16_t *to = static_cast<uint16_t *>(a.c) + (int64_t)(mh + r) * a.N + cn;
                    if (WHOLE || cnv == 8) {
                        __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any *>(to));
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (e < cnv) to[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
                    }
                }
                fence();
            }
        }
    };
    int now = 0;   // the stage of this step
    start_tile();
    fetch(0);
    fetch(kStage);
    wait_loads<kInFlight>();
    barrier();
    int tile = next((int)blockIdx.x);
    bool first = true;
    bool whole = false;  // the last tile stored by this workgroup had no edge
    constexpr int kStores = PARTIAL || sizeof(T) == 4 ? NM * NN : NM * WN / 32;
    for (; tile < count; tile = next(tile + (int)gridDim.x)) {
        place(tile);
        const int steps = (len + kBlock8 - 1) / kBlock8;
        const int tm0 = m0, tn0 = n0, tsplit = split;
        const bool ends = ragged && kb + len == a.K;
        // the bias of this tile's columns: a wave that is a tile ahead writes the other half
        turn ^= 1;
        if (!PARTIAL && t < BN)
            reinterpret_cast<float *>(lds + Shape::kBias)[turn * BN + t] = a.bias && tn0 + t < a.N ? a.bias[tn0 + t] : 0.0f;
        auto scales_of = [&](int stage, int i) {
            return reinterpret_cast<const float *>(lds + stage + kScales)[mrow + 16 * i + (lane & 15)];
        };
        if (first) {
            if (ends && steps == 1) clear_past(now);
            first = false;
#pragma unroll
            for (int i = 0; i < X; ++i) fr[0][i] = read_a(now, i);
#pragma unroll
            for (int j = 0; j < NN; ++j) fb[j] = read_b(now, j);
#pragma unroll
            for (int i = 0; i < X + Y; ++i) as[i] = scales_of(now, i);
        }
#pragma unroll
        for (int i = 0; i < NM; ++i)
#pragma unroll
            for (int j = 0; j < NN; ++j) acc[i][j] = f32x4{};
        auto step = [&](int st, auto parity) {
            constexpr int PX = Y > 0 ? parity() : 0, PY = 1 - PX;
            const int other = kStage - now;
            const float *sb = reinterpret_cast<const float *>(lds + now + kScales) + BM + ncol + (BTILE ? 0 : 4 * (lane >> 4));
            f32x4 bs[NN];
            float bt = 0.0f;
            if constexpr (BTILE) {
                bt = *sb;
            } else {
#pragma unroll
                for (int j = 0; j < NN; ++j) bs[j] = *reinterpret_cast<const f32x4 *>(sb + 16 * j);
            }
#pragma unroll
            for (int i = 0; i < Y; ++i) fr[PY][i] = read_a(now, X + i);
#pragma unroll
            for (int i = 0; i < Z; ++i) fz[i] = read_a(now, X + Y + i);
#pragma unroll
            for (int i = X + Y; i < NM; ++i) as[i] = scales_of(now, i);
            // Products kAhead of the sums they are added to, so that the matrix unit's
            // result is there; pinned, or the compiler moves the additions past the
            // barrier and keeps the products.  8,192 x 8,192 from 8,192: 484 us with 2, 460
            // with 3, 770 with 4, for which tiles of 256 have no registers; in tiles of 128
            // 15,443 x 2,112 from 3,648 149 with 2, 145 with 4, and 3,072 x 768 from
            // 50,432 in fp32, whose products take longer, 464 with 2, 475 with 4.
            constexpr int kAhead = CUT ? (BN == 256 ? 3 : 4) : 2;
            f32x4 p[kAhead + 1];
            auto add = [&](int slot, int i, int j) {
                const float s = BTILE ? as[i] * bt : as[i];
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(p[slot][v], BTILE ? s : s * bs[j][v], acc[i][j][v]);
                asm volatile("" : "+v"(acc[i][j]));
            };
            keep_order();
            constexpr int kFirst = (X + Y) * NN;
#pragma unroll
            for (int q = 0; q < kFirst + kAhead; ++q) {
                if (q < kFirst) {
                    const int i = q / NN, j = q % NN;
                    p[q % (kAhead + 1)] = block_product<CUT>(fb[j], i < X ? fr[PX][i < X ? i : 0] : fr[PY][i < X ? 0 : i - X]);
                    if (i < W && j == NN - 1) fr[PX][i] = read_a(now, X + Y + Z + i);
                }
                if (q >= kAhead) add((q - kAhead) % (kAhead + 1), (q - kAhead) / NN, (q - kAhead) % NN);
            }
            // memory operations end in the order of their issue: after a whole tile its
            // kStores stores stand behind the next step's fetches, and need not be waited
            // for
            if (st == 0 && whole)
                wait_loads<kStores>();
            else
                wait_loads<0>();
            barrier();
            if (ragged) {
                // (the next step is this tile's last, or the next tile's only one)
                const bool here = st + 1 < steps;
                bool past = here ? ends && st + 2 == steps : false;
                if (!here) {
                    const int b = next(tile + (int)gridDim.x);
                    if (b < count) {
                        place(b);
                        past = kb + len == a.K && len <= kBlock8;
                    }
                }
                if (past) clear_past(other);
            }
            fetch_begin();
#pragma unroll
            for (int i = 0; i < X; ++i) fr[Y > 0 ? PY : 0][i] = read_a(other, i);
            constexpr int R = Z + W, kRest = R * NN;
            keep_order();
#pragma unroll
            for (int q = 0; q < kRest + kAhead; ++q) {
                if (q < kRest) {
                    const int j = q / R, i = q % R;
                    p[q % (kAhead + 1)] = block_product<CUT>(fb[j], i < Z ? fz[i < Z ? i : 0] : fr[PX][i < Z ? 0 : i - Z]);
                    if (i == R - 1) fb[j] = read_b(other, j);
                    // the fetches, spread over the products
#pragma unroll
                    for (int k = q * kInFlight / kRest; k < (q + 1) * kInFlight / kRest; ++k) fetch_part(now, k);
                }
                if (q >= kAhead) add((q - kAhead) % (kAhead + 1), X + Y + (q - kAhead) % R, (q - kAhead) / R);
                if (q == kRest / 2) {
#pragma unroll
                    for (int i = 0; i < X + Y; ++i) as[i] = scales_of(other, i);
                }
            }
            fetch_end();
            now = other;
        };
        constexpr std::integral_constant<int, 0> zero;
        constexpr std::integral_constant<int, 1> one;
        if constexpr (Y == 0) {
            for (int st = 0; st < steps; ++st) step(st, zero);
        } else {
            int st = 0;
            for (; st + 1 < steps; st += 2) {
                step(st, zero);
                step(st + 1, one);
            }
            if (st < steps) {
                step(st, zero);
#pragma unroll
                for (int i = 0; i < X; ++i) fr[0][i] = fr[1][i];
            }
        }
        // Here `now` holds the next tile's first step (its first fragments are in
        // registers) and the other stage waits for its second.
        whole = tm0 + BM <= a.M && tn0 + BN <= a.N;
        if (whole)
            finish(std::true_type{}, tm0 + mrow, tn0 + ncol, tsplit);
        else
            finish(std::false_type{}, tm0 + mrow, tn0 + ncol, tsplit);
    }
    wait_loads<0>();  // nothing may still be on its way into LDS when the workgroup ends
}

// The splits' sums added in order, then bias and residual.  Bound: latency and the sums'
// bytes (7 x 3,072 x 768: 13 us, 66 MB read).
template <class T> __global__ __launch_bounds__(256) void grkan_product8_finish_kernel(Product8Args a) {
    const int quads = (a.N + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)quads * a.M) return;
    const int64_t m = i / quads, plane = (int64_t)a.M * a.N;
    const int n = (int)(i - m * quads) * 4, nv = min(a.N - n, 4);
    const float *p = a.partials + m * a.N + n;
    f32x4 h = {};
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s, p += plane) h += nv == 4 ? *reinterpret_cast<const f32x4_any *>(p) : load4<false>(p, nv);
    if (a.bias) h += load4<false>(a.bias + n, nv);
    if (a.residual) h += load4<false>(static_cast<const T *>(a.residual) + m * a.ldr + n, nv);
    store4<false>(static_cast<T *>(a.c) + m * a.N + n, nv, h);
}

// ------------------------------------------------------------ few rows

// Few rows of a, or a small result: a workgroup takes 16 columns of the result (16 rows of b) and
// 16 MT rows; its waves take the blocks of k in turn, straight from memory into
// operand registers, the loads of up to kTurns blocks on their way at once.  The
// waves' sums meet in LDS.  Bound: b's bytes, latency below (1 x 3,072 from 768: 3.3 us,
// the floor of a launch).
constexpr int kFewWaves = 8;

template <int MT, class T, bool CUT> __global__ __launch_bounds__(kFewWaves * 64) void grkan_product8_few_kernel(Product8Args a) {
    constexpr int kTurns = MT == 1 ? 4 : 2;
    __shared__ float red[kFewWaves][MT * 16][17];
    const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6;
    const int n0 = (int)blockIdx.x * 16, m0 = (int)blockIdx.y * 16 * MT;
    // rows past the end are the last once more (their results are not stored)
    const int kl = (lane >> 4) * 32, blocks = (a.K + kBlock8 - 1) / kBlock8;
    const uint8_t *pb = a.b.p + (int64_t)min(n0 + (lane & 15), a.N - 1) * a.b.ld + kl;
    const float *sb[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const int n = min(n0 + 4 * (lane >> 4) + v, a.N - 1);
        sb[v] = a.b.scale + (a.b_tile ? n / kBlock8 : n) * a.b.srow;
    }
    const uint8_t *pa[MT];
    const float *sa[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = min(m0 + 16 * i + (lane & 15), a.M - 1);
        pa[i] = a.a.p + m * a.a.ld + kl;
        sa[i] = a.a.scale + m * a.a.srow;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = f32x4{};
    auto turns = [&](int kb, auto count) {
        constexpr int U = count();
        u32x4 b[U][2], x[U][MT][2];
        f32x4 bs[U];
        float as[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = (int64_t)(kb + u * kFewWaves) * kBlock8;
            const int left = (int)min((int64_t)a.K - k - kl, (int64_t)32);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                b[u][h] = chunk16(pb + k + 16 * h, left - 16 * h);
#pragma unroll
                for (int i = 0; i < MT; ++i) x[u][i][h] = chunk16(pa[i] + k + 16 * h, left - 16 * h);
            }
            const int64_t at = kb + u * kFewWaves;
#pragma unroll
            for (int v = 0; v < 4; ++v) bs[u][v] = sb[v][at * a.b.sblock];
#pragma unroll
            for (int i = 0; i < MT; ++i) as[u][i] = sa[i][at * a.a.sblock];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            auto whole = [](const u32x4 (&c)[2]) {
                return i32x8{(int)c[0][0], (int)c[0][1], (int)c[0][2], (int)c[0][3], (int)c[1][0], (int)c[1][1], (int)c[1][2], (int)c[1][3]};
            };
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const f32x4 p = block_product<CUT>(whole(b[u]), whole(x[u][i]));
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[i][v] = fmaf(p[v], as[u][i] * bs[u][v], acc[i][v]);
            }
        }
    };
    int kb = wave;
    for (; kb + (kTurns - 1) * kFewWaves < blocks; kb += kTurns * kFewWaves) turns(kb, std::integral_constant<int, kTurns>{});
    for (; kb < blocks; kb += kFewWaves) turns(kb, std::integral_constant<int, 1>{});
    // lane: row lane mod 16, columns 4 (lane / 16) + v
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[wave][16 * i + (lane & 15)][4 * (lane >> 4) + v] = acc[i][v];
    __syncthreads();
    for (int q = t; q < MT * 256; q += kFewWaves * 64) {
        const int m = q >> 4, c = q & 15, n = n0 + c;
        if (m0 + m >= a.M || n >= a.N) continue;
        float h = 0.0f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) h += red[w][m][c];
        if (a.bias) h += a.bias[n];
        if (a.residual) h += load1(static_cast<const T *>(a.residual) + (int64_t)(m0 + m) * a.ldr + n);
        store1(static_cast<T *>(a.c) + (int64_t)(m0 + m) * a.N + n, h);
    }
}

// ------------------------------------------------------------ dispatch

template <int BM, int BN, class T, bool CUT, bool BTILE, bool PARTIAL> hipError_t launch_tile(const Product8Args &a, hipStream_t s) {
    auto kern = grkan_product8_tile_kernel<BM, BN, T, CUT, BTILE, PARTIAL>;
    using Shape = Tile8<BM, BN>;
    // Once on each device (twice if two threads come first: the same value).
    static uint64_t told = 0;
    int device = 0;
    hipError_t e = hipGetDevice(&device);
    if (e != hipSuccess) return e;
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (!(__atomic_load_n(&told, __ATOMIC_RELAXED) & bit)) {
        e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                (int)Shape::kLds);
        if (e != hipSuccess) return e;
        __atomic_fetch_or(&told, bit, __ATOMIC_RELAXED);
    }
    const int64_t mb = (a.M + BM - 1) / BM, nb = (a.N + BN - 1) / BN;
    int64_t grid = (mb * nb * (PARTIAL ? a.splits : 1) + 7) / 8 * 8;
    // as many workgroups as fit on the 256 CUs at once; each walks over its tiles
    constexpr int64_t resident = BN == 256 ? 256 : (BN == 128 ? 512 : 1024);
    if (grid > resident) grid = resident;
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(Shape::kThreads), Shape::kLds, s, a);
    return hipGetLastError();
}

template <int BM, int BN, class T, bool CUT> hipError_t launch_kind(const Product8Plan &p, const Product8Args &a, hipStream_t s) {
    if constexpr (BM == 256) {
        if (!a.b_tile) return hipErrorInvalidValue;  // (has no registers for a scale a column)
        return p.splits > 1 ? launch_tile<BM, BN, T, CUT, true, true>(a, s) : launch_tile<BM, BN, T, CUT, true, false>(a, s);
    } else if (p.splits > 1) {
        return a.b_tile ? launch_tile<BM, BN, T, CUT, true, true>(a, s) : launch_tile<BM, BN, T, CUT, false, true>(a, s);
    } else {
        return a.b_tile ? launch_tile<BM, BN, T, CUT, true, false>(a, s) : launch_tile<BM, BN, T, CUT, false, false>(a, s);
    }
}

template <class T, bool CUT> hipError_t launch_type(const Product8Plan &p, const Product8Args &a, hipStream_t s) {
    if (p.few > 0) {
        const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.M + 16 * p.few - 1) / (16 * p.few))), block(kFewWaves * 64);
        switch (p.few) {
            case 1: hipLaunchKernelGGL((grkan_product8_few_kernel<1, T, CUT>), grid, block, 0, s, a); break;
            case 2: hipLaunchKernelGGL((grkan_product8_few_kernel<2, T, CUT>), grid, block, 0, s, a); break;
            default: hipLaunchKernelGGL((grkan_product8_few_kernel<4, T, CUT>), grid, block, 0, s, a); break;
        }
        return hipGetLastError();
    }
    hipError_t e;
    if (p.tile == 256) {
        if constexpr (CUT)   // (has no registers for the wider products)
            e = launch_kind<256, 256, T, CUT>(p, a, s);
        else
            e = hipErrorInvalidValue;
    } else if (p.tile == 128) {
        e = launch_kind<128, 128, T, CUT>(p, a, s);
    } else {
        e = launch_kind<64, 64, T, CUT>(p, a, s);
    }
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t work = (int64_t)((a.N + 3) / 4) * a.M;
    hipLaunchKernelGGL((grkan_product8_finish_kernel<T>), dim3((unsigned)((work + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_product8(const Product8Plan &p, const Product8Args &args, hipStream_t s) {
    Product8Args a = args;
    a.M = (int32_t)p.rows;
    a.splits = p.splits;
    a.k_split = (int32_t)p.k_split;
    hipError_t e;
    if (!a.bf16)
        e = launch_type<float, false>(p, a, s);
    else
        e = a.cut ? launch_type<uint16_t, true>(p, a, s) : launch_type<uint16_t, false>(p, a, s);
    if (e != hipSuccess || p.rows == args.M) return e;
    const int64_t es = a.bf16 ? 2 : 4;
    a = args;
    a.M -= (int32_t)p.rows;
    a.a.p += p.rows * a.a.ld;
    a.a.scale += p.rows * a.a.srow;
    a.c = static_cast<char *>(a.c) + p.rows * a.N * es;
    if (a.residual) a.residual = static_cast<const char *>(a.residual) + p.rows * a.ldr * es;
    return launch_product8(plan_product8_whole(a.M, a.N, a.K, a.bf16, a.b_tile != 0, a.cut), a, s);
}

}  // namespace grkan
