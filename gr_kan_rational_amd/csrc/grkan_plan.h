// grkan_plan.h -- how the block operators' launches are laid out: plans of the
// group norm, the products and the slope pass from sizes, types and activation
// alone.  Host code without HIP; internal.
#pragma once

#include <limits.h>
#include <stddef.h>
#include <stdint.h>

#include "grkan_block.h"

namespace grkan {

inline size_t align256(size_t v) { return (v + 255) / 256 * 256; }

inline int io_bytes(grkan_dtype_t io) { return io == GRKAN_BF16 ? 2 : 4; }

inline bool act_valid(grkan_act_t act) {
    return act == GRKAN_ACT_NONE || act == GRKAN_ACT_SILU || act == GRKAN_ACT_GELU || act == GRKAN_ACT_RATIONAL;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline int pow2_at_most(int64_t v) {
    int p = 1;
    while (2 * (int64_t)p <= v) p *= 2;
    return p;
}

// Most workgroups of a launch whose kernel walks over what is left: a launch has
// to stay below 2^32 threads, 1,024 a workgroup.
constexpr int64_t kMaxBlocks = 1 << 20;

// ------------------------------------------------------------ norm plans

// How a (sample, group)'s positions x D values are covered.
//
//   kNormToken  positions = 1: T lanes (a power of two) hold a group's D
//               values, K accesses each; the reduction stays in a wave for
//               T <= 64.  Several groups ("slots") to a workgroup; each slot
//               keeps its columns and walks over the samples.
//   kNormSlab   a workgroup of TX x TY lanes holds a block of whole groups of
//               one sample in registers, `regs` rows to a lane: the tensor is
//               read once.
//   kNormSplit  a group that fits in no workgroup: a pass over row chunks that
//               leaves sums, a small kernel that adds them, a second pass that
//               applies them.
//
// A lane's access is `vec` elements, 16 bytes but for a rational whose groups
// would put two sets of coefficients into one (then the largest power of two
// that does not).  Slab and split cover a block of `width` columns with
// accesses side by side whatever the groups; `mixed` says that an access may
// straddle groups (vec does not divide D), which then takes statistics per
// element.  Token accesses start at their group's first column, the last one
// ragged.  A lane keeps its columns, so weight, bias and the rational's
// coefficients are read once and column sums stay in registers.
enum NormKind : int32_t { kNormToken = 0, kNormSlab = 1, kNormSplit = 2 };

struct NormPlan {
    int32_t kind;
    int32_t vec;
    bool mixed;
    bool straddle;           // token, rational: a lane's columns may lie in two activation groups
    int32_t T, K, spw;       // token: lanes per slot, accesses per lane, slots per workgroup
    int32_t vpg;             // token: lanes of a slot that hold columns
    int32_t width, ncb;      // slab, split: columns per block, blocks
    int32_t TX, TY;          // slab, split: accesses across, rows per pass
    int32_t groups;          // slab, split: most groups in a block
    int32_t parts;           // split: most blocks a group lies in
    int32_t regs;            // slab: rows per lane
    int32_t P, L;            // slab, split: lanes that add up one column's rows, one group's columns
    bool fused;              // split: the second pass adds the first's sums itself
    int32_t block;           // threads per workgroup
    int64_t blocks;          // workgroups
    int64_t chunks, chunk_rows;  // split: row chunks per sample; slab backward: chunks of samples
    int64_t cv;              // lanes that hold columns, over all groups or blocks
    int64_t prows, row;      // column partials (backward): rows, and floats per row
    size_t lds;
    size_t off_stats, off_means, off_partials, total;  // workspace
};

constexpr size_t kMaxLds = 160 << 10;  // of a CU
constexpr int kTokenMaxLanes = 256, kTokenMaxAccesses = 4;
constexpr int64_t kNormWorkgroups = 2048;  // target of the looping kernels: 8 workgroups a CU

// Largest power of two <= v elements per access such that accesses that start
// at multiples of `start` columns (and then every v) lie in one activation
// group each.
inline int rational_vec(int v, int64_t dga, int64_t start) {
    while (v > 1 && (dga % v != 0 || start % v != 0)) v /= 2;
    return v;
}

inline grkan_status_t norm_plan(int64_t N, int64_t S, int64_t C, int32_t G, int32_t ng, grkan_act_t act, grkan_dtype_t io,
                         bool backward, NormPlan *p) {
    if (io != GRKAN_F32 && io != GRKAN_BF16) return GRKAN_ERR_INVALID_ARG;
    if (!act_valid(act)) return GRKAN_ERR_INVALID_ARG;
    const bool rational = act == GRKAN_ACT_RATIONAL;
    if (N < 0 || S < 0 || C < 1 || G < 1 || C % G != 0) return GRKAN_ERR_INVALID_ARG;
    if (rational && (ng < 1 || C % ng != 0)) return GRKAN_ERR_INVALID_ARG;
    if (C >= (1 << 24) || S > INT32_MAX) return GRKAN_ERR_UNSUPPORTED;
    if (N > INT32_MAX / G) return GRKAN_ERR_UNSUPPORTED;
    const int es = io_bytes(io), vmax = 16 / es;
    const int64_t D = C / G, dga = rational ? C / ng : 0;
    *p = NormPlan{};
    if (N == 0 || S == 0) return GRKAN_OK;

    // Token: T lanes of K accesses of v elements with the fewest idle places for
    // a group, then the widest accesses (16 bytes or 8), then the fewest.  The
    // backward keeps two sums, a weight and a bias per element of a lane, so it
    // takes at most 16 (768 channels in bf16: 64 lanes x 3 x 4).  A rational's
    // lanes prefer runs inside one activation group; else a run may lie in two,
    // and has to be no longer than a group for that.
    int64_t best = INT64_MAX;
    if (S == 1) {
        for (int straddle = 0; straddle <= (rational ? 1 : 0) && best == INT64_MAX; ++straddle)
            for (int v = vmax; v >= 1; v /= 2) {
                if (!rational && v < vmax / 2) break;
                for (int K = 1; K <= kTokenMaxAccesses; ++K) {
                    const int run = K * v;
                    if (backward && run > 16) break;
                    // (the forward has coefficients per access, the backward per run)
                    const int unit = backward ? run : v;
                    if (rational && !straddle && dga % D != 0 && (dga % unit != 0 || D % unit != 0)) continue;
                    if (straddle && (run > dga || run < 4)) continue;
                    int T = 1;
                    while ((int64_t)T * run < D) T *= 2;
                    if (T > (run == 1 ? 1024 : kTokenMaxLanes) || (int64_t)T * run >= best) continue;
                    best = (int64_t)T * run;
                    p->vec = v;
                    p->T = T;
                    p->K = K;
                    p->straddle = straddle != 0;
                }
            }
    }
    if (best != INT64_MAX) {
        p->kind = kNormToken;
        p->vpg = (int32_t)ceil_div(D, p->K * p->vec);  // (read for a rational only)
        p->cv = (int64_t)G * p->vpg;
        int spw = p->T <= 64 ? 256 / p->T : 1;
        while (spw % G != 0 && G % spw != 0) --spw;
        p->spw = spw;
        p->block = spw * p->T;
        // Enough workgroups to fill the GPU, walking over the samples in as
        // many rounds each as the last of them needs.
        const int64_t unit = spw < G ? G / spw : 1;  // workgroups that cover one sample
        const int64_t wanted = ceil_div(N * G, spw), cap = backward ? kNormWorkgroups / 2 : kNormWorkgroups;
        const int64_t rounds = ceil_div(wanted, cap);
        p->blocks = ceil_div(ceil_div(wanted, rounds), unit) * unit;
        p->prows = spw > G ? p->blocks : p->blocks * spw / G;
        p->lds = (size_t)p->block * ((rational ? 10 : p->vec) + 3) * 4 + 256;
    } else {
        // A slab: whole groups side by side until they make 64 bytes or more of
        // every row, if a workgroup's registers hold all rows of that.
        const int threads = backward ? 512 : 1024, regs = backward ? 8 : 16;
        int64_t gpb = ceil_div(64, D * es);
        if (gpb > G) gpb = G;
        auto vec_of = [&](int64_t groups) { return rational ? rational_vec(vmax, dga, groups * D) : vmax; };
        auto rows_of = [&](int64_t groups) {  // rows a workgroup can hold
            const int64_t tx = ceil_div(groups * D, vec_of(groups));
            return tx <= threads ? threads / tx * regs : 0;
        };
        // LDS of the groups' sums (group_sum): every lane's and column's, and the groups'
        auto lds_of = [&](bool mixed) {
            const size_t value = p->kind == kNormSplit ? sizeof(double) : sizeof(float);
            const size_t values = p->kind == kNormSlab && !backward ? 1 : 2;
            return value * values * ((size_t)(p->block + p->TX) * (mixed ? p->vec : 1) + p->groups);
        };
        if (S > 1 && S <= rows_of(gpb)) {
            p->kind = kNormSlab;
            // wider blocks while many workgroups remain and rows are short
            while (gpb * 2 <= G && gpb * D * es < 256 && S <= rows_of(gpb * 2) && vec_of(gpb * 2) >= vec_of(gpb) &&
                   N * ceil_div(G, gpb * 2) >= kNormWorkgroups)
                gpb *= 2;
            p->vec = vec_of(gpb);
            p->width = (int32_t)(gpb * D);
            p->ncb = (int32_t)ceil_div(G, gpb);
            p->groups = (int32_t)gpb;
            p->TX = (int32_t)ceil_div(p->width, p->vec);
            // Row lanes: 256 threads if many workgroups share a CU, all there are
            // if not; at least what the registers need.  The backward walks over the
            // samples, the next one's values on their way: two workgroups of 256
            // threads a CU (128 x 197 x 192 in 8 groups, fp32: 28.5 us; one of 512: 30.7;
            // 64 x 256 x 512 in 32: 38.7, 46.4), one of 512 for 8 rounds or more of
            // wide rows (1,024 x 197 x 192: 132 us against 183; 256 x 197 x 768, bf16: 116
            // against 200).
            const bool long_walk = backward && N * p->ncb >= 2048 && gpb * D * es >= 96;
            const int64_t want = N * p->ncb >= 1024 && !long_walk ? 256 : threads;
            int64_t ty = want / p->TX;
            if (ty < ceil_div(S, regs)) ty = ceil_div(S, regs);
            if (ty > S) ty = S;
            p->regs = (int32_t)ceil_div(S, ty);
            p->TY = (int32_t)ceil_div(S, p->regs);
            p->block = (int32_t)(ceil_div((int64_t)p->TX * p->TY, 64) * 64);
            if (!backward) {
                p->blocks = (N >= 8 ? ceil_div(N, 8) * 8 : N) * p->ncb;
            } else {
                int64_t chunks = (long_walk ? 256 : 512) / p->ncb;
                if (chunks < 1) chunks = 1;
                if (chunks > N) chunks = N;
                if (chunks >= 8) chunks = chunks / 8 * 8;
                p->chunks = chunks;
                p->blocks = chunks * p->ncb;
                p->prows = chunks;
            }
        } else {
            p->kind = kNormSplit;
            p->vec = rational ? rational_vec(vmax, dga, 0) : vmax;
            const int64_t accesses = ceil_div(C, p->vec);
            // At most 256 accesses across (128 where every column is a group, for the
            // groups' sums in LDS).
            p->ncb = (int32_t)ceil_div(accesses, D == 1 ? 128 : 256);
            p->TX = (int32_t)ceil_div(accesses, p->ncb);
            p->width = p->TX * p->vec;
            p->ncb = (int32_t)ceil_div(C, p->width);
            p->groups = (int32_t)(p->width / D + 2 < G ? p->width / D + 2 : G);
            p->parts = (int32_t)(D / p->width + 2 < p->ncb ? D / p->width + 2 : p->ncb);
            // Chunks of 4 to 32 rows a lane, about a workgroup a CU; where those
            // leave a lane of the second pass more than 2 sums to add (few
            // samples), smaller workgroups, more of them, and a step between that
            // adds (65,536 x 128 in 32 groups: 26 us against 29).
            auto chunks_of = [&](int64_t lanes, int64_t wanted) {
                int64_t ty = lanes / p->TX;
                if (ty > S) ty = S;
                p->TY = (int32_t)ty;
                p->block = (int32_t)(ceil_div((int64_t)p->TX * ty, 64) * 64);
                int64_t chunks = ceil_div(wanted, N * p->ncb);
                const int64_t most = ceil_div(S, 4 * ty), least = ceil_div(S, 32 * ty);
                if (chunks > most) chunks = most;
                if (chunks < least) chunks = least;
                p->chunk_rows = ceil_div(S, chunks);
                p->chunks = ceil_div(S, p->chunk_rows);
                p->L = pow2_at_most(p->block / p->groups < 64 ? (p->block > p->groups ? p->block / p->groups : 1) : 64);
                p->fused = ceil_div(p->chunks * p->parts, p->L) <= 2;
            };
            if (backward) {
                chunks_of(512, 512);
            } else {
                chunks_of(1024, 256);
                // (1,024 lanes' fp64 sums of 8 elements each, where accesses straddle
                // groups, may pass what a CU has: half the lanes then.  2 x 1,024 x
                // 2,044 in 4 groups 23.7 us, with 256 lanes and the step between 26.6;
                // 64 x 197 x 2,046 in one 86, 82)
                if (p->fused && lds_of(D % p->vec != 0) > kMaxLds) chunks_of(512, 256);
                if (!p->fused) chunks_of(256, 1024);
            }
            p->blocks = N * p->chunks * p->ncb;
            p->prows = N * p->chunks;
        }
        p->cv = (int64_t)p->ncb * p->TX;
        p->mixed = D % p->vec != 0;
        p->L = pow2_at_most(p->block / p->groups < 64 ? (p->block > p->groups ? p->block / p->groups : 1) : 64);
        const int64_t cols_across = (int64_t)p->TX * (p->mixed ? p->vec : 1);
        p->P = pow2_at_most(p->block / cols_across < 1 ? 1 : (p->block / cols_across < 64 ? p->block / cols_across : 64));
        p->lds = lds_of(p->mixed);
        const size_t cols = (size_t)p->block * ((rational ? 10 : p->vec) + 3) * 4;
        if (backward && p->lds < cols) p->lds = cols;
    }
    p->row = 2 * C + (rational ? (p->straddle ? 20 : 10) * p->cv : 0);
    size_t at = 0;
    if (p->kind == kNormSplit) {
        p->off_stats = at;
        at += align256((size_t)N * G * p->chunks * p->parts * 16);
        p->off_means = at;
        if (backward) at += align256((size_t)N * G * 8);
    }
    p->off_partials = at;
    if (backward) at += align256((size_t)p->prows * p->row * 4);
    p->total = at;
    return GRKAN_OK;
}

// ------------------------------------------------------------ products

// Ways to multiply.
//   kTile     tiles of the result in registers, operands through LDS; with
//             splits > 1 (or an epilogue the tile kernel lacks) fp32 sums go
//             to memory and a second kernel adds them and applies the epilogue
//   kSkinny   few rows: 16 columns of the result a workgroup, its waves share
//             the k range, the weights go from memory straight to registers
enum ProductKind : int32_t { kTile = 0, kSkinny = 1 };

struct ProductPlan {
    int32_t kind;
    int32_t tile;            // kTile: index of the tile shape
    int32_t rest_tile;       // kTile: shape of the rows from `rows` on, when rows > 0
    int64_t rows;
    int32_t mt;              // kSkinny: 16-row blocks per workgroup
    int32_t splits, k_split;
    bool two_steps;          // partials, then grkan_linear_finish
    bool aligned;            // 16-byte chunks of both operands are aligned and whole
    size_t partials_bytes;
};

// The layouts of the three products.
enum ProductForm : int32_t {
    kFormForward = 0,   // Q = x [M][K], P = W [N][K]
    kFormDx = 1,        // Q = dpre [M][K], P = W [K][N]
    kFormDw = 2         // Q = dpre [K][M], P = x [K][N]
};

// Rows up to which the skinny kernel is taken (128 x 3,072 from 768: 9.4 us against
// 8.9 with tiles; 64: 6.9 against 8.7).
constexpr int64_t kSkinnyRows = 64;

constexpr int kTileM[] = {256, 128, 64}, kTileN[] = {256, 128, 64}, kTileK[] = {64, 32, 64};

// Whether a kernel exists for the plan: the 256-row tile takes aligned operands
// only, and what is cut into whole rounds of it and a rest runs the aligned
// kernels throughout.
inline bool plan_has_kernel(const ProductPlan &p) {
    return p.kind == kSkinny || p.aligned || (p.tile != 0 && p.rows == 0);
}

inline ProductPlan plan_product(int form, int64_t M, int64_t N, int64_t K, bool aligned, int32_t act, int64_t dga) {
    ProductPlan p{};
    p.aligned = aligned;
    p.splits = 1;
    p.k_split = (int32_t)(K > 0 ? K : 1);
    const bool any_groups = act == GRKAN_ACT_RATIONAL && dga % 8 != 0;
    if (form == kFormForward && M <= kSkinnyRows) {
        p.kind = kSkinny;
        // as many rows a workgroup as there are, while 192 workgroups remain (64 x
        // 768 from 3,072: 9.1, 10.6, 15.9 us with 1, 2, 4 blocks of 16 rows; 64 x 3,072
        // from 768: 8.6, 6.9, 6.9)
        p.mt = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
        while (p.mt > 1 && (N + 15) / 16 * ((M + 16 * p.mt - 1) / (16 * p.mt)) < 192) p.mt /= 2;
        return p;
    }
    // The tile and the number of k splits with the least estimated time.  Places
    // are the workgroups that the CUs hold at once; a step takes a workgroup
    // `alone` us while few are taken, in proportion to those that are up to
    // `full`, and a tile's result `tail` (M x N from K, rows of tiles 256 / 128 / 64,
    // us: 1,003 x 768 from 768 25 / 14.8 / 7.8; 4,096 x 768 from 3,072 66 / 42 / 34;
    // 4,096 x 3,072 from 768 29 / 32 / 40; 4,096 x 4,096 from 4,096 115 / 183 / 273;
    // 50,432 x 3,072 from 768 324 / 365 / 470).  Splits add a launch, a write and a
    // read of their fp32 sums (768 x 768 from 50,432 in tiles of 256 rows: 158, 88,
    // 75 us with 7, 16, 24; of 1,003 rows from 768 in tiles of 64: 7.8, 15 us with 1
    // and 2).  The operands reach the XCDs at about 10 TB/s, once or to each of
    // the 8 as the tiles' order has it (768 x 192 from 25,216: 33 us in 7 splits,
    // all of both to each; 25 us in 16, each k range to one).  No sum of a tile
    // runs over more than 16,384 values of k in fp32 (the few-row kernel's run over
    // an eighth of K each, whatever it is).
    static const double kAlone[] = {1.5, 0.4, 0.33}, kFull[] = {1.65, 1.2, 0.75}, kTail[] = {7.0, 2.0, 0.5};
    static const int64_t kPlaces[] = {256, 768, 768};
    auto tiles_us = [&](int i, int64_t wgs, int64_t steps) {
        const int64_t rounds = wgs / kPlaces[i], rest = wgs % kPlaces[i];
        const double part = kFull[i] * (double)rest / (double)kPlaces[i];
        double us = (double)rounds * (steps * kFull[i] + kTail[i]);
        if (rest) us += steps * (part > kAlone[i] ? part : kAlone[i]) + kTail[i];
        return us;
    };
    // (unaligned chunks are on their way in registers: a tile of 256 x 128 spilled,
    // 574 us against 75 with 128 x 128 at 8,003 x 1,501 from 777)
    const int first = aligned ? 0 : 1;
    double best = 1e30;
    p.kind = kTile;
    for (int i = first; i < 3; ++i) {
        const int64_t mt = (M + kTileM[i] - 1) / kTileM[i], nt = (N + kTileN[i] - 1) / kTileN[i], tiles = mt * nt;
        const int64_t steps = (K + kTileK[i] - 1) / kTileK[i], least = (K + 16383) / 16384;
        for (int64_t s = least < 1 ? 1 : least; s <= 64 || s == least; ++s) {
            if (s > 8 && s % 8 != 0 && s != least) continue;  // eighths: a k range to an XCD
            if (s > 1 && s > least && (steps < 4 * s || (double)s * M * N * 4 > 256e6)) break;
            const int64_t per = (steps + s - 1) / s;
            const double times = s % 8 == 0 ? 1 : 8.0 / (double)(s < 8 ? s : 8);
            const double fetch = 2.0 * (double)K * ((double)M + times * (double)N) / 10e6, work = tiles_us(i, tiles * s, per);
            double us = 3.0 + (work > fetch ? work : fetch);
            if (s > 1) us += 3.0 + 2.0 * (double)s * M * N * 4 / 6e6;
            if (us < best) {
                best = us;
                p.tile = i;
                p.rows = 0;
                p.k_split = (int32_t)(per * kTileK[i] < K ? per * kTileK[i] : (K > 0 ? K : 1));
            }
            // Rows that fill whole rounds of 256-row tiles, the rest in smaller ones
            // (50,432 x 768 from 3,072: 312 us whole, 198 + 57 us so)
            if (i == 0 && s == 1 && form != kFormDw && !any_groups) {
                const int64_t panels = tiles / kPlaces[0] * kPlaces[0] / nt, rows = panels * kTileM[0], left = M - rows;
                if (rows <= 0 || left <= 0) continue;
                for (int j = 1; j < 3; ++j) {
                    const int64_t rest = ((left + kTileM[j] - 1) / kTileM[j]) * ((N + kTileN[j] - 1) / kTileN[j]);
                    const double both = 6.0 + tiles_us(0, panels * nt, steps) + tiles_us(j, rest, (K + kTileK[j] - 1) / kTileK[j]);
                    if (both < best) {
                        best = both;
                        p.tile = 0;
                        p.k_split = (int32_t)K;
                        p.rows = rows;
                        p.rest_tile = j;
                    }
                }
            }
        }
    }
    p.splits = (int32_t)((K + p.k_split - 1) / p.k_split);
    if (p.splits < 1) p.splits = 1;
    p.two_steps = p.splits > 1 || any_groups;
    if (p.two_steps) p.partials_bytes = (size_t)p.splits * (size_t)M * (size_t)N * 4;
    return p;
}

// ------------------------------------------------------------ dpre, dbias

constexpr int kSlopeTx = 32, kSlopeTy = 8;
constexpr int64_t kSlopeBlocks = 1536;  // workgroups, 6 a CU

struct SlopePlan {
    int32_t vec, vpr, chunks;
    int64_t chunk_rows;
    size_t partials_bytes;
};

inline SlopePlan plan_slope(int64_t rows, int64_t N, int32_t act, int64_t dga) {
    SlopePlan p{};
    const bool rational = act == GRKAN_ACT_RATIONAL;
    p.vec = rational && dga % 8 != 0 ? 1 : 8;
    p.vpr = (int32_t)((N + p.vec - 1) / p.vec);
    const int64_t blocks = (p.vpr + kSlopeTx - 1) / kSlopeTx;
    int64_t chunks = (kSlopeBlocks + blocks - 1) / blocks;
    const int64_t most = (rows + 4 * kSlopeTy - 1) / (4 * kSlopeTy);
    if (chunks > most) chunks = most;
    if (chunks < 1) chunks = 1;
    p.chunk_rows = (rows + chunks - 1) / chunks;
    if (p.chunk_rows < 1) p.chunk_rows = 1;
    p.chunks = (int32_t)((rows + p.chunk_rows - 1) / p.chunk_rows);
    p.partials_bytes = (size_t)p.chunks * (size_t)(N + (rational ? 10 * (int64_t)p.vpr : 0)) * 4;
    return p;
}

// ------------------------------------------------------------ linear map

constexpr int64_t kMaxWidth = int64_t(1) << 22;
constexpr int64_t kMaxRows = INT32_MAX - 256;  // the tiles' row numbers, to the end of the last 256, are 32-bit

inline grkan_status_t linear_shape(int64_t rows, int64_t d_in, int64_t d_out, int32_t n_groups, grkan_act_t act) {
    if (!act_valid(act) || rows < 0 || d_in < 1 || d_out < 1) return GRKAN_ERR_INVALID_ARG;
    if (act == GRKAN_ACT_RATIONAL && (n_groups < 1 || d_out % n_groups != 0)) return GRKAN_ERR_INVALID_ARG;
    if (rows > kMaxRows || d_in > kMaxWidth || d_out > kMaxWidth) return GRKAN_ERR_UNSUPPORTED;
    // one thread per 8 elements of a result, in workgroups of 256, one launch
    const int64_t most = (int64_t(1) << 32) - 256;
    if (rows * ceil_div(d_out, 8) >= most || rows * ceil_div(d_in, 8) >= most || d_out * ceil_div(d_in, 8) >= most)
        return GRKAN_ERR_UNSUPPORTED;
    return GRKAN_OK;
}

inline int64_t act_group(int64_t d_out, int32_t n_groups, grkan_act_t act) {
    return act == GRKAN_ACT_RATIONAL ? d_out / n_groups : 8;
}

// Workspace of the forward that is enough whatever its operands' alignment (the
// unaligned plan may have more k splits).
inline size_t linear_fwd_bytes(int64_t rows, int64_t d_in, int64_t d_out, int32_t n_groups, grkan_act_t act) {
    size_t most = 0;
    for (int al = 0; al < 2; ++al) {
        const ProductPlan p = plan_product(kFormForward, rows, d_out, d_in, al != 0, act, act_group(d_out, n_groups, act));
        if (p.partials_bytes > most) most = p.partials_bytes;
    }
    return align256(most);
}

// The products are planned for the alignment that their operands have: the
// 256-row tile, alone or with the other rows in smaller ones, exists for
// aligned operands alone.
struct LinearBwdPlan {
    SlopePlan slope;
    ProductPlan dx, dw;
    size_t off_slope, off_sums, total;
};

inline void linear_bwd_plan(int64_t rows, int64_t d_in, int64_t d_out, int32_t n_groups, grkan_act_t act,
                            bool dx_aligned, bool dw_aligned, LinearBwdPlan *p) {
    p->slope = plan_slope(rows, d_out, act, act_group(d_out, n_groups, act));
    p->dx = plan_product(kFormDx, rows, d_in, d_out, dx_aligned, GRKAN_ACT_NONE, 8);
    p->dw = plan_product(kFormDw, d_out, d_in, rows, dw_aligned, GRKAN_ACT_NONE, 8);
    p->off_slope = act == GRKAN_ACT_NONE ? 0 : align256((size_t)rows * d_out * 2);
    p->off_sums = p->off_slope + align256(p->slope.partials_bytes);
    const size_t sums = p->dx.partials_bytes > p->dw.partials_bytes ? p->dx.partials_bytes : p->dw.partials_bytes;
    p->total = p->off_sums + align256(sums);
}

// Workspace that is enough whatever the operands' alignment.
inline size_t linear_bwd_bytes(int64_t rows, int64_t d_in, int64_t d_out, int32_t n_groups, grkan_act_t act) {
    size_t most = 0;
    for (int al = 0; al < 4; ++al) {
        LinearBwdPlan p;
        linear_bwd_plan(rows, d_in, d_out, n_groups, act, (al & 1) != 0, (al & 2) != 0, &p);
        if (p.total > most) most = p.total;
    }
    return most;
}

}  // namespace grkan
