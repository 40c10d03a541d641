// grkan_train_plan.h -- how the launches of the operators of grkan_train.h are
// laid out: plans from sizes and types alone.  Host code without HIP; internal.
#pragma once

#include "grkan_plan.h"
#include "grkan_train.h"

namespace grkan {

constexpr int kBlock8 = 128;  // values that share a scale

// ------------------------------------------------------------ quantiser

// Rows of a workgroup that takes rows alone (the others take 128), 128 columns each, 256 threads.
constexpr int kQuantizeRows = 64;

inline grkan_status_t quantize_shape(int64_t rows, int64_t cols, int64_t ldx, int32_t n_groups, grkan_act_t act,
                                     grkan_dtype_t io) {
    if (io != GRKAN_F32 && io != GRKAN_BF16) return GRKAN_ERR_INVALID_ARG;
    if (act != GRKAN_ACT_NONE && act != GRKAN_ACT_RATIONAL) return GRKAN_ERR_INVALID_ARG;
    if (rows < 0 || cols < 1 || ldx < cols) return GRKAN_ERR_INVALID_ARG;
    if (act == GRKAN_ACT_RATIONAL && (n_groups < 1 || cols % n_groups != 0)) return GRKAN_ERR_INVALID_ARG;
    if (rows > kMaxRows || cols > kMaxWidth || ldx > kMaxWidth) return GRKAN_ERR_UNSUPPORTED;
    // one launch, below 2^32 threads
    if (ceil_div(rows, kQuantizeRows) * ceil_div(cols, kBlock8) >= (int64_t(1) << 24)) return GRKAN_ERR_UNSUPPORTED;
    return GRKAN_OK;
}

// ------------------------------------------------------------ 8-bit product

// A scale's row stride: a tile's scales lie within 2^31 bytes.
constexpr int64_t kMaxScaleRow = int64_t(1) << 20;

// Few rows, or a small result: `few` blocks of 16 rows a workgroup.  Else tiles of the result of `tile` x
// `tile`; with splits > 1 fp32 sums of k ranges go to memory and a second kernel
// adds them.  The rows past the first `rows` follow by a plan of their own.
struct Product8Plan {
    int64_t rows;
    int32_t few;
    int32_t tile;
    int32_t splits;
    int64_t k_split;         // of a split, whole blocks
    size_t partials_bytes;
};

inline grkan_status_t product8_shape(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 1 || K < 1) return GRKAN_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxWidth || K > kMaxWidth) return GRKAN_ERR_UNSUPPORTED;
    // the second kernel's threads, 4 columns each, in one launch
    if (M * ceil_div(N, 4) >= (int64_t(1) << 32) - 256) return GRKAN_ERR_UNSUPPORTED;
    return GRKAN_OK;
}

constexpr int64_t kFewRows = 64;

// A CU holds 1, 2 or 4 workgroups of these tiles; a step (a block of k) takes a workgroup
// `alone` us, or `full` where the CU holds as many as it can, a tile's result `tail`,
// `tail_full`; by how blocks are summed, in fp32 first.
constexpr int kTiles8[] = {256, 128, 64};
constexpr double kTimes8[2][3][4] = {{{}, {0.9, 2.1, 2.2, 0.0}, {0.61, 1.5, 0.23, 0.0}},
                                     {{1.6, 1.7, 3.0, 5.5}, {0.5, 1.3, 2.0, 2.3}, {0.38, 1.0, 0.4, 1.9}}};
constexpr double kLaunch8 = 3.5;

// One plan for all rows, and its estimated time.
inline Product8Plan plan_product8_whole(int64_t M, int64_t N, int64_t K, bool bf16, bool b_tile, bool cut = false,
                                        double *time = nullptr) {
    cut = cut && bf16;   // (fp32 results have fp32 sums)
    Product8Plan p{};
    p.rows = M;
    p.splits = 1;
    p.k_split = ceil_div(K, kBlock8) * kBlock8;
    if (M <= kFewRows) {
        p.few = M <= 16 ? 1 : (M <= 32 ? 2 : 4);
        while (p.few > 1 && ceil_div(N, 16) * ceil_div(M, 16 * p.few) < 192) p.few /= 2;
        return p;
    }
    // The tile and the number of k splits with the least estimated time.  Splits add a
    // launch, a write and a read of their sums.  Fitted to 603 timings of
    // 58 shapes: the choice is 1.3% from the best one in the mean, 19% at most, of bf16
    // results with fp32 sums, planned as fp32 ones, 2.0% and 24%
    // (cut sums, 50,432 x 3,072 from 768, tiles of 256 / 128 / 64: 185 / 182 / 240 us; 8,192 x
    // 8,192 from 8,192: 537 / 656 / 1,260; 197 x 768 from 3,072 in tiles of 64: 9.7 us
    // in 4 splits, 20 in one).  256 x 256 is for sums by the 8-bit instruction and a
    // scale for each tile of b alone: it has no registers for the wider products or a scale a column.
    const int64_t steps = ceil_div(K, kBlock8), cus = 256;
    double best = 1e30;
    for (int i = cut && b_tile ? 0 : 1; i < 3; ++i) {
        const double *t = kTimes8[cut][i];
        const int64_t tiles = ceil_div(M, kTiles8[i]) * ceil_div(N, kTiles8[i]), held = 1 << i;
        for (int64_t s = 1; s <= 64; ++s) {
            if (s > 8 && s % 8 != 0) continue;  // eighths: a k range to an XCD
            if (s > 1 && (steps < 2 * s || (double)s * M * N * 4 > 256e6)) break;
            const int64_t per = ceil_div(steps, s), wgs = tiles * ceil_div(steps, per);
            const int64_t rounds = wgs / (held * cus), rest = wgs % (held * cus);
            const double share = (double)ceil_div(rest, cus) / (double)held;
            double us = kLaunch8 + (double)rounds * (per * t[1] + t[3]);
            if (rest) {
                us += per * (t[1] * share > t[0] ? t[1] * share : t[0]);
                us += t[3] * share > t[2] ? t[3] * share : t[2];
            }
            if (s > 1) us += 3.2 + 2.0 * (double)s * M * N * 4 / 7e6;
            if (us < best) {
                best = us;
                p.tile = kTiles8[i];
                p.k_split = per * kBlock8;
            }
        }
    }
    // The kernel of few rows, as long as a CU has one workgroup, with the fewest rows for
    // which that is so (cut sums, 160 x 768 from 3,072 7.2 us, in tiles 9.7; 256 x 512 from 2,048 5.5
    // and 9.3; 197 x 768 from 3,072 10.4 and 9.7).
    static const double kFewTimes[3][2] = {{2.6, 0.105}, {2.8, 0.185}, {3.0, 0.31}};
    for (int i = 0; i < 3; ++i) {
        if (ceil_div(N, 16) * ceil_div(M, 16 << i) > cus) continue;
        const double us = kFewTimes[i][0] + kFewTimes[i][1] * (double)steps;
        if (us < best) {
            best = us;
            p.few = 1 << i;
            p.tile = 0;
            p.k_split = steps * kBlock8;
        }
        break;
    }
    p.splits = p.few > 0 ? 1 : (int32_t)ceil_div(K, p.k_split);
    if (p.splits > 1) p.partials_bytes = (size_t)p.splits * (size_t)M * (size_t)N * 4;
    if (time) *time = best;
    return p;
}

// Tiles of 256 x 256 for as many rows as keep all CUs at work, the others by a plan of their
// own, if that takes less: a last round of few such tiles takes as long as a full one
// (50,432 x 768 from 3,072: 138 us whole, 141 in tiles of 128, 127 so; 15,443 x 2,112
// from 3,648: 160, 151 and 141; 50,432 x 3,072 from 768: 156, 165 and 154).
inline Product8Plan plan_product8(int64_t M, int64_t N, int64_t K, bool bf16, bool b_tile, bool cut = false) {
    if (M <= kFewRows || !bf16 || !cut || !b_tile) return plan_product8_whole(M, N, K, bf16, b_tile, cut);
    double whole, rest;
    Product8Plan p = plan_product8_whole(M, N, K, bf16, b_tile, true, &whole);
    const int64_t nb = ceil_div(N, kTiles8[0]), rounds = ceil_div(M, kTiles8[0]) * nb / 256;
    const int64_t rows = rounds * 256 / nb * kTiles8[0];
    if (rows < 1 || M - rows <= kFewRows) return p;
    const Product8Plan r = plan_product8_whole(M - rows, N, K, bf16, b_tile, true, &rest);
    const double *t = kTimes8[1][0];
    if (kLaunch8 + (double)rounds * (ceil_div(K, kBlock8) * t[1] + t[3]) + rest >= whole) return p;
    p.rows = rows;
    p.few = 0;
    p.tile = kTiles8[0];
    p.splits = 1;
    p.k_split = ceil_div(K, kBlock8) * kBlock8;
    p.partials_bytes = r.partials_bytes;
    return p;
}

// Workspace for every kind of sums and layout of scales (bf16 results with fp32 sums take fp32's plan).
inline size_t product8_bytes(int64_t M, int64_t N, int64_t K) {
    size_t most = 0;
    for (int i = 0; i < 4; ++i) {
        const size_t n = plan_product8(M, N, K, true, (i & 2) != 0, (i & 1) != 0).partials_bytes;
        if (n > most) most = n;
    }
    return align256(most);
}

// ------------------------------------------------------------ residual path

constexpr int64_t kMaxChannels = 16384;
constexpr int64_t kMaxStride = int64_t(1) << 31;

// A row is held by `waves` waves, 4 K values a lane.  The walkers (waves, or workgroups of
// `waves` > 1) each take `walk` rows one after another.
struct ResidualPlan {
    int32_t K, waves;
    int32_t per;             // rows that a workgroup holds at a time
    int64_t blocks;
    int64_t walk;
    int32_t sums;            // column sums that a workgroup leaves
    size_t off_sums, off_gate, total;
};

inline grkan_status_t residual_shape(int64_t rows, int64_t C, int64_t gates, int64_t gate_channels, grkan_dtype_t io) {
    if (io != GRKAN_F32 && io != GRKAN_BF16) return GRKAN_ERR_INVALID_ARG;
    if (rows < 0 || C < 1 || gates < 0) return GRKAN_ERR_INVALID_ARG;
    if (gates > 0 && (rows % gates != 0 || (gate_channels != 1 && gate_channels != C))) return GRKAN_ERR_INVALID_ARG;
    if (C > kMaxChannels || rows > INT32_MAX || gates > INT32_MAX) return GRKAN_ERR_UNSUPPORTED;
    return GRKAN_OK;
}

inline void residual_plan(int64_t rows, int64_t C, int64_t gates, int64_t gate_channels, grkan_norm_t post,
                          bool backward, ResidualPlan *p) {
    *p = ResidualPlan{};
    const int64_t quads = ceil_div(C, 4);
    // A wave holds up to 256 accesses of a row, 8 waves as many each, else 192, whatever the
    // type.  With a post norm's sums and a gate's for each channel in the backward a wave
    // alone takes 192 too (37,824 rows of 1,024 channels: 135 us, 232 with 256); 8 waves do not
    // (4,728 rows of 8,192: 380 us, spilled, against 531 in 16 waves of half the registers).
    // The backward's bf16 rows then fit 256 registers up to 6,144 channels, but for both norms with a
    // shared gate in three accesses.  What spills, in bytes of scratch a lane: that 44 to 176, in
    // fp32 144 to 260; fp32 rows of 769 to 1,024 channels 40 to 132; 8 waves of four accesses
    // up to 684; 16 waves (above 8,192 channels) 192 to 1,292.
    const bool many = backward && post != GRKAN_NORM_NONE && gates > 0 && gate_channels == C;
    const int64_t most = many ? 192 : 256;
    p->waves = 1;
    while (p->waves < 8 && quads > (p->waves == 1 ? most : 192) * p->waves) p->waves *= 2;
    if (quads > 2048) p->waves = 16;
    p->K = (int32_t)ceil_div(quads, 64 * p->waves);
    p->per = p->waves == 1 ? 4 : 1;
    // as many walkers as the CUs hold: 16 waves each, the backward 8 (16 of the widest
    // rows)
    const int64_t walkers = (backward && p->waves < 16 ? 2048 : 4096) / p->waves;
    p->walk = ceil_div(rows > 0 ? rows : 1, walkers);
    p->blocks = ceil_div(ceil_div(rows > 0 ? rows : 1, p->walk), p->per);
    if (!backward) return;
    p->sums = post == GRKAN_NORM_NONE ? 3 : 4;
    p->off_sums = 0;
    p->off_gate = align256((size_t)p->blocks * p->sums * (size_t)C * 4);
    // dgate: two places for each walker, or one for each row
    size_t gate = 0;
    if (gates > 0 && rows > gates)
        gate = gate_channels == C && C > 1 ? (size_t)p->blocks * p->per * 2 * (size_t)C * 4 : (size_t)rows * 4;
    p->total = p->off_gate + align256(gate);
}

// The last kernel of the backward, 1,024 threads a workgroup: 32 columns of the three kinds of sums a
// workgroup, then `gates` values of dgate, a value a thread, which walks on where they are more than a
// launch holds.
struct ResidualSums {
    int32_t columns;
    int64_t blocks;
};

inline ResidualSums residual_sums(int64_t C, bool sums, int64_t gates) {
    const int64_t columns = sums ? 3 * ceil_div(C, 32) : 0, more = ceil_div(gates, 1024);
    return ResidualSums{(int32_t)columns, columns + (more < kMaxBlocks ? more : kMaxBlocks)};
}

}  // namespace grkan
