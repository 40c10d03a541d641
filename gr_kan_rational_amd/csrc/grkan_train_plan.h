// grkan_train_plan.h -- how the launches of the operators of grkan_train.h are
// laid out: plans from sizes and types alone.  Host code without HIP; internal.
#pragma once

#include "grkan_plan.h"
#include "grkan_train.h"

namespace grkan {

constexpr int kBlock8 = 128;  // values that share a scale

// ------------------------------------------------------------ quantiser

inline grkan_status_t quantize_shape(int64_t rows, int64_t cols, int64_t ldx, int32_t n_groups, grkan_act_t act,
                                     grkan_dtype_t io) {
    if (io != GRKAN_F32 && io != GRKAN_BF16) return GRKAN_ERR_INVALID_ARG;
    if (act != GRKAN_ACT_NONE && act != GRKAN_ACT_RATIONAL) return GRKAN_ERR_INVALID_ARG;
    if (rows < 0 || cols < 1 || ldx < cols) return GRKAN_ERR_INVALID_ARG;
    if (act == GRKAN_ACT_RATIONAL && (n_groups < 1 || cols % n_groups != 0)) return GRKAN_ERR_INVALID_ARG;
    if (rows > kMaxRows || cols > kMaxWidth || ldx > kMaxWidth) return GRKAN_ERR_UNSUPPORTED;
    // a workgroup for at least 16 rows of 128 columns, in one launch
    if (ceil_div(rows, 16) * ceil_div(cols, kBlock8) >= (int64_t(1) << 24)) return GRKAN_ERR_UNSUPPORTED;
    return GRKAN_OK;
}

// ------------------------------------------------------------ 8-bit product

struct Product8Plan {
    int32_t splits;
    int64_t k_split;         // of a split, whole blocks
    size_t partials_bytes;
};

inline grkan_status_t product8_shape(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 1 || K < 1) return GRKAN_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxWidth || K > kMaxWidth) return GRKAN_ERR_UNSUPPORTED;
    if (ceil_div(M, 64) * ceil_div(N, 64) >= (int64_t(1) << 24)) return GRKAN_ERR_UNSUPPORTED;
    return GRKAN_OK;
}

inline Product8Plan plan_product8(int64_t M, int64_t N, int64_t K) {
    Product8Plan p{};
    p.splits = 1;
    p.k_split = K;
    return p;
}

// ------------------------------------------------------------ residual path

constexpr int64_t kMaxChannels = 16384;
constexpr int64_t kMaxStride = int64_t(1) << 31;

// A row is held by `waves` waves, 4 K values a lane.  The backward's waves (or
// workgroups of `waves` > 1) each walk over `unit_rows` rows that share a gate
// row if the gate has one per channel, so that its sum stays in registers.
struct ResidualPlan {
    int32_t K, waves;
    int32_t per;             // rows that a workgroup holds at a time
    int64_t blocks;
    int64_t units, unit_rows, units_per_gate;
    int32_t sums;            // column sums: dweight, dbias, dscale (, dpost_weight, dpost_bias)
    size_t off_sums, off_gate, total;
};

inline grkan_status_t residual_shape(int64_t rows, int64_t C, int64_t gates, int64_t gate_channels, grkan_dtype_t io) {
    if (io != GRKAN_F32 && io != GRKAN_BF16) return GRKAN_ERR_INVALID_ARG;
    if (rows < 0 || C < 1 || gates < 0) return GRKAN_ERR_INVALID_ARG;
    if (gates > 0 && (rows % gates != 0 || (gate_channels != 1 && gate_channels != C))) return GRKAN_ERR_INVALID_ARG;
    if (C > kMaxChannels || rows > INT32_MAX) return GRKAN_ERR_UNSUPPORTED;
    return GRKAN_OK;
}

// The backward's rows: about kResidualWalkers waves or workgroups, each a run of rows.
constexpr int64_t kResidualWalkers = 2048;

inline void residual_plan(int64_t rows, int64_t C, int64_t gates, int64_t gate_channels, grkan_norm_t post,
                          bool backward, ResidualPlan *p) {
    *p = ResidualPlan{};
    const int64_t quads = ceil_div(C, 4);
    p->waves = quads <= 256 ? 1 : (quads <= 1024 ? 4 : 16);
    p->K = (int32_t)ceil_div(quads, 64 * p->waves);
    p->per = p->waves == 1 ? 4 : 1;
    if (!backward) {
        p->blocks = ceil_div(rows, p->per);
        if (p->blocks > 4096) p->blocks = 4096;
        return;
    }
    const bool columns = gates > 0 && gate_channels == C && rows > gates && C > 1;
    const int64_t runs = columns ? gates : 1, run = rows / (runs > 0 ? runs : 1);
    const int64_t walkers = p->waves == 1 ? kResidualWalkers : kResidualWalkers / (2 * p->waves);
    int64_t per_run = ceil_div(walkers, runs);
    if (per_run > ceil_div(run, 4)) per_run = ceil_div(run, 4);
    if (per_run < 1) per_run = 1;
    p->unit_rows = ceil_div(run, per_run);
    if (p->unit_rows < 1) p->unit_rows = 1;
    p->units_per_gate = ceil_div(run, p->unit_rows);
    p->units = p->units_per_gate * runs;
    p->blocks = ceil_div(p->units < walkers ? p->units : walkers, p->per);
    if (p->blocks < 1) p->blocks = 1;
    p->sums = post == GRKAN_NORM_NONE ? 3 : 5;
    p->off_sums = 0;
    p->off_gate = align256((size_t)p->blocks * p->sums * (size_t)C * 4);
    size_t gate = 0;
    if (columns)
        gate = p->units_per_gate > 1 ? (size_t)p->units * (size_t)C * 4 : 0;
    else if (gates > 0 && rows > gates)
        gate = (size_t)rows * 4;
    p->total = p->off_gate + align256(gate);
}

}  // namespace grkan
