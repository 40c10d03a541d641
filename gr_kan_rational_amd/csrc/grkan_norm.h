// grkan_norm.h -- plans and kernel arguments of the group norm with an
// activation (grkan_norm.hip); internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grkan_block.h"
#include "grkan_device.h"

namespace grkan {

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

struct NormArgs {
    const void *x, *dy;
    void *y;                 // y, or dx
    float *mean, *rstd;      // outputs of the forward, inputs of the backward
    const float *w, *b, *A, *B;
    float *dw, *db, *dA, *dB;
    double *stats;           // split: [samples][groups][chunks * parts] pairs
    float *means;            // split backward: [samples][groups] pairs <t>, <t xh>
    float *partials;         // backward: [prows][dw, db of the channels; rational: 10 (straddle: 20) x cv]
    int64_t N, S, xs, xr, ds, dr;
    int32_t C, G, D, ng, dga;
    int32_t act;
    float eps;
    NormPlan p;
};

// grkan_norm.hip, one translation unit per I/O type and direction.
template <class IO> hipError_t launch_norm_forward(const NormArgs &a, hipStream_t s);
template <class IO> hipError_t launch_norm_backward(const NormArgs &a, hipStream_t s);

}  // namespace grkan
