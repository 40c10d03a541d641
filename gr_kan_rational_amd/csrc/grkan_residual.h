// grkan_residual.h -- kernel arguments of the residual path with its norms
// (grkan_residual.hip); internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grkan_fastdiv.h"
#include "grkan_train_plan.h"

namespace grkan {

struct ResidualArgs {
    const void *x, *f, *dh, *dz;     // x: forward; dh, dz: backward, either may be NULL
    void *h, *z;                     // forward: outputs; backward: h an input
    void *dx, *df, *dgate;
    float *stats;
    const float *weight, *bias, *scale, *post_weight, *post_bias;
    const void *gate;
    float *dweight, *dbias, *dscale, *dpost_weight, *dpost_bias;
    float *sums;                     // [blocks][sums][C]
    float *gate_sums;                // [units][C] or [rows]
    int64_t rows, ldx, ldf, lddh, lddz;
    int64_t gates;                   // gate rows
    int64_t gate_rows;               // rows that share one
    FastDiv gate_div;                // division by it
    int32_t C;
    int32_t norm, post;
    bool gate_wide;                  // a gate for each channel
    bool gate_bf16;
    bool vec;                        // every access of four elements is aligned and whole
    float eps;
    ResidualPlan p;
};

// grkan_residual.hip, one translation unit per I/O type and direction.
template <class T> hipError_t launch_residual_forward(const ResidualArgs &a, hipStream_t s);
template <class T> hipError_t launch_residual_backward(const ResidualArgs &a, hipStream_t s);

}  // namespace grkan
