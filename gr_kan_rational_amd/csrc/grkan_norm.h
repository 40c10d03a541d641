// grkan_norm.h -- kernel arguments of the group norm with an
// activation (grkan_norm.hip); internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grkan_device.h"
#include "grkan_plan.h"

namespace grkan {

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
