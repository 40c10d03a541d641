// grkan_adamw.h -- kernel arguments of the AdamW step (grkan_adamw.hip);
// internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grkan_train.h"

namespace grkan {

// Elements of a workgroup, and tensors of a launch: a launch's arguments stay
// below 4 KB.
constexpr int kAdamwChunk = 4096;
constexpr int kAdamwTensors = 48;

struct AdamwTensor {
    void *param;
    const void *grad;
    float *master;           // or NULL
    void *avg, *sq;
    float *avg_scale, *sq_scale;
    int64_t n;
};

// What a step is multiplied with.
struct AdamwFactors {
    float beta1, rest1, beta2, rest2, keep, rate, root, eps;
};

struct AdamwArgs {
    AdamwTensor t[kAdamwTensors];
    uint32_t first[kAdamwTensors + 1];   // each tensor's first workgroup of the launch
    uint32_t block[kAdamwTensors];       // 8 bits: its first block of 128, over all tensors
    uint8_t flags[kAdamwTensors];        // kAdamwBf16, kAdamwVec
    AdamwFactors f;          // unless lr or step are read on the device
    double lr, beta1, beta2, decay, eps;
    int64_t step;
    const float *lr_ptr;
    const int64_t *step_ptr;
    const float *grad_scale;
    uint32_t seed;
    int32_t count;
};
constexpr uint8_t kAdamwBf16 = 1, kAdamwVec = 2;
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");

void prepare_adamw(AdamwArgs &a);   // the factors, from the other arguments
hipError_t launch_adamw(const AdamwArgs &a, int bits, hipStream_t s);

}  // namespace grkan
