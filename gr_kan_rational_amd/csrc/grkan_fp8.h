// grkan_fp8.h -- kernel arguments of the 8-bit quantiser and product
// (grkan_quantize.hip, grkan_product8.hip); internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grkan_train_plan.h"

namespace grkan {

struct QuantizeArgs {
    const void *x;
    const float *A, *B;      // rational, or NULL
    uint8_t *q, *qt;         // either may be NULL
    float *scale, *scale_t;
    int64_t ldx, ldq, ldqt, lds, ldst;
    int32_t rows, cols;
    int32_t dga;             // columns per activation group
    int32_t tile;
    bool bf16;
};
hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t s);

struct Operand8 {
    const uint8_t *p;
    const float *scale;
    int64_t ld, srow, sblock;
};

struct Product8Args {
    Operand8 a, b;
    const float *bias;
    const void *residual;
    void *c;
    float *partials;         // [splits][M][N], when split
    int64_t ldr;
    int32_t M, N, K;
    int32_t splits, k_split;
    int32_t b_tile;
    bool bf16;
    bool cut;                // bf16: blocks summed by the 8-bit matrix instruction, which cuts products
};
hipError_t launch_product8(const Product8Plan &p, const Product8Args &a, hipStream_t s);

}  // namespace grkan
