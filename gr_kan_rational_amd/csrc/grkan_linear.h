// grkan_linear.h -- kernel arguments of the linear map with bias,
// activation and residual in its epilogue (grkan_linear.hip); internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grkan_plan.h"

namespace grkan {

// One matrix product C[m][n] = sum over k of Q(m, k) P(n, k), bf16 operands,
// fp32 sums.  An operand is a matrix of rows of `ld` elements; its rows run
// over its own index (K contiguous) or, `strided`, over k (its own index
// contiguous).
struct Operand {
    const void *p;
    int64_t ld;
};

// What becomes of a sum: h = sum + bias; pre = bf16(h) if pre; z = bf16(act(h)
// + residual).
struct Epilogue {
    const float *bias;
    const float *A, *B;      // rational
    const void *residual;    // bf16 [M][ldr]
    void *pre;               // bf16 [M][N]
    void *z;                 // bf16 [M][N]
    int64_t ldr;
    int32_t act, dga;        // dga: columns per activation group
};

struct ProductArgs {
    Operand q, p;
    int32_t M, N, K;
    int32_t splits, k_split; // k range of a split (a multiple of the K step)
    float *partials;         // [splits][M][N] sums, when split
    Epilogue e;
};

hipError_t launch_product(int form, const ProductPlan &p, const ProductArgs &a, hipStream_t s);

// dpre = dz act'(pre) (bf16 [rows][ldp]) with the column sums of dpre in fp32
// (dbias) and, for the rational, dA and dB.  act none: dbias alone.
struct SlopeArgs {
    const void *dz, *pre;    // bf16 [rows][lddz], [rows][N]
    void *dpre;
    const float *A, *B;
    float *dbias, *dA, *dB;
    float *partials;         // [chunks][N + (rational: 10 accesses)]
    int64_t rows, lddz, ldp;
    int32_t N, act, ng, dga;
    int32_t vec, vpr;        // elements per access, accesses per row
    int32_t chunks;
    int64_t chunk_rows;
};
hipError_t launch_slope(const SlopeArgs &a, hipStream_t s);

}  // namespace grkan
