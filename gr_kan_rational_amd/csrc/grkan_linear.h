// grkan_linear.h -- plans and kernel arguments of the linear map with bias,
// activation and residual in its epilogue (grkan_linear.hip); internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "grkan_block.h"

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

ProductPlan plan_product(int form, int64_t M, int64_t N, int64_t K, bool aligned, int32_t act, int64_t dga);
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
struct SlopePlan {
    int32_t vec, vpr, chunks;
    int64_t chunk_rows;
    size_t partials_bytes;
};
SlopePlan plan_slope(int64_t rows, int64_t N, int32_t act, int64_t dga);
hipError_t launch_slope(const SlopeArgs &a, hipStream_t s);

}  // namespace grkan
