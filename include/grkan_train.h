/*
 * grkan_train.h -- C ABI of the operators that a deep stack of GR-KAN blocks
 * is trained and served with, beside those of grkan_block.h (libgrkan.so,
 * MI355X / gfx950):
 *
 *   8-bit quantiser and matrix product, a scale for each block of 128;
 *   the residual path from one block to the next with the norms on either
 *   side of it, forward and backward;
 *   the AdamW step over many tensors at once, states in 32 bits or 8.
 *
 * The conventions of grkan.h hold: device pointers on the current device,
 * owned by the caller; nothing is allocated or kept; work is enqueued on
 * `stream` and the call returns without waiting; arguments are validated
 * before any HIP call; no C++ exception crosses the interface.  Results are
 * bitwise reproducible: every sum is taken in an order that depends on the
 * call's sizes, types, kind of sums, scale layout and norms alone, and no atomics are used.
 */
#ifndef GRKAN_TRAIN_H
#define GRKAN_TRAIN_H

#include "grkan_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantiser to e4m3 (4 exponent bits, 3 of mantissa, largest value 448, no
 * infinity; torch's float8_e4m3fn).  With x_i the values of a block, or F(x_i),
 * F the group-rational activation:
 *
 *     amax  = max |x_i| over the finite x_i
 *     scale = the smallest power of two (2^-126 at least) with
 *             amax <= 448 scale; 1 for amax = 0
 *     q_i   = x_i / scale rounded to nearest even; NaN for a NaN or infinity
 *
 * A power of two makes the division exact, so a value is rounded once.  A
 * block is 128 values of a row (q), 128 of a column (qt), or 128 x 128 (tile:
 * q and qt then hold the same values).
 *   x         dtype io [rows][cols], row r at x + r ldx (ldx >= cols), aligned to
 *             its element size.
 *   act       GRKAN_ACT_NONE, or GRKAN_ACT_RATIONAL with A, B and n_groups as in
 *             grkan.h (cols a multiple of n_groups; A, B NULL for NONE).
 *   q         e4m3 [rows][cols], row r at q + r ldq; or NULL.  16-byte aligned, ldq
 *             a multiple of 16, ldq >= cols; the bytes from cols to the next
 *             multiple of 16 are zeroed.
 *   scale     fp32; row r's block b at scale[b ld_scale + r], with tile row block r
 *             of 128 (ld_scale >= the rows or row blocks).
 *   qt        e4m3 [cols][rows], the transpose, as q (ldqt >= rows); or NULL.
 *   scale_t   fp32; column c's block b (of rows) at scale_t[b ld_scale_t + c], with
 *             tile column block c of 128.
 *   rows >= 0 (0 is a no-op), cols >= 1.
 * GRKAN_ERR_UNSUPPORTED: rows >= 2^31 - 256, cols or ldx above 2^22, 2^24 or more blocks of
 * 64 rows x 128 columns, a misaligned pointer or leading dimension.
 */
GRKAN_API grkan_status_t grkan_fp8_quantize(
    const void *x, const float *A, const float *B, void *q, float *scale, void *qt, float *scale_t,
    int64_t rows, int64_t cols, int64_t ldx, int64_t ldq, int64_t ld_scale, int64_t ldqt,
    int64_t ld_scale_t, int32_t tile, int32_t n_groups, grkan_act_t act, grkan_dtype_t io,
    hipStream_t stream);

/*
 * Matrix product of e4m3 operands, a scale for each block of 128 values of k:
 *
 *     c[m][n] = sum over blocks kb of a_scale(m, kb) b_scale(n, kb)
 *               sum over k in kb of a[m][k] b[n][k]   + bias[n] + residual[m][n]
 *
 * A block's products are summed on the matrix cores; its sum times
 * (a_scale b_scale), a product that has to be in fp32's range, is added in fp32, and c
 * is rounded once.  How a block is summed:
 *     in fp32 (1e-7 of the sum of the products' sizes);
 *     or, bf16 c with GRKAN_FP8_SUMS_CUT, twice the rate: the matrix cores cut the products
 *     of each 8 values of k off at 2^-13 of the largest one's power of two.  Over a result
 *     that is a fortieth of the rounding to bf16; a single value whose large products cancel may
 *     be off by up to 7 x 2^-13 of the largest of each 8, which can exceed its own rounding.
 *   a, b      e4m3 [m][k], [n][k]: 16-byte aligned, lda, ldb multiples of 16 and
 *             >= k.  Bytes past k, to the next multiple of 16, are read and not used.
 *   a_scale   fp32, any finite values: (m, kb) at m a_scale_row + kb a_scale_block;
 *             a stride may be 0 (one scale for all).
 *   b_scale   likewise; with b_tile (0 or 1) row block n / 128 in the place of n.
 *   b_tile    0 or 1, and GRKAN_FP8_SUMS_CUT or'ed in (without effect on an fp32 c).
 *   bias      fp32 [n], or NULL.
 *   residual  dtype out [m][n], row r at residual + r ldr (ldr >= n), or NULL.
 *   c         dtype out (fp32 or bf16) [m][n], dense; may be the residual itself
 *             if that is dense; any other overlap is GRKAN_ERR_INVALID_ARG.
 *   m >= 0 (0 is a no-op), n, k >= 1.
 *   workspace grkan_fp8_matmul_workspace_size() bytes (may be 0), 256-byte aligned.
 * GRKAN_ERR_UNSUPPORTED: m >= 2^31 - 256, n, k or a leading dimension above 2^22, a
 * scale's row stride above 2^20, its block stride above 2^31,
 * m x n past the launch limits, a misaligned pointer or leading dimension.
 */
#define GRKAN_FP8_SUMS_CUT 16

GRKAN_API grkan_status_t grkan_fp8_matmul(
    const void *a, const float *a_scale, const void *b, const float *b_scale, const float *bias,
    const void *residual, void *c, int64_t m, int64_t n, int64_t k, int64_t lda,
    int64_t a_scale_row, int64_t a_scale_block, int64_t ldb, int64_t b_scale_row,
    int64_t b_scale_block, int32_t b_tile, int64_t ldr, grkan_dtype_t out, void *workspace,
    size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace the product needs (0 for arguments it would reject).
 * Host-only. */
GRKAN_API size_t grkan_fp8_matmul_workspace_size(int64_t m, int64_t n, int64_t k);

/* The norm over a row of C values v: layer: mean = <v>, rms: mean = 0;
 * rstd = 1 / sqrt(<(v - mean)^2> + eps), (v - mean) rstd weight + bias. */
typedef enum GRKAN_ENUM_INT {
    GRKAN_NORM_NONE = 0,
    GRKAN_NORM_LAYER = 1,
    GRKAN_NORM_RMS = 2
} grkan_norm_t;

/*
 * The residual path from one block to the next.  f is the block's result, x
 * what goes past it:
 *
 *     u = post(f)      h = x + scale_c gate u      z = norm(h)
 *
 * post is the norm after the block (or none), norm the one before the next.
 *   x, f      dtype io [rows][channels], row r at x + r ldx, f + r ldf, aligned to
 *             the element size.
 *   h, z      dtype io [rows][channels], dense; h may be x itself if x is dense; any
 *             other overlap is GRKAN_ERR_INVALID_ARG.  z and the statistics are formed
 *             from h before it is rounded.
 *   stats     fp32 [2][rows] (mean, rstd of h) or, with a post norm, [4][rows] (then
 *             those of f); the backward needs them.
 *   weight    fp32 [channels] or NULL (1); bias fp32 [channels] or NULL (0).
 *   scale     fp32 [channels] or NULL (1).
 *   gate      [gates][gate_channels], dense, in gate_io (fp32 or io), or NULL (1): row r
 *             takes gate row r / (rows / gates), rows a multiple of gates, gate_channels
 *             1 or channels.  One row for a sample's positions, one value for a
 *             sample (stochastic depth) or a token, or one for each element.
 *   post_weight, post_bias   as weight and bias, for post; NULL without one.
 *   norm      GRKAN_NORM_LAYER or GRKAN_NORM_RMS.
 *   eps       > 0.
 *   rows >= 0 (0 is a no-op), channels >= 1.
 * Statistics are formed in fp32 about the mean from values held on chip.  A NaN or
 * infinity touches no row but its own.  There h is what its formula gives, channel by channel (in
 * all channels where a post norm's statistics become NaN); z is NaN throughout, but for an rms norm
 * of infinities without a NaN, whose rstd is 0: NaN at them and 0 elsewhere.
 * GRKAN_ERR_UNSUPPORTED: channels above 16384, rows or gates >= 2^31, a stride above 2^31, a
 * misaligned pointer.
 */
GRKAN_API grkan_status_t grkan_residual_norm_forward(
    const void *x, const void *f, const float *weight, const float *bias, const float *scale,
    const void *gate, const float *post_weight, const float *post_bias, void *h, void *z,
    float *stats, int64_t rows, int64_t channels, int64_t ldx, int64_t ldf, int64_t gates,
    int64_t gate_channels, float eps, grkan_norm_t norm, grkan_norm_t post, grkan_dtype_t io,
    grkan_dtype_t gate_io, hipStream_t stream);

/*
 * Its backward, from dh = dL/dh (what reaches h besides through z) and dz = dL/dz:
 *
 *     xh = (h - mean) rstd,  t = dz weight,  <.> the mean over a row
 *     g  = dh + rstd (t - <t> - xh <t xh>)       (rms: without <t>)
 *     dx = g
 *     d = g scale gate:  df = d without a post norm, else the post norm's
 *                        backward of d, formed likewise
 *     dweight = sum dz xh   dbias = sum dz   dscale = sum g gate u
 *     dgate   = sum g scale u  over what shares a gate
 *     dpost_weight = sum d fh   dpost_bias = sum d
 *
 *   h, stats  the forward's results (h dense); f as given to it.  u and the normalised
 *             values are formed again from them.
 *   dh, dz    dtype io, with strides of their own; one of them may be NULL (zeros).
 *   dx, df    dtype io, dense; dx may be dh itself and df dz itself if those are dense;
 *             any other overlap is GRKAN_ERR_INVALID_ARG.
 *   d...      fp32 [channels], overwritten; dgate [gates][gate_channels] in gate_io.
 *             dpost_weight and dpost_bias only with a post norm, dgate with a gate.
 *   Each output may be NULL (not computed).  rows = 0 writes zeros to the sums and dgate.
 *   workspace grkan_residual_norm_backward_workspace_size() bytes, 256-byte aligned.
 */
GRKAN_API grkan_status_t grkan_residual_norm_backward(
    const void *f, const void *h, const void *dh, const void *dz, const float *stats,
    const float *weight, const float *scale, const void *gate, const float *post_weight,
    const float *post_bias, void *dx, void *df, float *dscale, void *dgate, float *dweight,
    float *dbias, float *dpost_weight, float *dpost_bias, int64_t rows, int64_t channels,
    int64_t ldf, int64_t lddh, int64_t lddz, int64_t gates, int64_t gate_channels,
    grkan_norm_t norm, grkan_norm_t post, grkan_dtype_t io, grkan_dtype_t gate_io, void *workspace,
    size_t workspace_bytes, hipStream_t stream);

/* gates = 0: without a gate.  Host-only. */
GRKAN_API size_t grkan_residual_norm_backward_workspace_size(int64_t rows, int64_t channels,
                                                             int64_t gates, int64_t gate_channels,
                                                             grkan_norm_t post, grkan_dtype_t io);

/* One tensor of the step below. */
typedef struct {
    void *param;       /* dtype io [n]; the weights                                          */
    const void *grad;  /* dtype io [n]                                                       */
    float *master;     /* fp32 [n]: the weights in 32 bits, `param` their copy rounded to nearest
                          even (where it is not, another has written it, and `param` is taken);
                          or NULL: `param` is stepped and rounded to nearest even            */
    void *avg;         /* first moment: fp32 [n], or e4m3 [n to whole blocks of 128]         */
    void *sq;          /* second moment: fp32 [n], or its root in e4m3, as avg               */
    float *avg_scale;  /* 8 bits: fp32, one for each block of 128; else NULL                 */
    float *sq_scale;
    int64_t n;         /* >= 0 */
    grkan_dtype_t io;
} grkan_adamw_tensor_t;

typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;            /* 1 for the first                                              */
    const float *lr_ptr;     /* device, one value, read by the kernel in the place of lr; or
                                NULL                                                         */
    const int64_t *step_ptr; /* likewise for step                                            */
    const float *grad_scale; /* device, one value that every gradient is multiplied with; or
                                NULL                                                         */
    uint32_t seed;           /* of the 8-bit states' rounding                                */
} grkan_adamw_t;

/*
 * One AdamW step over `count` tensors:
 *
 *     m = beta1 m + (1 - beta1) g       v = beta2 v + (1 - beta2) g^2
 *     w = w (1 - lr weight_decay)
 *         - lr / (1 - beta1^step) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 *
 * in fp32, each operation rounded once (no fused multiply-add).
 *
 * bits = 32: m and v are kept in fp32.  bits = 8: m and r = sqrt(v) are kept in
 * e4m3 with a power-of-two scale for each 128 values of the flattened tensor (the
 * scales of grkan_fp8_quantize).  They are rounded up with the probability of the
 * remainder, so that a moving average that changes by less than a step of its
 * 8-bit type still moves; the update itself uses the values before rounding.  r > 0
 * is never rounded to 0.  The random numbers (16 bits for each of the two) are a
 * function of (seed, step, the block's number over all tensors in order, the place
 * in the block) alone:
 *
 *     mix(h): h ^= h >> 16; h *= 0x6A09E667; h ^= h >> 15; h *= 0xBB67AE85; h ^= h >> 16
 *     key = mix(mix(seed) + step)      r = mix(mix(key + block) + place), all mod 2^32
 *     m takes r mod 2^16, the root r / 2^16
 *
 * A NaN or infinity is kept as a NaN in its place and does not enter its block's
 * scale.  Codes past n in the last block are zeros.
 *   tensors   host array, read before the call returns.  All on the current device; no
 *             two of their pointers share memory (checked among the tensors of a launch,
 *             48 at a time; GRKAN_ERR_INVALID_ARG, before anything is launched), and lr_ptr,
 *             step_ptr and grad_scale lie in nothing that the step writes (likewise).
 *   Pointers are aligned to their element size; avg and sq in 8 bits to 16 bytes.
 *   lr >= 0, 0 <= beta < 1, eps >= 0, weight_decay >= 0, step >= 1 (host values; the
 *   device's are not checked), bits 8 or 32.
 * A host array and values: a graph captured around the call holds them as they
 * were; lr_ptr and step_ptr are read at each replay.
 */
GRKAN_API grkan_status_t grkan_adamw_step(const grkan_adamw_tensor_t *tensors, int64_t count,
                                          const grkan_adamw_t *hyper, int32_t bits,
                                          hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GRKAN_TRAIN_H */
