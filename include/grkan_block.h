/*
 * grkan_block.h -- C ABI of the operators around the group-rational
 * activation in a GR-KAN transformer block (libgrkan.so, MI355X / gfx950):
 *
 *   group norm with an activation, channels last, forward and backward;
 *   the linear map with bias, activation and residual in its epilogue,
 *   forward and backward.
 *
 * The pages describe a GR-KAN layer as the group-rational activation followed
 * by a linear map ("FlashKAT: Understanding and Addressing Performance
 * Bottlenecks in the Kolmogorov-Arnold Transformer", Paper-Notes page (AAAI
 * 2026), arXiv 2505.13813, section "1. 性能瓶颈诊断", Insight 2) that takes
 * the place of a ViT's MLP.  Such a block is
 *
 *     x + W2 F2(W1 F1(norm(x)) + b1) + b2 :
 *
 * F1 runs where the norm's result is formed and F2 where the first product's
 * result is formed, once per element each.
 *
 * The conventions of grkan.h hold: device pointers on the current device,
 * owned by the caller; nothing is allocated or kept; work is enqueued on
 * `stream` and the call returns without waiting; arguments are validated
 * before any HIP call; no C++ exception crosses the interface.  Results are
 * bitwise reproducible: every sum is taken in an order that depends on the
 * shape and, in the linear map's products, on whether the operands are whole
 * 16-byte vectors at aligned addresses.
 */
#ifndef GRKAN_BLOCK_H
#define GRKAN_BLOCK_H

#include "grkan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The activation applied to h.  GRKAN_ACT_RATIONAL is F of grkan.h with
 * degrees (5, 4): A fp32 [n_groups][6], B fp32 [n_groups][4], channel c in
 * group c / (channels / n_groups).  A, B (and dA, dB) are NULL for the others. */
typedef enum GRKAN_ENUM_INT {
    GRKAN_ACT_NONE = 0,    /* h                                        */
    GRKAN_ACT_SILU = 1,    /* h / (1 + e^-h)                           */
    GRKAN_ACT_GELU = 2,    /* h Phi(h), Phi the normal distribution's  */
    GRKAN_ACT_RATIONAL = 3 /* F(h), the group-rational activation      */
} grkan_act_t;

/*
 * Group norm with an activation, channels last.  x is [samples][positions]
 * [channels]; the channels are cut into norm_groups contiguous groups of
 * D = channels / norm_groups.  For sample n and group g, over its positions
 * x D values,
 *
 *     mean = sum x / (positions D)     var = sum (x - mean)^2 / (positions D)
 *     rstd = 1 / sqrt(var + eps)       xh  = (x - mean) rstd
 *     h    = xh weight_c + bias_c      y   = act(h)
 *
 * positions = 1 with norm_groups = 1 is the norm per token (layer norm).
 *   x         dtype io; element (n, s, c) at x[n x_sample + s x_row + c]
 *             (strides in elements, x_row >= channels, x_sample >= 0), aligned
 *             to its element size.
 *   y         dtype io, dense [samples][positions][channels]; may be x itself
 *             if x is dense; any other overlap is GRKAN_ERR_INVALID_ARG.
 *   mean,     fp32 [samples][norm_groups] outputs; the backward needs them.
 *   rstd
 *   weight,   fp32 [channels], or NULL (1 and 0).
 *   bias
 *   eps       > 0.
 *   samples, positions >= 0 (no element: nothing is written but, for samples
 *   without positions, mean = 0 and rstd = 1 / sqrt(eps)); channels >= 1, a
 *   multiple of norm_groups and, with GRKAN_ACT_RATIONAL, of n_groups.
 *   workspace grkan_group_norm_forward_workspace_size() bytes (may be 0, then
 *             it may be NULL), 256-byte aligned.
 * Statistics are formed in fp32 about the mean from values held on chip, or
 * from sums of x and x^2 in fp64 where a group's values do not fit there.  A
 * NaN or infinity among a group's values makes that group's outputs NaN and
 * touches no other group.
 * GRKAN_ERR_UNSUPPORTED: channels >= 2^24, samples x norm_groups or positions
 * >= 2^31, a misaligned pointer.
 */
GRKAN_API grkan_status_t grkan_group_norm_forward(
    const void *x, void *y, float *mean, float *rstd, const float *weight, const float *bias,
    const float *A, const float *B, int64_t samples, int64_t positions, int64_t channels,
    int64_t x_sample, int64_t x_row, int32_t norm_groups, int32_t n_groups, float eps,
    grkan_act_t act, grkan_dtype_t io, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace the forward needs (0 for arguments it would reject).
 * Host-only. */
GRKAN_API size_t grkan_group_norm_forward_workspace_size(
    int64_t samples, int64_t positions, int64_t channels, int32_t norm_groups, int32_t n_groups,
    grkan_act_t act, grkan_dtype_t io);

/*
 * Its backward.  With dh = dy act'(h), t = dh weight and <.> the mean over a
 * (sample, group),
 *
 *     dx      = rstd (t - <t> - xh <t xh>)
 *     dweight = sum dh xh     dbias = sum dh     over samples and positions
 *     dA, dB  as grkan_backward's, at h.
 *
 *   x, mean,  the forward's input and outputs (x with its strides).
 *   rstd
 *   dy        as x, with strides of its own.
 *   dx        dtype io, dense; may be x or dy itself if that is dense.
 *   dweight,  fp32 [channels], overwritten; each may be NULL (not computed).
 *   dbias
 *   dA, dB    fp32 [n_groups][6], [n_groups][4], overwritten; required with
 *             GRKAN_ACT_RATIONAL.
 *   workspace grkan_group_norm_backward_workspace_size() bytes, 256-byte
 *             aligned.
 * h is formed again in fp32 from x and the statistics; for the rational the
 * sign of Q is that of Q at this fp32 h.  With no element (samples or
 * positions 0), dweight, dbias, dA and dB are zeroed.
 */
GRKAN_API grkan_status_t grkan_group_norm_backward(
    const void *x, const void *dy, const float *mean, const float *rstd, const float *weight,
    const float *bias, const float *A, const float *B, void *dx, float *dweight, float *dbias,
    float *dA, float *dB, int64_t samples, int64_t positions, int64_t channels, int64_t x_sample,
    int64_t x_row, int64_t dy_sample, int64_t dy_row, int32_t norm_groups, int32_t n_groups,
    grkan_act_t act, grkan_dtype_t io, void *workspace, size_t workspace_bytes, hipStream_t stream);

GRKAN_API size_t grkan_group_norm_backward_workspace_size(
    int64_t samples, int64_t positions, int64_t channels, int32_t norm_groups, int32_t n_groups,
    grkan_act_t act, grkan_dtype_t io);

/*
 * Linear map with bias, activation and residual in its epilogue:
 *
 *     h = x W^T + bias        z = act(h) + residual
 *
 * bf16 x, W, residual, z, fp32 bias; products accumulate in fp32, the
 * epilogue is fp32 and z is rounded once to nearest-even bf16.
 *   x         bf16 [rows][d_in], row r at x + r ldx (ldx >= d_in).
 *   W         bf16 [d_out][d_in], dense.
 *   bias      fp32 [d_out], or NULL.
 *   residual  bf16 [rows][d_out], row r at residual + r ldr (ldr >= d_out), or
 *             NULL (ldr is then ignored).
 *   z         bf16 [rows][d_out], dense; may be the residual itself if that is
 *             dense; any other overlap is GRKAN_ERR_INVALID_ARG.
 *   pre       bf16 [rows][d_out], dense: h, for the backward; or NULL.
 *   A, B      with GRKAN_ACT_RATIONAL, channel groups of d_out / n_groups.
 *   rows >= 0 (0 is a no-op), d_in, d_out >= 1; any sizes, strides and element
 *   alignment are served, whole 16-byte vectors in both widths fastest.
 *
 * Without bias, activation and residual this is grkan_linear_forward (grkan.h)
 * for any shape; new callers take this one, which is the faster of the two but at
 * the largest products (1 x 3,072 from 768: 9 us a call against 22; 197 x 768 from
 * 3,072: 13 against 69; 50,432 x 768 from 3,072: 252 against 256; 201,728 x 3,072
 * from 768: 1,096 against 1,025).  Its sums are taken in another order.
 *   workspace grkan_linear_act_forward_workspace_size() bytes (may be 0),
 *             256-byte aligned; enough for any strides and alignment.
 * GRKAN_ERR_UNSUPPORTED: rows >= 2^31 - 256, a width or stride above 2^22, rows x
 * d_out past the launch limits, a misaligned pointer.
 */
GRKAN_API grkan_status_t grkan_linear_act_forward(
    const void *x, const void *W, const float *bias, const void *residual, const float *A,
    const float *B, void *z, void *pre, int64_t rows, int64_t d_in, int64_t d_out, int64_t ldx,
    int64_t ldr, int32_t n_groups, grkan_act_t act, void *workspace, size_t workspace_bytes,
    hipStream_t stream);

GRKAN_API size_t grkan_linear_act_forward_workspace_size(int64_t rows, int64_t d_in, int64_t d_out,
                                                         int32_t n_groups, grkan_act_t act);

/*
 * Its backward, given dz = dL/dz and the forward's pre:
 *
 *     dpre = dz act'(pre)     (bf16, internal; dz itself for GRKAN_ACT_NONE)
 *     dx   = dpre W           bf16 [rows][d_in]
 *     dW   = dpre^T x         bf16 [d_out][d_in]
 *     dbias = sum of dpre     fp32 [d_out], from dpre before its rounding
 *     dA, dB                  as grkan_backward's, at pre (Q in fp64 and the
 *                             decision of its sign included)
 *
 * and dL/dresidual is dz.  dpre is rounded to bf16 as the operand of the
 * matrix cores; that error is relative to each term, as that of any bf16
 * operand.
 *   dz        bf16 [rows][d_out], row r at dz + r lddz.
 *   pre       bf16 [rows][d_out], dense; not read for GRKAN_ACT_NONE.
 *   dx, dW,   outputs, dense, overwritten; each may be NULL (not computed).
 *   dbias
 *   dA, dB    required with GRKAN_ACT_RATIONAL.
 *   rows == 0 writes zeros to dW, dbias, dA and dB.
 *   workspace grkan_linear_act_backward_workspace_size() bytes, 256-byte
 *             aligned.
 */
GRKAN_API grkan_status_t grkan_linear_act_backward(
    const void *x, const void *W, const void *dz, const void *pre, const float *A, const float *B,
    void *dx, void *dW, float *dbias, float *dA, float *dB, int64_t rows, int64_t d_in,
    int64_t d_out, int64_t ldx, int64_t lddz, int32_t n_groups, grkan_act_t act, void *workspace,
    size_t workspace_bytes, hipStream_t stream);

GRKAN_API size_t grkan_linear_act_backward_workspace_size(int64_t rows, int64_t d_in, int64_t d_out,
                                                          int32_t n_groups, grkan_act_t act);

#ifdef __cplusplus
}
#endif

#endif /* GRKAN_BLOCK_H */
