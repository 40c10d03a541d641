// grkan_train_api.hip -- the C ABI of include/grkan_train.h: argument validation
// and dispatch.  Plans depend on shapes and types alone, so results have the
// same bits on every device.
#include <stdint.h>

#include <cstdlib>

#include "grkan_adamw.h"
#include "grkan_check.h"
#include "grkan_fp8.h"
#include "grkan_residual.h"
#include "grkan_train.h"

using namespace grkan;

namespace {

// Bytes from the first to the last element of `rows` rows of `width` elements,
// `ld` apart (the sizes are limited, so this fits).
size_t rows_bytes(int64_t rows, int64_t width, int64_t ld, size_t es) {
    return rows > 0 ? ((size_t)(rows - 1) * ld + width) * es : 0;
}

bool rows16(const void *p, int64_t ld) { return aligned(p, 16) && ld % 16 == 0; }

}  // namespace

// ------------------------------------------------------------ 8 bits

extern "C" grkan_status_t grkan_fp8_quantize(const void *x, const float *A, const float *B, void *q, float *scale,
                                             void *qt, float *scale_t, int64_t rows, int64_t cols, int64_t ldx,
                                             int64_t ldq, int64_t ld_scale, int64_t ldqt, int64_t ld_scale_t,
                                             int32_t tile, int32_t n_groups, grkan_act_t act, grkan_dtype_t io,
                                             hipStream_t stream) {
    grkan_status_t st = quantize_shape(rows, cols, ldx, n_groups, act, io);
    if (st != GRKAN_OK) return st;
    const bool rational = act == GRKAN_ACT_RATIONAL;
    if (rational ? (!A || !B) : (A || B)) return GRKAN_ERR_INVALID_ARG;
    if (tile != 0 && tile != 1) return GRKAN_ERR_INVALID_ARG;
    if (rows == 0) return GRKAN_OK;
    if ((!q && !qt) || !q != !scale || !qt != !scale_t) return GRKAN_ERR_INVALID_ARG;
    const int64_t rb = ceil_div(rows, kBlock8), cb = ceil_div(cols, kBlock8);
    const int64_t srows = tile ? rb : rows, scols = tile ? cb : cols;
    if (q && (ldq < cols || ld_scale < srows)) return GRKAN_ERR_INVALID_ARG;
    if (qt && (ldqt < rows || ld_scale_t < scols)) return GRKAN_ERR_INVALID_ARG;
    if ((q && (ldq > kMaxWidth || ld_scale > INT32_MAX)) || (qt && (ldqt > INT32_MAX || ld_scale_t > INT32_MAX)))
        return GRKAN_ERR_UNSUPPORTED;
    const int es = io_bytes(io);
    if (!aligned(x, es) || !aligned(A, 4) || !aligned(B, 4) || !aligned(scale, 4) || !aligned(scale_t, 4) ||
        (q && !rows16(q, ldq)) || (qt && !rows16(qt, ldqt)))
        return GRKAN_ERR_UNSUPPORTED;
    if (!x) return GRKAN_ERR_INVALID_ARG;
    const Range ins[] = {{x, rows_bytes(rows, cols, ldx, es)}, {A, rational ? (size_t)n_groups * 24 : 0},
                         {B, rational ? (size_t)n_groups * 16 : 0}};
    const Range outs[] = {{q, rows_bytes(rows, (cols + 15) / 16 * 16, ldq, 1)},
                          {scale, rows_bytes(cb, srows, ld_scale, 4)},
                          {qt, rows_bytes(cols, (rows + 15) / 16 * 16, ldqt, 1)},
                          {scale_t, rows_bytes(rb, scols, ld_scale_t, 4)}};
    if (outputs_overlap(outs, 4, ins, 3)) return GRKAN_ERR_INVALID_ARG;
    // ---- validation done; HIP calls from here on
    QuantizeArgs a{};
    a.x = x;
    a.A = A;
    a.B = B;
    a.q = static_cast<uint8_t *>(q);
    a.qt = static_cast<uint8_t *>(qt);
    a.scale = scale;
    a.scale_t = scale_t;
    a.ldx = ldx;
    a.ldq = ldq;
    a.ldqt = ldqt;
    a.lds = ld_scale;
    a.ldst = ld_scale_t;
    a.rows = (int32_t)rows;
    a.cols = (int32_t)cols;
    a.dga = rational ? (int32_t)(cols / n_groups) : 1;
    a.tile = tile;
    a.bf16 = io == GRKAN_BF16;
    return from_hip(launch_quantize(a, stream));
}

extern "C" size_t grkan_fp8_matmul_workspace_size(int64_t m, int64_t n, int64_t k) {
    if (product8_shape(m, n, k) != GRKAN_OK || m == 0) return 0;
    return product8_bytes(m, n, k);
}

extern "C" grkan_status_t grkan_fp8_matmul(const void *a, const float *a_scale, const void *b, const float *b_scale,
                                           const float *bias, const void *residual, void *c, int64_t m, int64_t n,
                                           int64_t k, int64_t lda, int64_t a_scale_row, int64_t a_scale_block,
                                           int64_t ldb, int64_t b_scale_row, int64_t b_scale_block, int32_t b_tile,
                                           int64_t ldr, grkan_dtype_t out, void *workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
    grkan_status_t st = product8_shape(m, n, k);
    if (st != GRKAN_OK) return st;
    if (out != GRKAN_F32 && out != GRKAN_BF16) return GRKAN_ERR_INVALID_ARG;
    const bool cut = (b_tile & GRKAN_FP8_SUMS_CUT) != 0;
    b_tile &= ~GRKAN_FP8_SUMS_CUT;
    if (b_tile != 0 && b_tile != 1) return GRKAN_ERR_INVALID_ARG;
    if (lda < k || ldb < k || (residual && ldr < n)) return GRKAN_ERR_INVALID_ARG;
    if (a_scale_row < 0 || a_scale_block < 0 || b_scale_row < 0 || b_scale_block < 0) return GRKAN_ERR_INVALID_ARG;
    if (lda > kMaxWidth || ldb > kMaxWidth || (residual && ldr > kMaxWidth)) return GRKAN_ERR_UNSUPPORTED;
    if (a_scale_row > kMaxScaleRow || a_scale_block > INT32_MAX || b_scale_row > kMaxScaleRow || b_scale_block > INT32_MAX)
        return GRKAN_ERR_UNSUPPORTED;
    if (!b || !b_scale) return GRKAN_ERR_INVALID_ARG;
    const int es = io_bytes(out);
    if ((a && !rows16(a, lda)) || lda % 16 != 0 || !rows16(b, ldb) || !aligned(a_scale, 4) || !aligned(b_scale, 4) ||
        !aligned(bias, 4) || !aligned(residual, es) || !aligned(c, es))
        return GRKAN_ERR_UNSUPPORTED;
    if (m == 0) return GRKAN_OK;
    if (!a || !a_scale || !c) return GRKAN_ERR_INVALID_ARG;
    const Product8Plan p = plan_product8(m, n, k, out == GRKAN_BF16, b_tile != 0, cut);
    const size_t need = align256(p.partials_bytes);
    const int64_t kb = ceil_div(k, kBlock8), nb = b_tile ? ceil_div(n, kBlock8) : n;
    auto scales = [&](int64_t r, int64_t row, int64_t block) { return (size_t)((r - 1) * row + (kb - 1) * block + 1) * 4; };
    const Range rr{residual, residual ? rows_bytes(m, n, ldr, es) : 0};
    const Range ins[] = {{a, rows_bytes(m, k, lda, 1)}, {b, rows_bytes(n, k, ldb, 1)},
                         {a_scale, scales(m, a_scale_row, a_scale_block)},
                         {b_scale, scales(nb, b_scale_row, b_scale_block)}, {bias, (size_t)n * 4}, rr};
    const Range outs[] = {{workspace, need}, {c, (size_t)m * n * es}};
    const bool in_place = residual == c && ldr == n;
    if (outputs_overlap(outs, 1, ins, 6) || outputs_overlap(outs, 2, ins, 5) || (!in_place && overlap(outs[1], rr)))
        return GRKAN_ERR_INVALID_ARG;
    if (need && (!workspace || workspace_bytes < need)) return GRKAN_ERR_INVALID_ARG;
    if (need && !aligned(workspace, 256)) return GRKAN_ERR_UNSUPPORTED;
    // ---- validation done; HIP calls from here on
    Product8Args g{};
    g.a = Operand8{static_cast<const uint8_t *>(a), a_scale, lda, a_scale_row, a_scale_block};
    g.b = Operand8{static_cast<const uint8_t *>(b), b_scale, ldb, b_scale_row, b_scale_block};
    g.bias = bias;
    g.residual = residual;
    g.c = c;
    g.partials = static_cast<float *>(workspace);
    g.ldr = ldr;
    g.M = (int32_t)m;
    g.N = (int32_t)n;
    g.K = (int32_t)k;
    g.b_tile = b_tile;
    g.bf16 = out == GRKAN_BF16;
    g.cut = cut;
    return from_hip(launch_product8(p, g, stream));
}

// ------------------------------------------------------------ residual path

namespace {

bool norm_valid(grkan_norm_t n) { return n == GRKAN_NORM_NONE || n == GRKAN_NORM_LAYER || n == GRKAN_NORM_RMS; }

// Four elements at a time, aligned and whole.
bool quads(const void *p, int64_t ld, int es) { return !p || (aligned(p, 4 * es) && ld % 4 == 0); }

// What both directions check of the norms, the gate and the vectors.
grkan_status_t residual_args(int64_t rows, int64_t C, int64_t gates, int64_t gate_channels, grkan_norm_t norm,
                             grkan_norm_t post, grkan_dtype_t io, grkan_dtype_t gate_io, const void *gate) {
    if (norm != GRKAN_NORM_LAYER && norm != GRKAN_NORM_RMS) return GRKAN_ERR_INVALID_ARG;
    if (!norm_valid(post)) return GRKAN_ERR_INVALID_ARG;
    if (gate && (gate_io != GRKAN_F32 && gate_io != io)) return GRKAN_ERR_INVALID_ARG;
    if (gate && gates < 1 && rows > 0) return GRKAN_ERR_INVALID_ARG;
    return residual_shape(rows, C, gate ? gates : 0, gate_channels, io);
}

}  // namespace

extern "C" grkan_status_t grkan_residual_norm_forward(
    const void *x, const void *f, const float *weight, const float *bias, const float *scale, const void *gate,
    const float *post_weight, const float *post_bias, void *h, void *z, float *stats, int64_t rows, int64_t channels,
    int64_t ldx, int64_t ldf, int64_t gates, int64_t gate_channels, float eps, grkan_norm_t norm, grkan_norm_t post,
    grkan_dtype_t io, grkan_dtype_t gate_io, hipStream_t stream) {
    grkan_status_t st = residual_args(rows, channels, gates, gate_channels, norm, post, io, gate_io, gate);
    if (st != GRKAN_OK) return st;
    if (!(eps > 0.0f) || eps > 3.0e38f) return GRKAN_ERR_INVALID_ARG;
    if (post == GRKAN_NORM_NONE && (post_weight || post_bias)) return GRKAN_ERR_INVALID_ARG;
    if (ldx < channels || ldf < channels) return GRKAN_ERR_INVALID_ARG;
    if (ldx > kMaxStride || ldf > kMaxStride) return GRKAN_ERR_UNSUPPORTED;
    const int es = io_bytes(io), gs = io_bytes(gate_io);
    if (!aligned(x, es) || !aligned(f, es) || !aligned(h, es) || !aligned(z, es) || !aligned(stats, 4) ||
        !aligned(weight, 4) || !aligned(bias, 4) || !aligned(scale, 4) || !aligned(post_weight, 4) ||
        !aligned(post_bias, 4) || (gate && !aligned(gate, gs)))
        return GRKAN_ERR_UNSUPPORTED;
    if (rows == 0) return GRKAN_OK;
    if (!x || !f || !h || !z || !stats) return GRKAN_ERR_INVALID_ARG;
    const size_t cb = (size_t)channels * 4, out = (size_t)rows * channels * es;
    const Range rx{x, rows_bytes(rows, channels, ldx, es)};
    const Range ins[] = {{f, rows_bytes(rows, channels, ldf, es)}, {weight, cb}, {bias, cb}, {scale, cb},
                         {post_weight, cb}, {post_bias, cb},
                         {gate, gate ? (size_t)gates * gate_channels * gs : 0}, rx};
    const Range outs[] = {{stats, (size_t)rows * 4 * (post == GRKAN_NORM_NONE ? 2 : 4)}, {z, out}, {h, out}};
    const bool in_place = h == x && (ldx == channels || rows == 1);
    if (outputs_overlap(outs, 2, ins, 8) || outputs_overlap(outs, 3, ins, 7) || (!in_place && overlap(outs[2], rx)))
        return GRKAN_ERR_INVALID_ARG;
    // ---- validation done; HIP calls from here on
    ResidualArgs a{};
    residual_plan(rows, channels, gate ? gates : 0, gate_channels, post, false, &a.p);
    a.x = x;
    a.f = f;
    a.h = h;
    a.z = z;
    a.stats = stats;
    a.weight = weight;
    a.bias = bias;
    a.scale = scale;
    a.post_weight = post_weight;
    a.post_bias = post_bias;
    a.gate = gate;
    a.rows = rows;
    a.ldx = ldx;
    a.ldf = ldf;
    a.gate_rows = gate ? rows / gates : 1;
    a.gate_div = make_fastdiv((uint32_t)a.gate_rows);
    a.C = (int32_t)channels;
    a.norm = norm;
    a.post = post;
    a.gate_wide = gate && gate_channels == channels && channels > 1;
    a.gate_bf16 = gate && gate_io == GRKAN_BF16;
    a.eps = eps;
    a.vec = channels % 4 == 0 && quads(x, ldx, es) && quads(f, ldf, es) && quads(h, 0, es) && quads(z, 0, es) &&
            quads(weight, 0, 4) && quads(bias, 0, 4) && quads(scale, 0, 4) && quads(post_weight, 0, 4) &&
            quads(post_bias, 0, 4) && (!a.gate_wide || quads(gate, 0, gs));
    return from_hip(io == GRKAN_BF16 ? launch_residual_forward<uint16_t>(a, stream)
                                     : launch_residual_forward<float>(a, stream));
}

extern "C" size_t grkan_residual_norm_backward_workspace_size(int64_t rows, int64_t channels, int64_t gates,
                                                              int64_t gate_channels, grkan_norm_t post,
                                                              grkan_dtype_t io) {
    if (!norm_valid(post) || residual_shape(rows, channels, gates, gate_channels, io) != GRKAN_OK || rows == 0) return 0;
    ResidualPlan p;
    residual_plan(rows, channels, gates, gate_channels, post, true, &p);
    return p.total;
}

extern "C" grkan_status_t grkan_residual_norm_backward(
    const void *f, const void *h, const void *dh, const void *dz, const float *stats, const float *weight,
    const float *scale, const void *gate, const float *post_weight, const float *post_bias, void *dx, void *df,
    float *dscale, void *dgate, float *dweight, float *dbias, float *dpost_weight, float *dpost_bias, int64_t rows,
    int64_t channels, int64_t ldf, int64_t lddh, int64_t lddz, int64_t gates, int64_t gate_channels, grkan_norm_t norm,
    grkan_norm_t post, grkan_dtype_t io, grkan_dtype_t gate_io, void *workspace, size_t workspace_bytes,
    hipStream_t stream) {
    grkan_status_t st = residual_args(rows, channels, gates, gate_channels, norm, post, io, gate_io, gate);
    if (st != GRKAN_OK) return st;
    if (post == GRKAN_NORM_NONE && (post_weight || post_bias || dpost_weight || dpost_bias)) return GRKAN_ERR_INVALID_ARG;
    if (dgate && !gate) return GRKAN_ERR_INVALID_ARG;
    if (ldf < channels || (dh && lddh < channels) || (dz && lddz < channels)) return GRKAN_ERR_INVALID_ARG;
    if (ldf > kMaxStride || (dh && lddh > kMaxStride) || (dz && lddz > kMaxStride)) return GRKAN_ERR_UNSUPPORTED;
    const int es = io_bytes(io), gs = io_bytes(gate_io);
    if (!aligned(f, es) || !aligned(h, es) || !aligned(dh, es) || !aligned(dz, es) || !aligned(dx, es) ||
        !aligned(df, es) || !aligned(stats, 4) || !aligned(weight, 4) || !aligned(scale, 4) ||
        !aligned(post_weight, 4) || !aligned(post_bias, 4) || !aligned(dscale, 4) || !aligned(dweight, 4) ||
        !aligned(dbias, 4) || !aligned(dpost_weight, 4) || !aligned(dpost_bias, 4) ||
        (gate && (!aligned(gate, gs) || !aligned(dgate, gs))))
        return GRKAN_ERR_UNSUPPORTED;
    if (rows > 0 && (!f || !h || !stats || (!dh && !dz))) return GRKAN_ERR_INVALID_ARG;
    ResidualArgs a{};
    residual_plan(rows, channels, gate ? gates : 0, gate_channels, post, true, &a.p);
    if (rows == 0) a.p.blocks = a.p.total = 0;
    const size_t cb = (size_t)channels * 4, out = (size_t)rows * channels * es;
    const size_t gb = gate ? (size_t)gates * gate_channels * gs : 0;
    const Range rdh{dh, dh ? rows_bytes(rows, channels, lddh, es) : 0};
    const Range rdz{dz, dz ? rows_bytes(rows, channels, lddz, es) : 0};
    const size_t some = rows > 0;
    const Range ins[] = {{f, rows_bytes(rows, channels, ldf, es)}, {h, out},
                         {stats, (size_t)rows * 4 * (post == GRKAN_NORM_NONE ? 2 : 4)}, {weight, cb * some},
                         {scale, cb * some}, {post_weight, cb * some}, {post_bias, cb * some}, {gate, gb}, rdh, rdz};
    const Range outs[] = {{dscale, cb}, {dgate, gb}, {dweight, cb}, {dbias, cb}, {dpost_weight, cb}, {dpost_bias, cb},
                          {workspace, a.p.total}, {dx, out}, {df, out}};
    if (outputs_overlap(outs, 7, ins, 10) || outputs_overlap(outs, 9, ins, 8)) return GRKAN_ERR_INVALID_ARG;
    const bool dx_on = dx == dh && (lddh == channels || rows == 1), df_on = df == dz && (lddz == channels || rows == 1);
    if (overlap(outs[7], rdz) || overlap(outs[8], rdh) || (!dx_on && overlap(outs[7], rdh)) ||
        (!df_on && overlap(outs[8], rdz)))
        return GRKAN_ERR_INVALID_ARG;
    if (a.p.total && (!workspace || workspace_bytes < a.p.total)) return GRKAN_ERR_INVALID_ARG;
    if (a.p.total && !aligned(workspace, 256)) return GRKAN_ERR_UNSUPPORTED;
    // ---- validation done; HIP calls from here on
    char *ws = static_cast<char *>(workspace);
    a.f = f;
    a.h = const_cast<void *>(h);
    a.dh = dh;
    a.dz = dz;
    a.dx = dx;
    a.df = df;
    a.dgate = dgate;
    a.stats = const_cast<float *>(stats);
    a.weight = weight;
    a.scale = rows > 0 ? scale : nullptr;  // (may be what no rows leave zero)
    a.post_weight = rows > 0 ? post_weight : nullptr;
    a.post_bias = rows > 0 ? post_bias : nullptr;
    a.gate = gate;
    a.gates = gate ? gates : 0;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dscale = dscale;
    a.dpost_weight = dpost_weight;
    a.dpost_bias = dpost_bias;
    a.sums = reinterpret_cast<float *>(ws + a.p.off_sums);
    a.gate_sums = reinterpret_cast<float *>(ws + a.p.off_gate);
    a.rows = rows;
    a.ldf = ldf;
    a.lddh = lddh;
    a.lddz = lddz;
    a.gate_rows = a.gates > 0 ? rows / gates : 1;
    a.gate_div = make_fastdiv((uint32_t)(rows > 0 ? a.gate_rows : 1));
    a.C = (int32_t)channels;
    a.norm = norm;
    a.post = post;
    a.gate_wide = gate && gate_channels == channels && channels > 1;
    a.gate_bf16 = gate && gate_io == GRKAN_BF16;
    a.vec = channels % 4 == 0 && quads(f, ldf, es) && quads(h, 0, es) && quads(dh, lddh, es) && quads(dz, lddz, es) &&
            quads(dx, 0, es) && quads(df, 0, es) && quads(weight, 0, 4) && quads(scale, 0, 4) &&
            quads(post_weight, 0, 4) && quads(post_bias, 0, 4) &&
            (!a.gate_wide || (quads(gate, 0, gs) && quads(dgate, 0, gs)));
    return from_hip(io == GRKAN_BF16 ? launch_residual_backward<uint16_t>(a, stream)
                                     : launch_residual_backward<float>(a, stream));
}

// ------------------------------------------------------------ AdamW

namespace {

int by_address(const void *a, const void *b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(static_cast<const Range *>(a)->p);
    const uintptr_t y = reinterpret_cast<uintptr_t>(static_cast<const Range *>(b)->p);
    return x < y ? -1 : x > y;
}

// Whether two of the ranges share a byte (sorts them).
bool any_overlap(Range *r, int n) {
    qsort(r, n, sizeof(Range), by_address);
    for (int i = 1; i < n; ++i)
        if (overlap(r[i - 1], r[i])) return true;
    return false;
}

constexpr int64_t kAdamwMaxGroups = int64_t(1) << 23;  // workgroups of a launch

grkan_status_t adamw_tensor_ok(const grkan_adamw_tensor_t &t, int bits) {
    if (t.n < 0 || (t.io != GRKAN_F32 && t.io != GRKAN_BF16)) return GRKAN_ERR_INVALID_ARG;
    if (t.n == 0) return GRKAN_OK;
    if (!t.param || !t.grad || !t.avg || !t.sq) return GRKAN_ERR_INVALID_ARG;
    if (bits == 8 ? (!t.avg_scale || !t.sq_scale) : (t.avg_scale || t.sq_scale)) return GRKAN_ERR_INVALID_ARG;
    if (t.n > kAdamwMaxGroups * kAdamwChunk) return GRKAN_ERR_UNSUPPORTED;
    const int es = io_bytes(t.io), state = bits == 8 ? 16 : 4;
    if (!aligned(t.param, es) || !aligned(t.grad, es) || !aligned(t.master, 4) || !aligned(t.avg, state) ||
        !aligned(t.sq, state) || !aligned(t.avg_scale, 4) || !aligned(t.sq_scale, 4))
        return GRKAN_ERR_UNSUPPORTED;
    return GRKAN_OK;
}

}  // namespace

extern "C" grkan_status_t grkan_adamw_step(const grkan_adamw_tensor_t *tensors, int64_t count,
                                           const grkan_adamw_t *hyper, int32_t bits, hipStream_t stream) {
    if (count < 0 || (count > 0 && !tensors) || !hyper || (bits != 8 && bits != 32)) return GRKAN_ERR_INVALID_ARG;
    const grkan_adamw_t &y = *hyper;
    auto in01 = [](double v) { return v >= 0.0 && v < 1.0; };
    auto size = [](double v) { return v >= 0.0 && v < 1e30; };
    if (!in01(y.beta1) || !in01(y.beta2) || !size(y.eps) || !size(y.weight_decay) || (!y.lr_ptr && !size(y.lr)) ||
        (!y.step_ptr && y.step < 1))
        return GRKAN_ERR_INVALID_ARG;
    if (!aligned(y.lr_ptr, 4) || !aligned(y.step_ptr, 8) || !aligned(y.grad_scale, 4)) return GRKAN_ERR_UNSUPPORTED;
    int64_t blocks = 0;
    for (int64_t i = 0; i < count; ++i) {
        const grkan_status_t st = adamw_tensor_ok(tensors[i], bits);
        if (st != GRKAN_OK) return st;
        blocks += ceil_div(tensors[i].n, kBlock8);
    }
    if (blocks > UINT32_MAX) return GRKAN_ERR_UNSUPPORTED;
    AdamwArgs a;
    a.lr = y.lr;
    a.beta1 = y.beta1;
    a.beta2 = y.beta2;
    a.decay = y.weight_decay;
    a.step = y.step;
    a.lr_ptr = y.lr_ptr;
    a.step_ptr = y.step_ptr;
    a.grad_scale = y.grad_scale;
    a.eps = y.eps;
    a.seed = y.seed;
    if (!a.lr_ptr && !a.step_ptr) prepare_adamw(a);
    // What every workgroup reads: nothing that one of them writes.
    const Range scalars[] = {{y.lr_ptr, 4}, {y.step_ptr, 8}, {y.grad_scale, 4}};
    // First all launches' overlaps, then the launches.
    for (int pass = 0; pass < 2; ++pass) {
        int64_t groups = 0, block = 0;
        Range r[kAdamwTensors * 7];
        int n = 0;
        a.count = 0;
        auto flush = [&]() {
            grkan_status_t st = GRKAN_OK;
            if (pass == 0)
                st = any_overlap(r, n) ? GRKAN_ERR_INVALID_ARG : GRKAN_OK;
            else if (a.count > 0)
                st = from_hip(launch_adamw(a, bits, stream));
            a.count = 0;
            groups = 0;
            n = 0;
            return st;
        };
        for (int64_t i = 0; i < count; ++i) {
            const grkan_adamw_tensor_t &t = tensors[i];
            if (t.n == 0) continue;
            const int64_t wg = ceil_div(t.n, kAdamwChunk);
            if (a.count == kAdamwTensors || groups + wg > kAdamwMaxGroups) {
                const grkan_status_t st = flush();
                if (st != GRKAN_OK) return st;
            }
            const int64_t nb = ceil_div(t.n, kBlock8);
            const int es = io_bytes(t.io);
            if (pass == 0) {
                const size_t state = bits == 8 ? (size_t)nb * kBlock8 : (size_t)t.n * 4;
                const size_t sc = bits == 8 ? (size_t)nb * 4 : 0;
                const Range own[] = {{t.param, (size_t)t.n * es}, {t.grad, (size_t)t.n * es},
                                     {t.master, t.master ? (size_t)t.n * 4 : 0}, {t.avg, state}, {t.sq, state},
                                     {t.avg_scale, sc}, {t.sq_scale, sc}};
                const Range gradient = own[1];
                for (const Range &o : own) {
                    if (!o.p || !o.n) continue;
                    r[n++] = o;
                    for (const Range &s : scalars)
                        if (o.p != gradient.p && overlap(o, s)) return GRKAN_ERR_INVALID_ARG;
                }
            }
            AdamwTensor &d = a.t[a.count];
            d = AdamwTensor{t.param, t.grad, t.master, t.avg, t.sq, t.avg_scale, t.sq_scale, t.n};
            const bool vec = aligned(t.param, 4 * es) && aligned(t.grad, 4 * es) && aligned(t.master, 16) &&
                             aligned(t.avg, 16) && aligned(t.sq, 16);
            a.flags[a.count] = (uint8_t)((t.io == GRKAN_BF16 ? kAdamwBf16 : 0) | (vec ? kAdamwVec : 0));
            a.block[a.count] = (uint32_t)block;
            a.first[a.count] = (uint32_t)groups;
            groups += wg;
            block += nb;
            a.first[++a.count] = (uint32_t)groups;
        }
        const grkan_status_t st = flush();
        if (st != GRKAN_OK) return st;
    }
    return GRKAN_OK;
}
