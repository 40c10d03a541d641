// grkan_block_api.hip -- the C ABI of include/grkan_block.h: argument
// validation and dispatch.  Plans depend on shapes, types, the activation and,
// for the products, on whether the operands' 16-byte chunks are aligned and whole,
// so results have the same bits on every device.
#include <limits.h>
#include <stdint.h>

#include "grkan_block.h"
#include "grkan_launch.h"
#include "grkan_linear.h"
#include "grkan_norm.h"

using namespace grkan;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A byte range an argument covers; empty if absent.
struct Range {
    const void *p;
    size_t n;
};

bool overlap(const Range &a, const Range &b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

// Every output apart from every other argument.
bool outputs_overlap(const Range *outs, int no, const Range *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return true;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return true;
    }
    return false;
}

grkan_status_t from_hip(hipError_t e) { return e == hipSuccess ? GRKAN_OK : GRKAN_ERR_HIP; }

__global__ __launch_bounds__(256) void grkan_norm_empty_kernel(float *mean, float *rstd, int64_t n, float value) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    mean[i] = 0.0f;
    rstd[i] = value;
}

// Statistics of samples without positions.
hipError_t launch_norm_empty(const NormArgs &a, hipStream_t s) {
    const int64_t n = a.N * a.G;
    hipLaunchKernelGGL(grkan_norm_empty_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a.mean, a.rstd, n,
                       1.0f / sqrtf(a.eps));
    return hipGetLastError();
}

// Elements from the first to the last of a strided [N][S][C] tensor, or -1 if
// that does not fit an address.
int64_t span(int64_t N, int64_t S, int64_t C, int64_t sample, int64_t row) {
    if (N == 0 || S == 0) return 0;
    __int128 v = (__int128)(N - 1) * sample + (__int128)(S - 1) * row + C;
    return v > INT64_MAX / 8 ? -1 : (int64_t)v;
}

grkan_status_t strides_ok(int64_t N, int64_t S, int64_t C, int64_t sample, int64_t row) {
    if (row < C || sample < 0) return GRKAN_ERR_INVALID_ARG;
    if (span(N, S, C, sample, row) < 0) return GRKAN_ERR_INVALID_ARG;
    return GRKAN_OK;
}

bool dense(int64_t N, int64_t S, int64_t C, int64_t sample, int64_t row) {
    return (row == C || S <= 1) && (sample == S * C || N <= 1);
}

// What both directions check of the coefficients.
grkan_status_t coefs_ok(const float *A, const float *B, grkan_act_t act) {
    if (act != GRKAN_ACT_RATIONAL) return A || B ? GRKAN_ERR_INVALID_ARG : GRKAN_OK;
    if (!A || !B) return GRKAN_ERR_INVALID_ARG;
    return aligned(A, 4) && aligned(B, 4) ? GRKAN_OK : GRKAN_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" size_t grkan_group_norm_forward_workspace_size(int64_t samples, int64_t positions, int64_t channels,
                                                          int32_t norm_groups, int32_t n_groups, grkan_act_t act,
                                                          grkan_dtype_t io) {
    NormPlan p;
    return norm_plan(samples, positions, channels, norm_groups, n_groups, act, io, false, &p) == GRKAN_OK ? p.total
                                                                                                          : 0;
}

extern "C" size_t grkan_group_norm_backward_workspace_size(int64_t samples, int64_t positions, int64_t channels,
                                                           int32_t norm_groups, int32_t n_groups, grkan_act_t act,
                                                           grkan_dtype_t io) {
    NormPlan p;
    return norm_plan(samples, positions, channels, norm_groups, n_groups, act, io, true, &p) == GRKAN_OK ? p.total
                                                                                                         : 0;
}

extern "C" grkan_status_t grkan_group_norm_forward(const void *x, void *y, float *mean, float *rstd,
                                                   const float *weight, const float *bias, const float *A,
                                                   const float *B, int64_t samples, int64_t positions,
                                                   int64_t channels, int64_t x_sample, int64_t x_row,
                                                   int32_t norm_groups, int32_t n_groups, float eps, grkan_act_t act,
                                                   grkan_dtype_t io, void *workspace, size_t workspace_bytes,
                                                   hipStream_t stream) {
    NormArgs a{};
    grkan_status_t st = norm_plan(samples, positions, channels, norm_groups, n_groups, act, io, false, &a.p);
    if (st != GRKAN_OK) return st;
    if (!(eps > 0.0f) || eps > 3.0e38f) return GRKAN_ERR_INVALID_ARG;
    if ((st = coefs_ok(A, B, act)) != GRKAN_OK) return st;
    if ((st = strides_ok(samples, positions, channels, x_sample, x_row)) != GRKAN_OK) return st;
    const int es = io_bytes(io);
    if (!aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(x, es) ||
        !aligned(y, es))
        return GRKAN_ERR_UNSUPPORTED;
    if (samples == 0) return GRKAN_OK;
    if (!mean || !rstd) return GRKAN_ERR_INVALID_ARG;
    if (positions > 0 && (!x || !y)) return GRKAN_ERR_INVALID_ARG;
    const size_t sg = (size_t)samples * norm_groups * 4;
    const bool rational = act == GRKAN_ACT_RATIONAL;
    const Range rx{x, (size_t)span(samples, positions, channels, x_sample, x_row) * es};
    const Range ry{y, (size_t)samples * positions * channels * es};
    const Range ins[] = {{weight, (size_t)channels * 4}, {bias, (size_t)channels * 4},
                         {A, rational ? (size_t)n_groups * 24 : 0}, {B, rational ? (size_t)n_groups * 16 : 0}, rx};
    const Range outs[] = {{mean, sg}, {rstd, sg}, {workspace, a.p.total}, ry};
    const bool in_place = x == y && dense(samples, positions, channels, x_sample, x_row);
    if (outputs_overlap(outs, 3, ins, 5) || outputs_overlap(outs, 4, ins, 4) || (!in_place && overlap(rx, ry)))
        return GRKAN_ERR_INVALID_ARG;
    if (a.p.total && (!workspace || workspace_bytes < a.p.total)) return GRKAN_ERR_INVALID_ARG;
    if (a.p.total && !aligned(workspace, 256)) return GRKAN_ERR_UNSUPPORTED;
    // ---- validation done; HIP calls from here on
    a.x = x;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.w = weight;
    a.b = bias;
    a.A = A;
    a.B = B;
    a.N = samples;
    a.S = positions;
    a.xs = x_sample;
    a.xr = x_row;
    a.C = (int32_t)channels;
    a.G = norm_groups;
    a.D = (int32_t)(channels / norm_groups);
    a.ng = n_groups;
    a.dga = rational ? (int32_t)(channels / n_groups) : 1;
    a.act = act;
    a.eps = eps;
    if (positions == 0) return from_hip(launch_norm_empty(a, stream));
    a.stats = reinterpret_cast<double *>(static_cast<char *>(workspace) + a.p.off_stats);
    return from_hip(io == GRKAN_BF16 ? launch_norm_forward<bf16io>(a, stream) : launch_norm_forward<float>(a, stream));
}

extern "C" grkan_status_t grkan_group_norm_backward(
    const void *x, const void *dy, const float *mean, const float *rstd, const float *weight, const float *bias,
    const float *A, const float *B, void *dx, float *dweight, float *dbias, float *dA, float *dB, int64_t samples,
    int64_t positions, int64_t channels, int64_t x_sample, int64_t x_row, int64_t dy_sample, int64_t dy_row,
    int32_t norm_groups, int32_t n_groups, grkan_act_t act, grkan_dtype_t io, void *workspace,
    size_t workspace_bytes, hipStream_t stream) {
    NormArgs a{};
    grkan_status_t st = norm_plan(samples, positions, channels, norm_groups, n_groups, act, io, true, &a.p);
    if (st != GRKAN_OK) return st;
    if ((st = coefs_ok(A, B, act)) != GRKAN_OK) return st;
    const bool rational = act == GRKAN_ACT_RATIONAL;
    if (rational ? (!dA || !dB) : (dA || dB)) return GRKAN_ERR_INVALID_ARG;
    if ((st = strides_ok(samples, positions, channels, x_sample, x_row)) != GRKAN_OK) return st;
    if ((st = strides_ok(samples, positions, channels, dy_sample, dy_row)) != GRKAN_OK) return st;
    const int es = io_bytes(io);
    if (!aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) ||
        !aligned(dbias, 4) || !aligned(dA, 4) || !aligned(dB, 4) || !aligned(x, es) || !aligned(dy, es) ||
        !aligned(dx, es))
        return GRKAN_ERR_UNSUPPORTED;
    const bool empty = samples == 0 || positions == 0;
    if (!empty && (!x || !dy || !dx || !mean || !rstd)) return GRKAN_ERR_INVALID_ARG;
    const size_t sg = (size_t)samples * norm_groups * 4, cb = (size_t)channels * 4;
    const size_t ab = rational ? (size_t)n_groups * 24 : 0, bb = rational ? (size_t)n_groups * 16 : 0;
    const Range rx{x, (size_t)span(samples, positions, channels, x_sample, x_row) * es};
    const Range rdy{dy, (size_t)span(samples, positions, channels, dy_sample, dy_row) * es};
    const Range rdx{dx, (size_t)samples * positions * channels * es};
    const Range ins[] = {{mean, sg}, {rstd, sg}, {weight, cb}, {bias, cb}, {A, ab}, {B, bb}, rx, rdy};
    const Range outs[] = {{dweight, cb}, {dbias, cb}, {dA, ab}, {dB, bb}, {workspace, a.p.total}, rdx};
    if (outputs_overlap(outs, 5, ins, 8) || outputs_overlap(outs, 6, ins, 6)) return GRKAN_ERR_INVALID_ARG;
    const bool on_x = dx == x && dense(samples, positions, channels, x_sample, x_row);
    const bool on_dy = dx == dy && dense(samples, positions, channels, dy_sample, dy_row);
    if ((!on_x && overlap(rdx, rx)) || (!on_dy && overlap(rdx, rdy))) return GRKAN_ERR_INVALID_ARG;
    if (a.p.total && (!workspace || workspace_bytes < a.p.total)) return GRKAN_ERR_INVALID_ARG;
    if (a.p.total && !aligned(workspace, 256)) return GRKAN_ERR_UNSUPPORTED;
    // ---- validation done; HIP calls from here on
    a.x = x;
    a.dy = dy;
    a.y = dx;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.w = weight;
    a.b = bias;
    a.A = A;
    a.B = B;
    a.dw = dweight;
    a.db = dbias;
    a.dA = dA;
    a.dB = dB;
    a.N = samples;
    a.S = positions;
    a.xs = x_sample;
    a.xr = x_row;
    a.ds = dy_sample;
    a.dr = dy_row;
    a.C = (int32_t)channels;
    a.G = norm_groups;
    a.D = (int32_t)(channels / norm_groups);
    a.ng = n_groups;
    a.dga = rational ? (int32_t)(channels / n_groups) : 1;
    a.act = act;
    if (empty) {
        hipError_t e = hipSuccess;
        if (dweight) e = launch_zero(dweight, dweight, channels, 0, stream);
        if (e == hipSuccess && dbias) e = launch_zero(dbias, dbias, channels, 0, stream);
        if (e == hipSuccess && rational) e = launch_zero(dA, dB, (int64_t)n_groups * 6, (int64_t)n_groups * 4, stream);
        return from_hip(e);
    }
    char *ws = static_cast<char *>(workspace);
    a.stats = reinterpret_cast<double *>(ws + a.p.off_stats);
    a.means = reinterpret_cast<float *>(ws + a.p.off_means);
    a.partials = reinterpret_cast<float *>(ws + a.p.off_partials);
    return from_hip(io == GRKAN_BF16 ? launch_norm_backward<bf16io>(a, stream)
                                     : launch_norm_backward<float>(a, stream));
}

// ------------------------------------------------------------ linear map

namespace {

bool chunks_aligned(const void *p, int64_t ld, int64_t width) {
    return aligned(p, 16) && ld % 8 == 0 && width % 8 == 0;
}

__global__ __launch_bounds__(256) void grkan_zero16_kernel(uint16_t *p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

}  // namespace

extern "C" size_t grkan_linear_act_forward_workspace_size(int64_t rows, int64_t d_in, int64_t d_out,
                                                          int32_t n_groups, grkan_act_t act) {
    if (linear_shape(rows, d_in, d_out, n_groups, act) != GRKAN_OK || rows == 0) return 0;
    return linear_fwd_bytes(rows, d_in, d_out, n_groups, act);
}

extern "C" grkan_status_t grkan_linear_act_forward(const void *x, const void *W, const float *bias,
                                                   const void *residual, const float *A, const float *B, void *z,
                                                   void *pre, int64_t rows, int64_t d_in, int64_t d_out, int64_t ldx,
                                                   int64_t ldr, int32_t n_groups, grkan_act_t act, void *workspace,
                                                   size_t workspace_bytes, hipStream_t stream) {
    grkan_status_t st = linear_shape(rows, d_in, d_out, n_groups, act);
    if (st != GRKAN_OK) return st;
    if (ldx < d_in || (residual && ldr < d_out)) return GRKAN_ERR_INVALID_ARG;
    if (ldx > kMaxWidth || (residual && ldr > kMaxWidth)) return GRKAN_ERR_UNSUPPORTED;
    if ((st = coefs_ok(A, B, act)) != GRKAN_OK) return st;
    if (!W) return GRKAN_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(W, 2) || !aligned(residual, 2) || !aligned(z, 2) || !aligned(pre, 2) ||
        !aligned(bias, 4))
        return GRKAN_ERR_UNSUPPORTED;
    if (rows == 0) return GRKAN_OK;
    if (!x || !z) return GRKAN_ERR_INVALID_ARG;
    const int64_t dga = act_group(d_out, n_groups, act);
    const bool al = chunks_aligned(x, ldx, d_in) && chunks_aligned(W, d_in, d_in);
    const ProductPlan p = plan_product(kFormForward, rows, d_out, d_in, al, act, dga);
    const size_t need = align256(p.partials_bytes), zb = (size_t)rows * d_out * 2;
    const bool rational = act == GRKAN_ACT_RATIONAL;
    const Range rr{residual, residual ? (size_t)((rows - 1) * ldr + d_out) * 2 : 0};
    const Range ins[] = {{x, (size_t)((rows - 1) * ldx + d_in) * 2}, {W, (size_t)d_out * d_in * 2},
                         {bias, (size_t)d_out * 4}, {A, rational ? (size_t)n_groups * 24 : 0},
                         {B, rational ? (size_t)n_groups * 16 : 0}, rr};
    const Range outs[] = {{workspace, need}, {pre, zb}, {z, zb}};
    const bool in_place = residual == z && ldr == d_out;
    if (outputs_overlap(outs, 2, ins, 6) || outputs_overlap(outs, 3, ins, 5) || (!in_place && overlap(outs[2], rr)))
        return GRKAN_ERR_INVALID_ARG;
    if (need && (!workspace || workspace_bytes < need)) return GRKAN_ERR_INVALID_ARG;
    if (need && !aligned(workspace, 256)) return GRKAN_ERR_UNSUPPORTED;
    // ---- validation done; HIP calls from here on
    ProductArgs a{};
    a.q = Operand{x, ldx};
    a.p = Operand{W, d_in};
    a.M = (int32_t)rows;
    a.N = (int32_t)d_out;
    a.K = (int32_t)d_in;
    a.partials = static_cast<float *>(workspace);
    a.e = Epilogue{bias, A, B, residual, pre, z, ldr, act, (int32_t)dga};
    return from_hip(launch_product(kFormForward, p, a, stream));
}

extern "C" size_t grkan_linear_act_backward_workspace_size(int64_t rows, int64_t d_in, int64_t d_out,
                                                           int32_t n_groups, grkan_act_t act) {
    if (linear_shape(rows, d_in, d_out, n_groups, act) != GRKAN_OK || rows == 0) return 0;
    return linear_bwd_bytes(rows, d_in, d_out, n_groups, act);
}

extern "C" grkan_status_t grkan_linear_act_backward(const void *x, const void *W, const void *dz, const void *pre,
                                                    const float *A, const float *B, void *dx, void *dW, float *dbias,
                                                    float *dA, float *dB, int64_t rows, int64_t d_in, int64_t d_out,
                                                    int64_t ldx, int64_t lddz, int32_t n_groups, grkan_act_t act,
                                                    void *workspace, size_t workspace_bytes, hipStream_t stream) {
    grkan_status_t st = linear_shape(rows, d_in, d_out, n_groups, act);
    if (st != GRKAN_OK) return st;
    if (ldx < d_in || lddz < d_out) return GRKAN_ERR_INVALID_ARG;
    if (ldx > kMaxWidth || lddz > kMaxWidth) return GRKAN_ERR_UNSUPPORTED;
    if ((st = coefs_ok(A, B, act)) != GRKAN_OK) return st;
    const bool rational = act == GRKAN_ACT_RATIONAL;
    if (rational ? (!dA || !dB) : (dA || dB)) return GRKAN_ERR_INVALID_ARG;
    if (!aligned(x, 2) || !aligned(W, 2) || !aligned(dz, 2) || !aligned(pre, 2) || !aligned(dx, 2) || !aligned(dW, 2) ||
        !aligned(dbias, 4) || !aligned(dA, 4) || !aligned(dB, 4))
        return GRKAN_ERR_UNSUPPORTED;
    LinearBwdPlan p{};
    if (rows > 0) {
        if (!x || !W || !dz || (act != GRKAN_ACT_NONE && !pre)) return GRKAN_ERR_INVALID_ARG;
        // dpre: dz itself, or dense at the workspace's 256-byte aligned start
        const bool q_ok = act == GRKAN_ACT_NONE ? chunks_aligned(dz, lddz, d_out) : d_out % 8 == 0;
        linear_bwd_plan(rows, d_in, d_out, n_groups, act, q_ok && chunks_aligned(W, d_in, d_in),
                        q_ok && chunks_aligned(x, ldx, d_in), &p);
    }
    const size_t ab = rational ? (size_t)n_groups * 24 : 0, bb = rational ? (size_t)n_groups * 16 : 0;
    const size_t wb = (size_t)d_out * d_in * 2;
    const size_t rows1 = rows > 0 ? (size_t)rows - 1 : 0, some = rows > 0;
    const Range ins[] = {{x, (rows1 * ldx + d_in) * 2 * some}, {W, wb * some}, {dz, (rows1 * lddz + d_out) * 2 * some},
                         {pre, act == GRKAN_ACT_NONE ? 0 : (size_t)rows * d_out * 2}, {A, ab}, {B, bb}};
    const Range outs[] = {{dx, (size_t)rows * d_in * 2}, {dW, wb}, {dbias, (size_t)d_out * 4}, {dA, ab}, {dB, bb},
                          {workspace, p.total}};
    if (outputs_overlap(outs, 6, ins, 6)) return GRKAN_ERR_INVALID_ARG;
    if (p.total && (!workspace || workspace_bytes < p.total)) return GRKAN_ERR_INVALID_ARG;
    if (p.total && !aligned(workspace, 256)) return GRKAN_ERR_UNSUPPORTED;
    // ---- validation done; HIP calls from here on
    if (rows == 0) {
        hipError_t e = hipSuccess;
        if (dW) {
            const int64_t n = d_out * d_in;
            const int64_t blocks = ceil_div(n, 256);
            hipLaunchKernelGGL(grkan_zero16_kernel, dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), dim3(256), 0, stream,
                               static_cast<uint16_t *>(dW), n);
            e = hipGetLastError();
        }
        if (e == hipSuccess && dbias) e = launch_zero(dbias, dbias, d_out, 0, stream);
        if (e == hipSuccess && rational) e = launch_zero(dA, dB, (int64_t)n_groups * 6, (int64_t)n_groups * 4, stream);
        return from_hip(e);
    }
    char *ws = static_cast<char *>(workspace);
    const void *dpre = act == GRKAN_ACT_NONE ? dz : ws;
    const int64_t ldp = act == GRKAN_ACT_NONE ? lddz : d_out;
    if (act != GRKAN_ACT_NONE || dbias) {
        SlopeArgs s{};
        s.dz = dz;
        s.pre = pre;
        s.dpre = ws;
        s.A = A;
        s.B = B;
        s.dbias = dbias;
        s.dA = dA;
        s.dB = dB;
        s.partials = reinterpret_cast<float *>(ws + p.off_slope);
        s.rows = rows;
        s.lddz = lddz;
        s.ldp = ldp;
        s.N = (int32_t)d_out;
        s.act = act;
        s.ng = n_groups;
        s.dga = (int32_t)act_group(d_out, n_groups, act);
        s.vec = p.slope.vec;
        s.vpr = p.slope.vpr;
        s.chunks = p.slope.chunks;
        s.chunk_rows = p.slope.chunk_rows;
        st = from_hip(launch_slope(s, stream));
        if (st != GRKAN_OK) return st;
    }
    ProductArgs a{};
    a.partials = reinterpret_cast<float *>(ws + p.off_sums);
    a.q = Operand{dpre, ldp};
    if (dx) {
        a.p = Operand{W, d_in};
        a.M = (int32_t)rows;
        a.N = (int32_t)d_in;
        a.K = (int32_t)d_out;
        a.e.z = dx;
        st = from_hip(launch_product(kFormDx, p.dx, a, stream));
        if (st != GRKAN_OK) return st;
    }
    if (dW) {
        a.p = Operand{x, ldx};
        a.M = (int32_t)d_out;
        a.N = (int32_t)d_in;
        a.K = (int32_t)rows;
        a.e.z = dW;
        return from_hip(launch_product(kFormDw, p.dw, a, stream));
    }
    return GRKAN_OK;
}
