// grkan_block_api.hip -- the C ABI of include/grkan_block.h: argument
// validation, plans and dispatch.  Plans depend on shapes, types and the
// activation alone, so results have the same bits on every device.
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

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

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

int io_bytes(grkan_dtype_t io) { return io == GRKAN_BF16 ? 2 : 4; }

bool act_valid(grkan_act_t act) {
    return act == GRKAN_ACT_NONE || act == GRKAN_ACT_SILU || act == GRKAN_ACT_GELU || act == GRKAN_ACT_RATIONAL;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int pow2_at_most(int64_t v) {
    int p = 1;
    while (2 * (int64_t)p <= v) p *= 2;
    return p;
}

// ------------------------------------------------------------ norm plans

constexpr int kTokenMaxLanes = 256, kTokenMaxAccesses = 4;
constexpr int64_t kNormWorkgroups = 2048;  // target of the looping kernels: 8 workgroups a CU

// Largest power of two <= v elements per access such that accesses that start
// at multiples of `start` columns (and then every v) lie in one activation
// group each.
int rational_vec(int v, int64_t dga, int64_t start) {
    while (v > 1 && (dga % v != 0 || start % v != 0)) v /= 2;
    return v;
}

grkan_status_t norm_plan(int64_t N, int64_t S, int64_t C, int32_t G, int32_t ng, grkan_act_t act, grkan_dtype_t io,
                         bool backward, NormPlan *p) {
    if (io != GRKAN_F32 && io != GRKAN_BF16) return GRKAN_ERR_INVALID_ARG;
    if (!act_valid(act)) return GRKAN_ERR_INVALID_ARG;
    const bool rational = act == GRKAN_ACT_RATIONAL;
    if (N < 0 || S < 0 || C < 1 || G < 1 || C % G != 0) return GRKAN_ERR_INVALID_ARG;
    if (rational && (ng < 1 || C % ng != 0)) return GRKAN_ERR_INVALID_ARG;
    if (C >= (1 << 24) || S > INT32_MAX) return GRKAN_ERR_UNSUPPORTED;
    if (N > INT32_MAX / G) return GRKAN_ERR_UNSUPPORTED;
    const int es = io_bytes(io), vmax = 16 / es;
    const int64_t D = C / G, dga = rational ? C / ng : 0;
    *p = NormPlan{};
    if (N == 0 || S == 0) return GRKAN_OK;

    // Token: T lanes of K accesses of v elements with the fewest idle places for
    // a group, then the widest accesses (16 bytes or 8), then the fewest.  The
    // backward keeps two sums, a weight and a bias per element of a lane, so it
    // takes at most 16 (768 channels in bf16: 64 lanes x 3 x 4).  A rational's
    // lanes prefer runs inside one activation group; else a run may lie in two,
    // and has to be no longer than a group for that.
    int64_t best = INT64_MAX;
    if (S == 1) {
        for (int straddle = 0; straddle <= (rational ? 1 : 0) && best == INT64_MAX; ++straddle)
            for (int v = vmax; v >= 1; v /= 2) {
                if (!rational && v < vmax / 2) break;
                for (int K = 1; K <= kTokenMaxAccesses; ++K) {
                    const int run = K * v;
                    if (backward && run > 16) break;
                    // (the forward has coefficients per access, the backward per run)
                    const int unit = backward ? run : v;
                    if (rational && !straddle && dga % D != 0 && (dga % unit != 0 || D % unit != 0)) continue;
                    if (straddle && (run > dga || run < 4)) continue;
                    int T = 1;
                    while ((int64_t)T * run < D) T *= 2;
                    if (T > (run == 1 ? 1024 : kTokenMaxLanes) || (int64_t)T * run >= best) continue;
                    best = (int64_t)T * run;
                    p->vec = v;
                    p->T = T;
                    p->K = K;
                    p->straddle = straddle != 0;
                }
            }
    }
    if (best != INT64_MAX) {
        p->kind = kNormToken;
        p->vpg = (int32_t)ceil_div(D, p->K * p->vec);  // (read for a rational only)
        p->cv = (int64_t)G * p->vpg;
        int spw = p->T <= 64 ? 256 / p->T : 1;
        while (spw % G != 0 && G % spw != 0) --spw;
        p->spw = spw;
        p->block = spw * p->T;
        // Enough workgroups to fill the GPU, walking over the samples in as
        // many rounds each as the last of them needs.
        const int64_t unit = spw < G ? G / spw : 1;  // workgroups that cover one sample
        const int64_t wanted = ceil_div(N * G, spw), cap = backward ? kNormWorkgroups / 2 : kNormWorkgroups;
        const int64_t rounds = ceil_div(wanted, cap);
        p->blocks = ceil_div(ceil_div(wanted, rounds), unit) * unit;
        p->prows = spw > G ? p->blocks : p->blocks * spw / G;
        p->lds = (size_t)p->block * ((rational ? 10 : p->vec) + 3) * 4 + 256;
    } else {
        // A slab: whole groups side by side until they make 64 bytes or more of
        // every row, if a workgroup's registers hold all rows of that.
        const int threads = backward ? 512 : 1024, regs = backward ? 8 : 16;
        int64_t gpb = ceil_div(64, D * es);
        if (gpb > G) gpb = G;
        auto vec_of = [&](int64_t groups) { return rational ? rational_vec(vmax, dga, groups * D) : vmax; };
        auto rows_of = [&](int64_t groups) {  // rows a workgroup can hold
            const int64_t tx = ceil_div(groups * D, vec_of(groups));
            return tx <= threads ? threads / tx * regs : 0;
        };
        if (S > 1 && S <= rows_of(gpb)) {
            p->kind = kNormSlab;
            // wider blocks while many workgroups remain and rows are short
            while (gpb * 2 <= G && gpb * D * es < 256 && S <= rows_of(gpb * 2) && vec_of(gpb * 2) >= vec_of(gpb) &&
                   N * ceil_div(G, gpb * 2) >= kNormWorkgroups)
                gpb *= 2;
            p->vec = vec_of(gpb);
            p->width = (int32_t)(gpb * D);
            p->ncb = (int32_t)ceil_div(G, gpb);
            p->groups = (int32_t)gpb;
            p->TX = (int32_t)ceil_div(p->width, p->vec);
            // Row lanes: 256 threads if many workgroups share a CU, all there are
            // if not; at least what the registers need.  The backward walks over the
            // samples, the next one's values on their way: two workgroups of 256
            // threads a CU (128 x 197 x 192 in 8 groups, fp32: 28.5 us; one of 512: 30.7;
            // 64 x 256 x 512 in 32: 38.7, 46.4), one of 512 for 8 rounds or more of
            // wide rows (1,024 x 197 x 192: 132 us against 183; 256 x 197 x 768, bf16: 116
            // against 200).
            const bool long_walk = backward && N * p->ncb >= 2048 && gpb * D * es >= 96;
            const int64_t want = N * p->ncb >= 1024 && !long_walk ? 256 : threads;
            int64_t ty = want / p->TX;
            if (ty < ceil_div(S, regs)) ty = ceil_div(S, regs);
            if (ty > S) ty = S;
            p->regs = (int32_t)ceil_div(S, ty);
            p->TY = (int32_t)ceil_div(S, p->regs);
            p->block = (int32_t)(ceil_div((int64_t)p->TX * p->TY, 64) * 64);
            if (!backward) {
                p->blocks = (N >= 8 ? ceil_div(N, 8) * 8 : N) * p->ncb;
            } else {
                int64_t chunks = (long_walk ? 256 : 512) / p->ncb;
                if (chunks < 1) chunks = 1;
                if (chunks > N) chunks = N;
                if (chunks >= 8) chunks = chunks / 8 * 8;
                p->chunks = chunks;
                p->blocks = chunks * p->ncb;
                p->prows = chunks;
            }
        } else {
            p->kind = kNormSplit;
            p->vec = rational ? rational_vec(vmax, dga, 0) : vmax;
            const int64_t accesses = ceil_div(C, p->vec);
            // At most 256 accesses across (128 where every column is a group, for the
            // groups' sums in LDS).
            p->ncb = (int32_t)ceil_div(accesses, D == 1 ? 128 : 256);
            p->TX = (int32_t)ceil_div(accesses, p->ncb);
            p->width = p->TX * p->vec;
            p->ncb = (int32_t)ceil_div(C, p->width);
            p->groups = (int32_t)(p->width / D + 2 < G ? p->width / D + 2 : G);
            p->parts = (int32_t)(D / p->width + 2 < p->ncb ? D / p->width + 2 : p->ncb);
            // Chunks of 4 to 32 rows a lane, about a workgroup a CU; where those
            // leave a lane of the second pass more than 2 sums to add (few
            // samples), smaller workgroups, more of them, and a step between that
            // adds (65,536 x 128 in 32 groups: 26 us against 29).
            auto chunks_of = [&](int64_t lanes, int64_t wanted) {
                int64_t ty = lanes / p->TX;
                if (ty > S) ty = S;
                p->TY = (int32_t)ty;
                p->block = (int32_t)(ceil_div((int64_t)p->TX * ty, 64) * 64);
                int64_t chunks = ceil_div(wanted, N * p->ncb);
                const int64_t most = ceil_div(S, 4 * ty), least = ceil_div(S, 32 * ty);
                if (chunks > most) chunks = most;
                if (chunks < least) chunks = least;
                p->chunk_rows = ceil_div(S, chunks);
                p->chunks = ceil_div(S, p->chunk_rows);
                p->L = pow2_at_most(p->block / p->groups < 64 ? (p->block > p->groups ? p->block / p->groups : 1) : 64);
                p->fused = ceil_div(p->chunks * p->parts, p->L) <= 2;
            };
            if (backward) {
                chunks_of(512, 512);
            } else {
                chunks_of(1024, 256);
                if (!p->fused) chunks_of(256, 1024);
            }
            p->blocks = N * p->chunks * p->ncb;
            p->prows = N * p->chunks;
        }
        p->cv = (int64_t)p->ncb * p->TX;
        p->mixed = D % p->vec != 0;
        p->L = pow2_at_most(p->block / p->groups < 64 ? (p->block > p->groups ? p->block / p->groups : 1) : 64);
        const int64_t cols_across = (int64_t)p->TX * (p->mixed ? p->vec : 1);
        p->P = pow2_at_most(p->block / cols_across < 1 ? 1 : (p->block / cols_across < 64 ? p->block / cols_across : 64));
        const size_t value = p->kind == kNormSplit ? sizeof(double) : sizeof(float);
        const size_t values = p->kind == kNormSlab && !backward ? 1 : 2;
        p->lds = value * values * ((size_t)(p->block + p->TX) * (p->mixed ? p->vec : 1) + p->groups);
        const size_t cols = (size_t)p->block * ((rational ? 10 : p->vec) + 3) * 4;
        if (backward && p->lds < cols) p->lds = cols;
    }
    p->row = 2 * C + (rational ? (p->straddle ? 20 : 10) * p->cv : 0);
    size_t at = 0;
    if (p->kind == kNormSplit) {
        p->off_stats = at;
        at += align256((size_t)N * G * p->chunks * p->parts * 16);
        p->off_means = at;
        if (backward) at += align256((size_t)N * G * 8);
    }
    p->off_partials = at;
    if (backward) at += align256((size_t)p->prows * p->row * 4);
    p->total = at;
    return GRKAN_OK;
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

constexpr int64_t kMaxWidth = int64_t(1) << 22;

grkan_status_t linear_shape(int64_t rows, int64_t d_in, int64_t d_out, int32_t n_groups, grkan_act_t act) {
    if (!act_valid(act) || rows < 0 || d_in < 1 || d_out < 1) return GRKAN_ERR_INVALID_ARG;
    if (act == GRKAN_ACT_RATIONAL && (n_groups < 1 || d_out % n_groups != 0)) return GRKAN_ERR_INVALID_ARG;
    if (rows > INT32_MAX || d_in > kMaxWidth || d_out > kMaxWidth) return GRKAN_ERR_UNSUPPORTED;
    // one thread per 8 elements of a result, one launch
    if (rows * ceil_div(d_out, 8) >= (int64_t(1) << 32) || rows * ceil_div(d_in, 8) >= (int64_t(1) << 32) ||
        d_in * ceil_div(d_out, 8) >= (int64_t(1) << 32))
        return GRKAN_ERR_UNSUPPORTED;
    return GRKAN_OK;
}

bool chunks_aligned(const void *p, int64_t ld, int64_t width) {
    return aligned(p, 16) && ld % 8 == 0 && width % 8 == 0;
}

int64_t act_group(int64_t d_out, int32_t n_groups, grkan_act_t act) {
    return act == GRKAN_ACT_RATIONAL ? d_out / n_groups : 8;
}

// Plans and workspace do not depend on alignment.
struct LinearBwdPlan {
    SlopePlan slope;
    ProductPlan dx, dw;
    size_t off_slope, off_sums, total;
};

void linear_bwd_plan(int64_t rows, int64_t d_in, int64_t d_out, int32_t n_groups, grkan_act_t act, LinearBwdPlan *p) {
    p->slope = plan_slope(rows, d_out, act, act_group(d_out, n_groups, act));
    p->dx = plan_product(kFormDx, rows, d_in, d_out, true, GRKAN_ACT_NONE, 8);
    p->dw = plan_product(kFormDw, d_out, d_in, rows, true, GRKAN_ACT_NONE, 8);
    p->off_slope = act == GRKAN_ACT_NONE ? 0 : align256((size_t)rows * d_out * 2);
    p->off_sums = p->off_slope + align256(p->slope.partials_bytes);
    const size_t sums = p->dx.partials_bytes > p->dw.partials_bytes ? p->dx.partials_bytes : p->dw.partials_bytes;
    p->total = p->off_sums + align256(sums);
}

__global__ __launch_bounds__(256) void grkan_zero16_kernel(uint16_t *p, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = 0;
}

}  // namespace

extern "C" size_t grkan_linear_act_forward_workspace_size(int64_t rows, int64_t d_in, int64_t d_out,
                                                          int32_t n_groups, grkan_act_t act) {
    if (linear_shape(rows, d_in, d_out, n_groups, act) != GRKAN_OK || rows == 0) return 0;
    return align256(
        plan_product(kFormForward, rows, d_out, d_in, true, act, act_group(d_out, n_groups, act)).partials_bytes);
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
    LinearBwdPlan p;
    linear_bwd_plan(rows, d_in, d_out, n_groups, act, &p);
    return p.total;
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
        linear_bwd_plan(rows, d_in, d_out, n_groups, act, &p);
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
            hipLaunchKernelGGL(grkan_zero16_kernel, dim3((unsigned)ceil_div(n, 256)), dim3(256), 0, stream,
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
    const bool q_ok = chunks_aligned(dpre, ldp, d_out);
    ProductArgs a{};
    a.partials = reinterpret_cast<float *>(ws + p.off_sums);
    a.q = Operand{dpre, ldp};
    if (dx) {
        p.dx.aligned = q_ok && chunks_aligned(W, d_in, d_in);
        a.p = Operand{W, d_in};
        a.M = (int32_t)rows;
        a.N = (int32_t)d_in;
        a.K = (int32_t)d_out;
        a.e.z = dx;
        st = from_hip(launch_product(kFormDx, p.dx, a, stream));
        if (st != GRKAN_OK) return st;
    }
    if (dW) {
        p.dw.aligned = q_ok && chunks_aligned(x, ldx, d_in);
        a.p = Operand{x, ldx};
        a.M = (int32_t)d_out;
        a.N = (int32_t)d_in;
        a.K = (int32_t)rows;
        a.e.z = dW;
        return from_hip(launch_product(kFormDw, p.dw, a, stream));
    }
    return GRKAN_OK;
}
