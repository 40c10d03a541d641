"""fp64 definitions of the operators of include/grkan_train.h and the error bounds their evaluation is held to.

Roundings (u = 2^-24) as in block_ref.py: a mean or sum in fp32 costs 64 u times the sum of the absolute values
(runs of at most ~40 values a lane or wave, a tree above them), an elementary step u of its result, a reciprocal
root 4 u; a bf16 result is rounded once.  What each operator adds to this stands at its function."""
from __future__ import annotations

import math

import torch

from block_ref import SUM, U, activation, check, per_channel, rounding  # noqa: F401

BLOCK = 128
F8 = torch.float8_e4m3fn


def ceil(n, d):
    return -(-n // d)


# ---------------------------------------------------------------- e4m3

def powers_of_two(device):
    """2^-126 .. 2^127, exact (a GPU's exp2 and pow need not be)."""
    return torch.tensor([math.ldexp(1.0, e) for e in range(-126, 128)], dtype=torch.float64).to(device)


def binade(a):
    """The largest power of two at most a, for a within 2^-126 .. 2^127."""
    powers = powers_of_two(a.device)
    return powers[torch.searchsorted(powers, a.double().contiguous(), right=True) - 1]


def scale_of(amax):
    """The smallest 2^e >= amax / 448, e >= -126; 1 for 0: by comparison with every power (fp64)."""
    powers = powers_of_two(amax.device)
    at = torch.searchsorted(448.0 * powers, amax.double().contiguous())
    return torch.where(amax == 0, 1.0, powers[at.clamp_max(253)])


def e4m3_values():
    """Every finite value >= 0 of the type, ascending (code = index)."""
    return torch.tensor([(2.0 ** (max(c >> 3, 1) - 7)) * ((c & 7) / 8 + (1 if c >> 3 else 0)) for c in range(127)],
                        dtype=torch.float64)


def to_e4m3(y):
    """fp64 y, |y| <= 448 or not finite, rounded to the nearest value of the type, halves to the even code; NaN
    for what is not finite."""
    v = e4m3_values().to(y.device)
    a = torch.where(y.isfinite(), y.abs(), 0.0)
    hi = torch.searchsorted(v, a.contiguous()).clamp_max(126)
    lo = (hi - 1).clamp_min(0)
    down, up = a - v[lo], v[hi] - a
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = torch.where(a >= v[hi], hi, code)
    return torch.where(y.isfinite(), v[code] * torch.where(y < 0, -1.0, 1.0), torch.nan)


def quantized(x, tile=False):
    """(values of the codes, scales) in fp64 of x [rows, cols]."""
    rows, cols = x.shape
    rb, cb = ceil(rows, BLOCK) if tile else rows, ceil(cols, BLOCK)
    pad = torch.zeros((rb * (BLOCK if tile else 1), cb * BLOCK), dtype=torch.float64, device=x.device)
    pad[:rows, :cols] = x.double()
    v = pad.view(rb, BLOCK if tile else 1, cb, BLOCK)
    s = scale_of(torch.where(v.isfinite(), v.abs(), 0.0).amax(dim=(1, 3)))
    q = to_e4m3((v / s[:, None, :, None]).view(pad.shape))
    return q[:rows, :cols], s


def values(codes, scale, tile=False):
    """What codes and scales stand for, fp64."""
    s = scale.double().repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]
    if tile:
        s = s.repeat_interleave(BLOCK, 0)[:codes.shape[0]]
    return codes.float().double() * s


def matmul(a, a_scale, b, b_scale, tile, bias=None, residual=None, dtype=torch.bfloat16):
    """(value, bound).  fp32 results: exact products, K of them summed in fp32 and scaled, (K + 12) u of the sum of
    their absolute values.  bf16: besides, the products of each 8 values of k are cut off, towards zero, at 2^-13
    of the power of two of the largest among them: 7 of the 8 by less than 2^-13 of the largest product each."""
    k = a.shape[1]
    av, bv = values(a, a_scale), values(b, b_scale, tile)
    v, mag = av @ bv.t(), av.abs() @ bv.abs().t()
    err = (k + 12) * U * mag
    if dtype == torch.bfloat16:
        for at in range(0, k, 8):
            p = (av[:, None, at:at + 8] * bv[None, :, at:at + 8]).abs().amax(-1)
            err += 7 * 2.0 ** -13 * p
    for t in (bias, residual):
        if t is not None:
            v = v + t.double()
            err = err + U * (v.abs() + t.double().abs())
    return v, err + rounding(v.abs() + err, dtype)


# ---------------------------------------------------------------- residual path

EPS = 1e-5


def moments(v, ev, kind):
    """(mean, rstd and their bounds) of rows v with error bounds ev: the variance moves by the values' errors and
    its own sum's."""
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    em = (SUM * v.abs() + ev).mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(mean)
    d = v - mean
    var = d.square().mean(1, keepdim=True)
    evar = SUM * var + (2 * d.abs() * (ev + em + U * d.abs()) + (ev + em).square()).mean(1, keepdim=True)
    rstd = (var + EPS) ** -0.5
    return mean, rstd, em, rstd * (0.5 * evar / (var + EPS) * 1.01 + 4 * U)


def norm(v, ev, kind, w, b):
    """(norm of v, bound, stats and bounds)."""
    mean, rstd, em, er = moments(v, ev, kind)
    d, ed = v - mean, ev + em + U * (v - mean).abs()
    y, ey = d * rstd, ed * rstd + d.abs() * er + 2 * U * (d * rstd).abs()
    if w is not None:
        y, ey = y * w.double(), ey * w.double().abs() + U * (y * w.double()).abs()
    if b is not None:
        y, ey = y + b.double(), ey + U * ((y + b.double()).abs() + y.abs())
    return y, ey, (mean, rstd, em + U * mean.abs(), er + U * rstd)


def rows_of(gate, shape):
    """The gate at each row [rows, 1 or channels], fp64."""
    if gate is None:
        return torch.ones((1, 1), dtype=torch.float64, device="cpu")
    g = gate.double()
    return g.expand(*shape[:-1], g.shape[-1]).reshape(-1, g.shape[-1])


def residual_forward(x, f, kind, weight, bias, scale, gate, post, post_weight, post_bias):
    """{name: (value, bound)} of h, z, stats."""
    shape, c = x.shape, x.shape[-1]
    u, xd = f.double().reshape(-1, c), x.double().reshape(-1, c)
    eu, stats = torch.zeros_like(u), []
    if post != "none":
        u, eu, s = norm(u, eu, post, post_weight, post_bias)
        stats = [s]
    k = rows_of(gate, shape).to(x.device) * (1.0 if scale is None else scale.double())
    h = xd + k * u
    eh = k.abs() * eu + 4 * U * (xd.abs() + (k * u).abs())
    z, ez, s = norm(h, eh, kind, weight, bias)
    stats = [s] + stats
    return {"h": (h.view(shape), (eh + rounding(h.abs() + eh, x.dtype)).view(shape)),
            "z": (z.view(shape), (ez + rounding(z.abs() + ez, x.dtype)).view(shape)),
            "stats": (torch.cat([t.reshape(1, -1) for s in stats for t in s[:2]]),
                      torch.cat([t.reshape(1, -1) for s in stats for t in s[2:]]))}


def norm_backward(t, et, xh, exh, rstd, kind):
    m2, e2 = (t * xh).mean(1, keepdim=True), (et * xh.abs() + t.abs() * exh + SUM * (t * xh).abs()).mean(1, keepdim=True)
    m1 = t.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(m2)
    e1 = (et + SUM * t.abs()).mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(m2)
    v = rstd * (t - m1 - xh * m2)
    return v, rstd * (et + e1 + exh * m2.abs() + xh.abs() * e2 + 5 * U * (t.abs() + m1.abs() + (xh * m2).abs()))


def residual_backward(f, h, dh, dz, stats, kind, weight, bias, scale, gate, post, post_weight, post_bias):
    """{name: (value, bound)} of every gradient, from the given fp32 statistics."""
    shape, c = h.shape, h.shape[-1]
    dev = h.device
    st = stats.double()[:, :, None]
    one = torch.ones(c, dtype=torch.float64, device=dev)
    zero = torch.zeros((h.numel() // c, c), dtype=torch.float64, device=dev)
    w = one if weight is None else weight.double()
    s = one if scale is None else scale.double()
    g = rows_of(gate, shape).to(dev)
    z = zero if dz is None else dz.double().reshape(-1, c)
    xh = (h.double().reshape(-1, c) - st[0]) * st[1]
    exh = 3 * U * xh.abs()
    t = z * w
    d, ed = norm_backward(t, U * t.abs(), xh, exh, st[1], kind)
    if dh is not None:
        d = d + dh.double().reshape(-1, c)
    ed = ed + U * d.abs()
    out = {"dx": (d.view(shape), (ed + rounding(d.abs() + ed, h.dtype)).view(shape)),
           "dweight": ((z * xh).sum(0), (z.abs() * exh).sum(0) + SUM * (z * xh).abs().sum(0))}
    if bias is not None:
        out["dbias"] = (z.sum(0), SUM * z.abs().sum(0))
    u, eu = f.double().reshape(-1, c), zero
    if post != "none":
        fh = (u - st[2]) * st[3]
        efh = 3 * U * fh.abs()
        pw = one if post_weight is None else post_weight.double()
        u, eu = fh * pw, efh * pw.abs() + U * (fh * pw).abs()
        if post_bias is not None:
            u, eu = u + post_bias.double(), eu + U * ((u + post_bias.double()).abs() + u.abs())

    def product(*terms):
        v, e = torch.ones_like(d), torch.zeros_like(d)
        for a, ea in terms:
            v, e = v * a, e * a.abs() + (v * ea).abs() + U * (v * a).abs()
        return v, e

    v, e = product((d, ed), (u, eu), (g, zero))
    out["dscale"] = (v.sum(0), e.sum(0) + SUM * v.abs().sum(0))
    if gate is not None:
        v, e = product((d, ed), (u, eu), (s, zero))
        e = e + SUM * v.abs()
        v, e = v.view(shape), e.view(shape)
        over = [k for k in range(h.dim()) if gate.shape[k] == 1 and shape[k] > 1]
        if over:
            v, e = v.sum(over, keepdim=True), e.sum(over, keepdim=True)
        out["dgate"] = (v, e + rounding(v.abs() + e, gate.dtype))
    b, eb = product((d, ed), (s, zero), (g, zero))
    if post != "none":
        v, e = product((b, eb), (fh, efh))
        if post_weight is not None:
            out["dpost_weight"] = (v.sum(0), e.sum(0) + SUM * v.abs().sum(0))
        if post_bias is not None:
            out["dpost_bias"] = (b.sum(0), eb.sum(0) + SUM * b.abs().sum(0))
        b, eb = norm_backward(b * pw, eb * pw.abs() + U * (b * pw).abs(), fh, efh, st[3], post)
    out["df"] = (b.view(shape), (eb + rounding(b.abs() + eb, h.dtype)).view(shape))
    return out


# ---------------------------------------------------------------- AdamW

M32 = 0xFFFFFFFF


def mix(h):
    h = ((h ^ (h >> 16)) * 0x6A09E667) & M32
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & M32
    return h ^ (h >> 16)


def random32(seed, step, first_block, blocks):
    """The 32 random bits of each value [blocks, 128]."""
    key = mix((mix(torch.tensor([seed & M32])) + step) & M32)
    block = torch.arange(first_block, first_block + blocks)
    return mix((mix((key + block) & M32)[:, None] + torch.arange(BLOCK)) & M32)


def root(v):
    return v.double().sqrt().float()


def adamw_fp32(w, g, m, v, step, lr, beta1, beta2, eps, decay, clip=None):
    """(w, m, v) in fp32, each operation rounded once (torch's products, sums and quotients on the CPU are; its root
    is not, so that is rounded from fp64)."""
    f = lambda s: torch.tensor(s, dtype=torch.float64).float()  # noqa: E731
    if clip is not None:
        g = g * clip
    m = f(beta1) * m + f(1.0 - beta1) * g
    v = f(beta2) * v + f(1.0 - beta2) * g * g
    d = root(v) * f(1.0 / math.sqrt(1.0 - beta2 ** step)) + f(eps)
    return w * f(1.0 - lr * decay) - f(lr / (1.0 - beta1 ** step)) * (m / d), m, v


def round_up_sometimes(v, random16, root):
    """(codes' values, scales) of fp32 blocks [n, 128] in e4m3, up with the probability of the remainder."""
    s = scale_of(torch.where(v.isfinite(), v.abs(), 0.0).amax(1))
    y = (v.double() / s[:, None]).abs()
    step = binade(torch.where(v.isfinite(), y, 1.0).clamp_min(2.0 ** -6)) / 8
    q = torch.floor(y / step + (random16.double() + 0.5) / 65536) * step
    if root:
        q = torch.where(y > 0, q.clamp_min(2.0 ** -9), q)
    return torch.where(v.isfinite(), q * torch.where(v < 0, -1.0, 1.0), torch.nan), s
