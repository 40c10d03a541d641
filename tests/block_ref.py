"""fp64 definitions of the block operators (group norm with an activation, linear map with epilogue) and
the error bounds their fp32 evaluation is held to.

Every value comes with a bound on its error, carried through the formulas to first order from these
roundings (u = 2^-24):

* a mean or sum over m values in fp32, added in a tree of lanes and workgroups with runs of at most ~40
  values a lane: 64 u times the sum of the absolute values (a run of k additions costs k u, the tree
  adds ~10 u, and the products inside cost 2 u);
* an elementary step costs u of its result, a hardware exponential, reciprocal or square root 2 u;
* silu and gelu: their value within 8 u (|h| + 1), their slope within 16 u (1 + |h|);
* the rational: 16 u times the sum of the absolute values of its terms, as for the activation alone;
* an error of h passes through the activation by its slope, through the slope by the second derivative;
* a bf16 result is rounded once: half a unit of its last place.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
SUM = 64 * U


def poly_terms(h, A, B):
    """P, P', P'', Q, Q', Q'' and the sums of absolute terms of each, for h [..., c] and
    per-channel coefficients A [c, 6], B [c, 4] (fp64)."""
    a = [A[:, i] for i in range(6)]
    b = [None] + [B[:, j] for j in range(4)]
    z = torch.zeros_like(h)

    def sums(cs):
        out, mag = [z.clone() for _ in range(3)], [z.clone() for _ in range(3)]
        for i, k in cs:
            for d in range(3):
                if i >= d:
                    t = math.perm(i, d) * k * h ** (i - d)
                    out[d] = out[d] + t
                    mag[d] = mag[d] + t.abs()
        return out, mag

    return sums(list(enumerate(a))), sums([(j, b[j]) for j in range(1, 5)])


def per_channel(A, B, channels):
    g = A.shape[0]
    return (A.double().repeat_interleave(channels // g, 0), B.double().repeat_interleave(channels // g, 0))


def activation(h, eh, act, A=None, B=None):
    """(y, bound of y, slope, bound of slope, extra) at h with error bound eh; extra is (D, s, P, rounding
    scales) for the rational's coefficient terms."""
    if act == "none":
        return h, eh, torch.ones_like(h), torch.zeros_like(h), None
    if act == "silu":
        s = torch.sigmoid(h)
        y, d1 = h * s, s + h * s * (1 - s)
        d2 = s * (1 - s) * (2 + h * (1 - 2 * s))
    elif act == "gelu":
        cdf = 0.5 * torch.erfc(-h / math.sqrt(2))
        phi = torch.exp(-h * h / 2) / math.sqrt(2 * math.pi)
        y, d1 = h * cdf, cdf + h * phi
        d2 = phi * (2 - h * h)
    else:
        Ac, Bc = per_channel(A, B, h.shape[-1])
        (P, mP), (Q, mQ) = poly_terms(h, Ac, Bc)
        s, D = torch.sign(Q[0]), 1 + Q[0].abs()
        y = P[0] / D
        d1 = P[1] / D - s * P[0] * Q[1] / D ** 2
        d2 = (P[2].abs() + 2 * (P[1] * Q[1]).abs() / D + (P[0] * Q[2]).abs() / D + 2 * (P[0] * Q[1] ** 2).abs() / D ** 2) / D
        my = mP[0] / D + P[0].abs() * mQ[0] / D ** 2
        md = mP[1] / D + mP[0] * mQ[1] / D ** 2 + (P[1].abs() * mQ[0] + P[0].abs() * mQ[1]) / D ** 2 \
            + 2 * P[0].abs() * Q[1].abs() * mQ[0] / D ** 3
        return y, d1.abs() * eh + d2 * eh ** 2 + 16 * U * my, d1, d2 * eh + 16 * U * md, (D, s, P[0], mP[0], mQ[0])
    return y, d1.abs() * eh + 8 * U * (h.abs() + 1), d1, d2.abs() * eh + eh ** 2 + 16 * U * (1 + h.abs()), None


def rounding(v, dtype):
    """Bound of the last rounding of a result."""
    if dtype == torch.bfloat16:
        return torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -126))) - 7) * 0.5 * 1.01
    return v.abs() * 2 * U


def coefficient_sums(h, eh, dy, A, extra, groups):
    """(dA, dB, their bounds) for rows of h [rows, c] and exact dy."""
    c = h.shape[-1]
    D, s, P, mP, mQ = (t.reshape(-1, c) for t in extra)
    vals, errs = [], []
    for k in range(10):
        if k < 6:
            t = dy * h ** k / D
            dt = dy.abs() * (k * h.abs() ** max(k - 1, 0) * eh / D + 16 * U * h.abs() ** k * (1 + mQ / D) / D)
            dt = dt + t.abs() * eh * mQ / D
        else:
            j = k - 5
            t = -dy * s * P * h ** j / D ** 2
            dt = dy.abs() * (16 * U * h.abs() ** j * (mP + 2 * P.abs() * mQ / D) / D ** 2)
            dt = dt + dy.abs() * eh * (j * h.abs() ** (j - 1) * mP + h.abs() ** j * (mP * 5 + mP * 2 * mQ)) / D ** 2
        t, dt = t.reshape(-1, groups, c // groups), dt.reshape(-1, groups, c // groups)
        vals.append(t.sum((0, 2)))
        errs.append(dt.sum((0, 2)) + SUM * t.abs().sum((0, 2)))
    v, e = torch.stack(vals, 1), torch.stack(errs, 1)
    return v[:, :6], v[:, 6:], e[:, :6], e[:, 6:]


def norm_forward(x, groups, weight, bias, eps, act, A=None, B=None):
    """{name: (value, bound)} of y, mean, rstd for x [n, ..., c]."""
    n, c = x.shape[0], x.shape[-1]
    d = x.double().reshape(n, -1, groups, c // groups)
    mean = d.mean((1, 3))
    var = (d - mean[:, None, :, None]).square().mean((1, 3))
    rstd = 1 / torch.sqrt(var + eps)
    em = SUM * d.abs().mean((1, 3))
    er = rstd * (SUM * var / (var + eps) + em ** 2 / (var + eps) + 4 * U)
    m4, r4, em4, er4 = (t[:, None, :, None] for t in (mean, rstd, em, er))
    xh = (d - m4) * r4
    exh = (em4 + U * (d - m4).abs()) * r4 + (d - m4).abs() * er4 + 2 * U * xh.abs()
    xh, exh = xh.reshape(n, -1, c), exh.reshape(n, -1, c)
    w = torch.ones(c, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(c, dtype=torch.float64) if bias is None else bias.double()
    h = xh * w + b
    eh = exh * w.abs() + 2 * U * ((xh * w).abs() + b.abs())
    y, ey, _, _, _ = activation(h, eh, act, A, B)
    y, ey = y.reshape(x.shape), ey.reshape(x.shape)
    return {"y": (y, ey + rounding(y, x.dtype)), "mean": (mean, em + U * mean.abs()), "rstd": (rstd, er)}


def norm_backward(x, dy, mean, rstd, groups, weight, bias, act, A=None, B=None):
    """{name: (value, bound)} of dx, dweight, dbias (dA, dB) with the given fp32 statistics."""
    n, c = x.shape[0], x.shape[-1]
    d = x.double().reshape(n, -1, groups, c // groups)
    m4, r4 = mean.double()[:, None, :, None], rstd.double()[:, None, :, None]
    xh = ((d - m4) * r4).reshape(n, -1, c)
    exh = 3 * U * xh.abs()
    w = torch.ones(c, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(c, dtype=torch.float64) if bias is None else bias.double()
    h = xh * w + b
    eh = exh * w.abs() + 2 * U * ((xh * w).abs() + b.abs())
    _, _, slope, es, extra = activation(h, eh, act, A, B)
    g = dy.double().reshape(n, -1, c)
    dh, edh = g * slope, g.abs() * es + 2 * U * (g * slope).abs()
    out = {}
    tw = dh * xh
    out["dweight"] = (tw.sum((0, 1)), (edh * xh.abs() + dh.abs() * exh).sum((0, 1)) + SUM * tw.abs().sum((0, 1)))
    out["dbias"] = (dh.sum((0, 1)), edh.sum((0, 1)) + SUM * dh.abs().sum((0, 1)))
    if act == "rational":
        ng = A.shape[0]
        dA, dB, eA, eB = coefficient_sums(h.reshape(-1, c), eh.reshape(-1, c), g.reshape(-1, c), A, extra, ng)
        out["dA"], out["dB"] = (dA, eA), (dB, eB)
    shape = (n, -1, groups, c // groups)
    t, et = (dh * w).reshape(shape), (edh * w.abs() + U * (dh * w).abs()).reshape(shape)
    xg, exg = xh.reshape(shape), exh.reshape(shape)
    m1, m2 = t.mean((1, 3), keepdim=True), (t * xg).mean((1, 3), keepdim=True)
    e1 = et.mean((1, 3), keepdim=True) + SUM * t.abs().mean((1, 3), keepdim=True)
    e2 = (et * xg.abs() + t.abs() * exg).mean((1, 3), keepdim=True) + SUM * (t * xg).abs().mean((1, 3), keepdim=True)
    dx = r4 * (t - m1 - xg * m2)
    edx = r4 * (et + e1 + xg.abs() * e2 + exg * m2.abs() + 4 * U * (t.abs() + m1.abs() + (xg * m2).abs()))
    dx, edx = dx.reshape(x.shape), edx.reshape(x.shape)
    out["dx"] = (dx, edx + rounding(dx, x.dtype))
    return out


def check(what, got, ref, bound):
    """Every element within its bound (and finite where the reference is)."""
    g = got.detach().double().to(ref.device).reshape(ref.shape)
    err = (g - ref).abs()
    bad = ~(err <= bound + 1e-37)
    if bad.any():
        i = int(torch.argmax(torch.where(bad, err / (bound + 1e-37), torch.zeros_like(err)).reshape(-1)))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; worst at {i}: got "
                             f"{g.reshape(-1)[i]!r}, reference {ref.reshape(-1)[i]!r}, bound {bound.reshape(-1)[i]!r}")


def bf16_neighbours(v, e):
    """(nearest bf16 of v, allowance): 0 where every value within e of v rounds the same way, else the
    distance between the two candidates."""
    lo, hi = (v - e).to(torch.bfloat16).double(), (v + e).to(torch.bfloat16).double()
    return v.to(torch.bfloat16).double(), (hi - lo).abs()


def linear_forward(x, W, bias, act, A=None, B=None, residual=None):
    """{name: (value, bound)} of z and pre; K exact products summed in fp32 cost at most (K + 8) u of the
    sum of their absolute values."""
    xd, wd = x.double(), W.double()
    h, mag = xd @ wd.t(), xd.abs() @ wd.abs().t()
    eh = (x.shape[-1] + 8) * U * mag
    if bias is not None:
        h = h + bias.double()
        eh = eh + 2 * U * (h.abs() + bias.double().abs())
    y, ey, _, _, _ = activation(h, eh, act, A, B)
    if residual is not None:
        y = y + residual.double()
        ey = ey + U * (y.abs() + residual.double().abs())
    return {"z": (y, ey + rounding(y.abs() + ey, torch.bfloat16)), "pre": (h, eh + rounding(h.abs() + eh, torch.bfloat16))}


def linear_backward(x, W, dz, pre, act, A=None, B=None):
    """{name: (value, bound)} of dx, dW, dbias (dA, dB).  dpre is rounded to bf16 as the products' operand:
    the reference rounds its own and allows for the elements whose rounding its error does not settle."""
    g = dz.double()
    d, e = g, torch.zeros_like(g)
    out = {}
    if act != "none":
        h = pre.double()
        zero = torch.zeros_like(h)
        _, _, slope, es, extra = activation(h, zero, act, A, B)
        d, e = g * slope, g.abs() * es + 2 * U * (g * slope).abs()
        if act == "rational":
            dA, dB, eA, eB = coefficient_sums(h, zero, g, A, extra, A.shape[0])
            out["dA"], out["dB"] = (dA, eA), (dB, eB)
    out["dbias"] = (d.sum(0), e.sum(0) + SUM * d.abs().sum(0))
    q, amb = bf16_neighbours(d, e)
    xd, wd = x.double(), W.double()
    for name, v, mag, a, k in (("dx", q @ wd, q.abs() @ wd.abs(), amb @ wd.abs(), W.shape[0]),
                               ("dW", q.t() @ xd, q.abs().t() @ xd.abs(), amb.t() @ xd.abs(), x.shape[0])):
        err = a + (k + 8) * U * mag
        out[name] = (v, err + rounding(v.abs() + err, torch.bfloat16))
    return out
