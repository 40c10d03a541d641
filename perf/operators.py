"""Cases of the two operators that surround the group-rational activation in a GR-KAN block, and
their plain forms: group norm with an activation (channels last), and the matrix product with
bias, activation and residual in its epilogue, each forward and backward.

    listed()         the cases; each comment says what the case stands for in use
    draw(rng)        one more case of the same ranges
    prepare(case, s) the inputs a program has in hand before the call, from the seed alone
    run(state)       one pass: elementary torch operations in fp32 (``own`` false), or the
                     library's entry points (``own`` true)
    exact(case, s)   the same outputs from the definitions in fp64
    work(case)       bytes and flops the pass cannot do without
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# A rational (5, 4) least-squares fit of the Swish function x / (1 + e^-x) on [-5, 5] with an even,
# positive denominator: the usual starting point of a rational unit that replaces a Swish.
SWISH_A = (0.0, 0.5, 0.249944, 0.0526866, 0.00555034, 0.000244433)
SWISH_B = (0.0, 0.105373, 0.0, 0.000488866)


def _norm(name, way, io, n, s, c, groups, act, act_groups=8):
    """x is [n, s, c]: n samples of s positions, c channels in `groups` normalisation groups."""
    return {"name": name, "op": "norm", "way": way, "io": io, "n": n, "s": s, "c": c, "groups": groups,
            "act": act, "act_groups": act_groups}


def _linear(name, way, rows, d_in, d_out, act, residual, keep, act_groups=8):
    """z = act(x W^T + b) + r for x [rows, d_in], W [d_out, d_in], bf16; keep: the forward also
    returns the product before the activation, as training does."""
    return {"name": name, "op": "linear", "way": way, "rows": rows, "d_in": d_in, "d_out": d_out, "act": act,
            "residual": residual, "keep": keep, "act_groups": act_groups}


def listed():
    return [
        # one token of a served KAT-B: pre-norm and the first activation; latency alone counts
        _norm("norm-fwd-token", "fwd", "bf16", 1, 1, 768, 1, "rational"),
        # the pre-norm of a KAT-B block over 256 images of 197 tokens, one statistic per token
        _norm("norm-fwd-tokens", "fwd", "bf16", 256 * 197, 1, 768, 1, "rational"),
        # a convolutional stage's feature maps, 10 channels a group: groups end inside 16 bytes
        _norm("norm-fwd-maps", "fwd", "bf16", 8, 64 * 64, 320, 32, "silu"),
        # one large fp32 feature map, 4 channels a group: few, long sums
        _norm("norm-fwd-map-large", "fwd", "f32", 1, 256 * 256, 128, 32, "silu"),
        # KAT-T training, 8 groups over an image's 197 tokens, fp32
        _norm("norm-bwd-images", "bwd", "f32", 128, 197, 192, 8, "gelu"),
        # KAT-B training at full batch, one statistic per token: the largest of the norms
        _norm("norm-bwd-tokens", "bwd", "bf16", 1024 * 197, 1, 768, 1, "rational"),
        # one token through the first product of a KAT-B MLP: the weights' bytes alone
        _linear("linear-fwd-token", "fwd", 1, 768, 3072, "rational", False, False),
        # one image through the second product, with the block's residual
        _linear("linear-fwd-image", "fwd", 197, 3072, 768, "none", True, False),
        # odd sizes in every direction: nothing is a multiple of a vector or a tile
        _linear("linear-fwd-odd", "fwd", 1003, 777, 1501, "gelu", True, True),
        # KAT-B training at full batch, 1024 images of 197 tokens: the largest of all
        _linear("linear-fwd-full", "fwd", 1024 * 197, 768, 3072, "rational", False, True),
        # KAT-T training: its first product's gradients
        _linear("linear-bwd-images", "bwd", 128 * 197, 192, 768, "rational", False, True),
        # KAT-B training with a quarter of the batch: the second product's gradients
        _linear("linear-bwd-batch", "bwd", 256 * 197, 3072, 768, "silu", True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MAX_NORM = 1024 * 197 * 768             # elements
MAX_LINEAR = 1024 * 197 * 768 * 3072    # products


def draw(rng):
    way = rng.choice(("fwd", "bwd"))
    act = rng.choice(("none", "silu", "gelu", "rational"))
    if rng.random() < 0.5:
        io = rng.choice(("f32", "bf16"))
        groups = rng.choice((1, 1, 2, 4, 8, 16, 32))
        c = groups * max(4, _log(rng, 32, 4096) // groups)
        act_groups = 8 if c % 8 == 0 else groups
        kind = rng.choice(("tokens", "images", "maps"))
        if kind == "tokens":     # one statistic per token (and group)
            s = 1
            n = _log(rng, 1, 1024 * 197)
        elif kind == "images":   # a sequence of tokens, odd lengths among them
            s = _log(rng, 2, 1024)
            n = _log(rng, 1, 1024)
        else:                    # square maps
            s = _log(rng, 7, 256) ** 2
            n = _log(rng, 1, 64)
        cap = MAX_NORM // (2 if io == "f32" else 1)
        n = max(1, min(n, cap // (s * c)))
        s = max(1, min(s, cap // (n * c)))
        return _norm("", way, io, n, s, c, groups, act, act_groups)
    d_in, d_out = _log(rng, 48, 4096), _log(rng, 48, 4096)
    if rng.random() < 0.7:       # most widths are whole vectors, as a model's are
        d_in, d_out = max(64, d_in // 64 * 64), max(64, d_out // 64 * 64)
    if act == "rational" and d_out % 8:
        act = "gelu"
    rows = _log(rng, 1, 1024 * 197)
    cap = MAX_LINEAR // (2 if way == "bwd" else 1)
    rows = max(1, min(rows, cap // (d_in * d_out)))
    keep = way == "bwd" or rng.random() < 0.5
    return _linear("", way, rows, d_in, d_out, act, rng.random() < 0.5, keep)


def _normal(gen, shape, std, dtype, mean=0.0):
    t = torch.empty(shape, dtype=torch.float32, device=DEV).normal_(mean, std, generator=gen)
    return t.to(dtype)


def _swish_like(gen, groups):
    """A [groups, 6], B [groups, 4]: the fit above, every group's coefficients 10% off it."""
    A = torch.tensor(SWISH_A, device=DEV).repeat(groups, 1)
    B = torch.tensor(SWISH_B, device=DEV).repeat(groups, 1)
    A = A * (1.0 + _normal(gen, A.shape, 0.1, torch.float32).clamp(-0.3, 0.3))
    B = B * (1.0 + _normal(gen, B.shape, 0.1, torch.float32).clamp(-0.3, 0.3))
    return A.contiguous(), B.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": dict(case)}
    rational = case["act"] == "rational"
    if case["op"] == "norm":
        io, c = TYPES[case["io"]], case["c"]
        shape = (case["n"], case["s"], c)
        st["x"] = _normal(gen, shape, 1.5, io, 0.3)
        st["w"] = 1.0 + _normal(gen, (c,), 0.1, torch.float32)
        st["b"] = _normal(gen, (c,), 0.1, torch.float32)
        st["A"], st["B"] = _swish_like(gen, case["act_groups"]) if rational else (None, None)
        if case["way"] == "bwd":
            st["dy"] = _normal(gen, shape, 1e-2, io)
            # the forward pass kept its statistics
            st["mean"], st["rstd"] = _stats(st["x"].float(), case["groups"])
        return st
    rows, d_in, d_out = case["rows"], case["d_in"], case["d_out"]
    bf = torch.bfloat16
    st["x"] = _normal(gen, (rows, d_in), 1.0, bf)
    st["W"] = _normal(gen, (d_out, d_in), 1.0 / math.sqrt(d_in), bf)
    st["b"] = _normal(gen, (d_out,), 0.1, torch.float32)
    st["A"] = _normal(gen, (case["act_groups"], 6), 0.5, torch.float32) if rational else None
    st["B"] = _normal(gen, (case["act_groups"], 4), 0.5, torch.float32) if rational else None
    if case["way"] == "fwd":
        st["r"] = _normal(gen, (rows, d_out), 1.0, bf) if case["residual"] else None
    else:
        st["dz"] = _normal(gen, (rows, d_out), 1e-2, bf)
        # the forward pass kept the product before the activation
        st["pre"] = None
        if case["act"] != "none":
            st["pre"] = (st["x"].float() @ st["W"].float().t() + st["b"]).to(bf)
    return st


# ---------------------------------------------------------------- the operators' plain forms

def _stats(x, groups):
    """Mean and 1 / sqrt(var + eps) [n, groups] over the positions and channels of each group."""
    n, s, c = x.shape
    v = x.view(n, s, groups, c // groups)
    mean = v.mean(dim=(1, 3))
    var = (v - mean.view(n, 1, groups, 1)).square().mean(dim=(1, 3))
    return mean, (var + EPS).rsqrt()


def _act(h, act, A, B):
    """act(h) for fp32 h [..., c]."""
    if act == "none":
        return h
    if act == "silu":
        return h / (1.0 + torch.exp(-h))
    if act == "gelu":
        return 0.5 * h * (1.0 + torch.erf(h * math.sqrt(0.5)))
    g = A.shape[0]
    v = h.view(-1, g, h.shape[-1] // g)
    a = [A[:, i].view(1, g, 1) for i in range(6)]
    b = [B[:, j].view(1, g, 1) for j in range(4)]
    P = ((((a[5] * v + a[4]) * v + a[3]) * v + a[2]) * v + a[1]) * v + a[0]
    Q = (((b[3] * v + b[2]) * v + b[1]) * v + b[0]) * v
    return (P / (1.0 + Q.abs())).view(h.shape)


def _act_backward(h, dy, act, A, B):
    """(dh, dA, dB) of y = act(h) for fp32 h, dy [..., c]; dA and dB None but for the rational."""
    if act == "none":
        return dy, None, None
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-h))
        return dy * sg * (1.0 + h * (1.0 - sg)), None, None
    if act == "gelu":
        phi = torch.exp(-0.5 * h * h) * (1.0 / math.sqrt(2.0 * math.pi))
        return dy * (0.5 * (1.0 + torch.erf(h * math.sqrt(0.5))) + h * phi), None, None
    g = A.shape[0]
    shape = (-1, g, h.shape[-1] // g)
    v, dv = h.reshape(shape), dy.reshape(shape)
    a = [A[:, i].view(1, g, 1) for i in range(6)]
    b = [B[:, j].view(1, g, 1) for j in range(4)]
    P = ((((a[5] * v + a[4]) * v + a[3]) * v + a[2]) * v + a[1]) * v + a[0]
    dP = (((5.0 * a[5] * v + 4.0 * a[4]) * v + 3.0 * a[3]) * v + 2.0 * a[2]) * v + a[1]
    Q = (((b[3] * v + b[2]) * v + b[1]) * v + b[0]) * v
    dQ = ((4.0 * b[3] * v + 3.0 * b[2]) * v + 2.0 * b[1]) * v + b[0]
    D = 1.0 + Q.abs()
    w = dv / D
    u = w * (P / D) * torch.sign(Q)
    dh = (w * dP - u * dQ).view(h.shape)
    dA, dB = [], []
    for i in range(6):
        dA.append(w.sum(dim=(0, 2)))
        w = w * v
    for j in range(4):
        u = u * v
        dB.append(-u.sum(dim=(0, 2)))
    return dh, torch.stack(dA, 1), torch.stack(dB, 1)


def _plain_norm(st):
    case = st["case"]
    n, s, c = case["n"], case["s"], case["c"]
    g = case["groups"]
    x = st["x"].float()
    io = st["x"].dtype
    if case["way"] == "fwd":
        mean, rstd = _stats(x, g)
        xh = (x.view(n, s, g, -1) - mean.view(n, 1, g, 1)) * rstd.view(n, 1, g, 1)
        h = xh.view(n, s, c) * st["w"] + st["b"]
        return _act(h, case["act"], st["A"], st["B"]).to(io), mean, rstd
    mean, rstd = st["mean"], st["rstd"]
    xh = ((x.view(n, s, g, -1) - mean.view(n, 1, g, 1)) * rstd.view(n, 1, g, 1)).view(n, s, c)
    h = xh * st["w"] + st["b"]
    dh, dA, dB = _act_backward(h, st["dy"].float(), case["act"], st["A"], st["B"])
    dw, db = (dh * xh).sum(dim=(0, 1)), dh.sum(dim=(0, 1))
    t = (dh * st["w"]).view(n, s, g, -1)
    xg = xh.view(n, s, g, -1)
    m1 = t.mean(dim=(1, 3), keepdim=True)
    m2 = (t * xg).mean(dim=(1, 3), keepdim=True)
    dx = ((t - m1 - xg * m2) * rstd.view(n, 1, g, 1)).view(n, s, c).to(io)
    return (dx, dw, db) if dA is None else (dx, dw, db, dA, dB)


def _plain_linear(st):
    case = st["case"]
    x, W = st["x"].float(), st["W"].float()
    bf = torch.bfloat16
    if case["way"] == "fwd":
        pre = x @ W.t() + st["b"]
        z = _act(pre, case["act"], st["A"], st["B"])
        if st["r"] is not None:
            z = z + st["r"].float()
        return (z.to(bf), pre.to(bf)) if case["keep"] else (z.to(bf),)
    dz = st["dz"].float()
    h = None if st["pre"] is None else st["pre"].float()
    dpre, dA, dB = _act_backward(h, dz, case["act"], st["A"], st["B"])
    dx, dW, db = (dpre @ W).to(bf), (dpre.t() @ x).to(bf), dpre.sum(0)
    return (dx, dW, db) if dA is None else (dx, dW, db, dA, dB)


# ---------------------------------------------------------------- the library's operators

def _own_norm(st):
    from gr_kan_rational_amd import grkan_group_norm_backward, grkan_group_norm_forward

    case = st["case"]
    if case["way"] == "fwd":
        return grkan_group_norm_forward(st["x"], case["groups"], st["w"], st["b"], EPS, case["act"],
                                        st["A"], st["B"], case["act_groups"])
    out = grkan_group_norm_backward(st["x"], st["dy"], st["mean"], st["rstd"], case["groups"], st["w"], st["b"],
                                    case["act"], st["A"], st["B"], case["act_groups"])
    return out if case["act"] == "rational" else out[:3]


def _own_linear(st):
    from gr_kan_rational_amd import grkan_linear_act_backward, grkan_linear_act_forward

    case = st["case"]
    if case["way"] == "fwd":
        z, pre = grkan_linear_act_forward(st["x"], st["W"], st["b"], case["act"], st["A"], st["B"],
                                          case["act_groups"], residual=st["r"], keep=case["keep"])
        return (z, pre) if case["keep"] else (z,)
    out = grkan_linear_act_backward(st["x"], st["W"], st["dz"], st["pre"], case["act"], st["A"], st["B"],
                                    case["act_groups"])
    return out if case["act"] == "rational" else out[:3]


def run(state):
    norm = state["case"]["op"] == "norm"
    if own:
        return _own_norm(state) if norm else _own_linear(state)
    return _plain_norm(state) if norm else _plain_linear(state)


# ---------------------------------------------------------------- the definitions in fp64

def _value_and_slope(h, act, A, B):
    """act(h), act'(h) and, for the rational, what its coefficients' gradients sum: the factors
    x^i / D (6 of them) and -s P x^j / D^2 (4), one at a time through a function."""
    if act == "none":
        return h, torch.ones_like(h), None
    if act == "silu":
        sg = torch.sigmoid(h)
        return h * sg, sg + h * sg * (1.0 - sg), None
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-h / math.sqrt(2.0))
        return h * cdf, cdf + h * torch.exp(-h * h / 2.0) / math.sqrt(2.0 * math.pi), None
    c, g = h.shape[-1], A.shape[0]
    a = A.double().repeat_interleave(c // g, dim=0)
    b = B.double().repeat_interleave(c // g, dim=0)
    P, dP = torch.zeros_like(h), torch.zeros_like(h)
    for i in range(6):
        P += a[:, i] * h ** i
        if i:
            dP += i * a[:, i] * h ** (i - 1)
    Q, dQ = torch.zeros_like(h), torch.zeros_like(h)
    for j in range(1, 5):
        Q += b[:, j - 1] * h ** j
        dQ += j * b[:, j - 1] * h ** (j - 1)
    s, D = Q.sign(), Q.abs() + 1.0

    def factor(k):
        return h ** k / D if k < 6 else -s * P * h ** (k - 5) / (D * D)

    return P / D, (dP * D - s * P * dQ) / (D * D), factor


def _coefficient_sums(dy, factor, groups):
    sums = []
    for k in range(10):
        t = dy * factor(k)
        sums.append(t.reshape(-1, groups, t.shape[-1] // groups).sum(dim=(0, 2)))
    return torch.stack(sums[:6], 1), torch.stack(sums[6:], 1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        n, s, c, g = case["n"], case["s"], case["c"], case["groups"]
        x = st["x"].double().view(n, s, g, c // g)
        gamma, beta = st["w"].double(), st["b"].double()
        if case["way"] == "fwd":
            var, mean = torch.var_mean(x, dim=(1, 3), correction=0)
            rstd = 1.0 / torch.sqrt(var + EPS)
        else:
            mean, rstd = st["mean"].double(), st["rstd"].double()
        xh = ((x - mean[:, None, :, None]) * rstd[:, None, :, None]).view(n * s, c)
        del x
        y, slope, factor = _value_and_slope(xh * gamma + beta, case["act"], st["A"], st["B"])
        if case["way"] == "fwd":
            return y.view(n, s, c), mean, rstd
        dy = st["dy"].double().view(n * s, c)
        dh = dy * slope
        out = [None, (dh * xh).sum(0), dh.sum(0)]
        if factor is not None:
            out += _coefficient_sums(dy, factor, case["act_groups"])
        del factor, slope, y
        v = (dh * gamma).view(n, s, g, c // g)
        xh = xh.view(n, s, g, c // g)
        k = s * (c // g)
        proj = (v.sum(dim=(1, 3)) / k)[:, None, :, None] + xh * ((v * xh).sum(dim=(1, 3)) / k)[:, None, :, None]
        out[0] = ((v - proj) * rstd[:, None, :, None]).view(n, s, c)
        return tuple(out)
    x, W = st["x"].double(), st["W"].double()
    if case["way"] == "fwd":
        pre = torch.addmm(st["b"].double(), x, W.t())
        z, _, _ = _value_and_slope(pre, case["act"], st["A"], st["B"])
        if st["r"] is not None:
            z = z + st["r"].double()
        return (z, pre) if case["keep"] else (z,)
    dz = st["dz"].double()
    dpre, sums = dz, ()
    if case["act"] != "none":
        _, slope, factor = _value_and_slope(st["pre"].double(), case["act"], st["A"], st["B"])
        dpre = dz * slope
        if factor is not None:
            sums = _coefficient_sums(dz, factor, case["act_groups"])
    return (torch.mm(dpre, W), torch.mm(dpre.t(), x), dpre.sum(0), *sums)


# ---------------------------------------------------------------- the least work

ACT_FLOPS = {"none": 0, "silu": 4, "gelu": 12, "rational": 21}
ACT_BACKWARD_FLOPS = {"none": 0, "silu": 7, "gelu": 16, "rational": 60}


def work(case):
    rational = 80 * case["act_groups"] if case["act"] == "rational" else 0
    if case["op"] == "norm":
        n, s, c, g = case["n"], case["s"], case["c"], case["groups"]
        e, es = n * s * c, 4 if case["io"] == "f32" else 2
        if case["way"] == "fwd":
            return {"bytes": 2 * e * es + 8 * c + 8 * n * g + rational // 2,
                    "flops": e * (8 + ACT_FLOPS[case["act"]])}
        return {"bytes": 3 * e * es + 16 * c + 8 * n * g + rational,
                "flops": e * (14 + ACT_BACKWARD_FLOPS[case["act"]])}
    rows, d_in, d_out = case["rows"], case["d_in"], case["d_out"]
    if case["way"] == "fwd":
        outs = 1 + case["residual"] + case["keep"]
        return {"bytes": 2 * (rows * d_in + d_in * d_out + rows * d_out * outs) + 4 * d_out + rational // 2,
                "flops": 2 * rows * d_in * d_out}
    outs = 1 if case["act"] == "none" else 2
    return {"bytes": 2 * (2 * rows * d_in + 2 * d_in * d_out + rows * d_out * outs) + 4 * d_out + rational,
            "flops": 4 * rows * d_in * d_out}
