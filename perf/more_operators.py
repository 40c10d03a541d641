"""Cases of the operators of a training step (and a served token) of a deep GR-KAN stack, and their plain
forms: the 8-bit quantiser and the matrix product of its results, a scale for each block of 128; the residual
path between two blocks with the norms on either side of it; the AdamW step over many tensors.

    listed()         the cases; each comment says what the case stands for in use
    draw(rng)        one more case of the same ranges
    prepare(case, s) what a program has in hand before the call, from the seed alone
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
BLOCK = 128                # values that share a scale
E4M3_MAX = 448.0
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn

# A rational (5, 4) least-squares fit of the Swish function x / (1 + e^-x) on [-5, 5] with an even,
# positive denominator: the usual starting point of a rational unit that replaces a Swish.
SWISH_A = (0.0, 0.5, 0.249944, 0.0526866, 0.00555034, 0.000244433)
SWISH_B = (0.0, 0.105373, 0.0, 0.000488866)


def _quantize(name, rows, cols, io, act, outputs, tile):
    """e4m3 codes and scales of x (or F(x)) [rows, cols]: a scale for each 128 of a row and / or of a column,
    or (tile) for each 128 x 128."""
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "io": io, "act": act, "outputs": outputs,
            "tile": tile}


def _matmul(name, m, n, k, tile, bias, residual, out):
    """a [m, k], b [n, k] e4m3 with their scales (b's for each 128 x 128 where tile) -> a b^T [m, n]."""
    return {"name": name, "op": "matmul", "m": m, "n": n, "k": k, "tile": tile, "bias": bias, "residual": residual,
            "out": out}


def _residual(name, way, io, samples, positions, c, norm, post, gate):
    """h = x + scale gate post(f), z = norm(h) over samples x positions rows of c channels."""
    return {"name": name, "op": "residual", "way": way, "io": io, "samples": samples, "positions": positions, "c": c,
            "norm": norm, "post": post, "gate": gate}


def _adamw(name, bits, blocks, dim, hidden, clip):
    """The tensors of `blocks` channel mixers (two bf16 matrices with fp32 masters and eight fp32 tensors each)."""
    return {"name": name, "op": "adamw", "bits": bits, "blocks": blocks, "dim": dim, "hidden": hidden, "clip": clip}


def listed():
    return [
        # KAT-B served: a batch's normalised tokens through the layer's first rational into 8 bits
        _quantize("quantize-rational", 128 * 197, 768, "bf16", "rational", "rows", False),
        # KAT-B training: a hidden gradient, by rows for dx and by columns for dW, read once
        _quantize("quantize-both", 128 * 197, 3072, "bf16", "none", "both", False),
        # one token of a served KAT-B through the first product: the weights' bytes alone
        _matmul("matmul-token", 1, 3072, 768, True, True, False, "bf16"),
        # odd sizes in every direction: nothing is a multiple of a vector, a block or a tile
        _matmul("matmul-odd", 1003, 1501, 777, True, True, True, "bf16"),
        # KAT-B training with a quarter of the batch: the first product
        _matmul("matmul-batch", 256 * 197, 3072, 768, True, True, False, "bf16"),
        # KAT-B training: the weight gradient of the same product, both operands scaled along their rows
        _matmul("matmul-gradient", 3072, 768, 256 * 197, False, False, False, "f32"),
        # one token of a served stack: the residual and the next block's norm; latency alone
        _residual("residual-token", "fwd", "bf16", 1, 1, 768, "rms", "none", "none"),
        # KAT-B training at a quarter batch, pre-norm blocks with a residual scale and stochastic depth
        _residual("residual-fwd", "fwd", "bf16", 256, 197, 768, "layer", "none", "sample"),
        # the backward of a block with norms on both sides and a gate per image and channel
        _residual("residual-bwd", "bwd", "bf16", 256, 197, 768, "rms", "rms", "channel"),
        # one KAT-T mixer's ten tensors: latency
        _adamw("adamw-one", 32, 1, 192, 768, False),
        # the mixers of a KAT-B, 12 blocks, 57 million parameters, states in 32 bits
        _adamw("adamw-base", 32, 12, 768, 3072, True),
        # the same with states in 8 bits
        _adamw("adamw8-base", 8, 12, 768, 3072, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MAX_QUANTIZE = 128 * 197 * 3072          # elements
MAX_MATMUL = 256 * 197 * 768 * 3072      # products
MAX_RESIDUAL = 256 * 197 * 768           # elements
MAX_ADAMW = 12 * 2 * 768 * 3072          # parameters


def draw(rng):
    op = rng.choice(("quantize", "matmul", "matmul", "residual", "residual", "adamw"))
    if op == "quantize":
        cols = _log(rng, 48, 4096)
        if rng.random() < 0.7:      # most widths are whole vectors, as a model's are
            cols = max(64, cols // 64 * 64)
        act = rng.choice(("none", "rational")) if cols % 8 == 0 else "none"
        rows = min(_log(rng, 1, 256 * 197), MAX_QUANTIZE // cols)
        tile = act == "none" and rng.random() < 0.3
        return _quantize("", rows, cols, rng.choice(("f32", "bf16")), act, rng.choice(("rows", "columns", "both")), tile)
    if op == "matmul":
        if rng.random() < 0.3:      # a weight gradient: a long k
            m, n, k = _log(rng, 48, 4096), _log(rng, 48, 4096), _log(rng, 200, 256 * 197)
            tile, out = False, "f32"
        else:
            m, n, k = _log(rng, 1, 256 * 197), _log(rng, 48, 4096), _log(rng, 48, 4096)
            tile, out = True, "bf16"
        if rng.random() < 0.7:
            n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
        if m * n * k > MAX_MATMUL:
            if tile:
                m = MAX_MATMUL // (n * k)
            else:
                k = MAX_MATMUL // (m * n)
        return _matmul("", m, n, k, tile, rng.random() < 0.5, rng.random() < 0.3, out)
    if op == "residual":
        c = _log(rng, 32, 8192)
        if rng.random() < 0.7:
            c = max(64, c // 64 * 64)
        io = rng.choice(("f32", "bf16"))
        cap = MAX_RESIDUAL // (2 if io == "f32" else 1)
        positions = min(_log(rng, 1, 1024), cap // c)
        samples = max(1, min(_log(rng, 1, 1024), cap // (c * positions)))
        return _residual("", rng.choice(("fwd", "bwd")), io, samples, positions, c, rng.choice(("layer", "rms")),
                         rng.choice(("none", "none", "layer", "rms")),
                         rng.choice(("none", "sample", "token", "channel", "element")))
    dim = _log(rng, 64, 1024) // 8 * 8
    hidden = dim * rng.choice((1, 2, 4))
    blocks = max(1, min(_log(rng, 1, 24), MAX_ADAMW // (2 * dim * hidden)))
    return _adamw("", rng.choice((32, 8)), blocks, dim, hidden, rng.random() < 0.5)


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


def _ceil(n, d):
    return -(-n // d)


def _weights8(gen, rows, cols, tile):
    """e4m3 codes [rows, cols] (rows 16 bytes apart or a multiple) and scales of a normal matrix, quantised
    elsewhere: any scale, the largest value of a block at 448.  The values spread over some binades along the
    columns, as a model's channels do."""
    x = _normal(gen, (rows, cols), 1.0, torch.float32)
    x *= torch.exp2(torch.randint(-3, 4, (cols,), generator=gen, device=DEV).float())
    rb, cb = _ceil(rows, BLOCK) if tile else rows, _ceil(cols, BLOCK)
    pad = torch.zeros((rb * BLOCK if tile else rows, cb * BLOCK), device=DEV)
    pad[:rows, :cols] = x
    v = pad.view(rb, BLOCK if tile else 1, cb, BLOCK)
    scale = (v.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp_min(1e-30)
    q = (v / scale[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(F8).view(pad.shape)
    codes = torch.zeros((rows, _ceil(cols, 16) * 16), dtype=torch.uint8, device=DEV)
    codes[:, :cols] = q[:rows, :cols].view(torch.uint8)
    scale = scale / scale.square().mean().sqrt()     # products of order 1
    return codes.view(F8)[:, :cols], scale.contiguous() if tile else scale.t().contiguous().t()


def _shapes(case):
    """(bf16 matrices, fp32 tensors) of one mixer."""
    d, h = case["dim"], case["hidden"]
    return [(h, d), (d, h)], [(d,), (d,), (8, 6), (8, 4), (8, 6), (8, 4), (h,), (d,)]


def _views(arena, shapes):
    """One tensor of each shape, one after another in the arena, each from a multiple of BLOCK on."""
    out, at = [], 0
    for s in shapes:
        n = math.prod(s)
        out.append(arena[at:at + n].view(s))
        at += _ceil(n, BLOCK) * BLOCK
    return out


def _flat(arena, shapes, per=BLOCK):
    """The states of the same tensors: their part of the arena, whole blocks (per: values kept of a block)."""
    out, at = [], 0
    for s in shapes:
        n = _ceil(math.prod(s), BLOCK) * per
        out.append(arena[at:at + n])
        at += n
    return out


def _arena(gen, shapes, std, dtype):
    """Values of all shapes with zeros between them."""
    arena = torch.zeros(sum(_ceil(math.prod(s), BLOCK) for s in shapes) * BLOCK, dtype=dtype, device=DEV)
    for v in _views(arena, shapes):
        v.copy_(_normal(gen, v.shape, std, dtype))
    return arena


def _prepare_adamw(case, gen):
    st = {"case": dict(case), "step": 1000, "lr": 1e-3, "seed": 12345}
    mats, vecs = _shapes(case)
    mats, vecs = mats * case["blocks"], vecs * case["blocks"]
    st["grad_scale"] = torch.tensor([0.7], device=DEV) if case["clip"] else None
    for k, shapes, dtype, std in (("w", mats, torch.bfloat16, 0.02), ("b", vecs, torch.float32, 0.1)):
        st[k + "_master"] = _arena(gen, shapes, std, torch.float32)
        st[k + "_grad"] = _arena(gen, shapes, 1e-3, dtype)
        m, r = _arena(gen, shapes, 3e-4, torch.float32), _arena(gen, shapes, 1e-3, torch.float32).abs()
        if case["bits"] == 32:
            st[k + "_m"], st[k + "_v"] = m, r * r
        else:
            st[k + "_m"], st[k + "_ms"] = _to_codes(m.view(-1, BLOCK))
            st[k + "_r"], st[k + "_rs"] = _to_codes(r.view(-1, BLOCK))
    # the bf16 copy that the products read
    st["w_param"] = st["w_master"].to(torch.bfloat16)
    # the lists that the program keeps of its tensors
    w, b = _views(st["w_param"], mats), _views(st["b_master"], vecs)
    st["params"] = w + b
    st["grads"] = _views(st["w_grad"], mats) + _views(st["b_grad"], vecs)
    st["masters"] = _views(st["w_master"], mats) + [None] * len(b)
    if case["bits"] == 32:
        st["avgs"] = _views(st["w_m"], mats) + _views(st["b_m"], vecs)
        st["sqs"] = _views(st["w_v"], mats) + _views(st["b_v"], vecs)
    else:
        for name, k, per in (("avgs", "m", BLOCK), ("sqs", "r", BLOCK), ("avg_scales", "ms", 1), ("sq_scales", "rs", 1)):
            st[name] = _flat(st["w_" + k].view(-1), mats, per) + _flat(st["b_" + k].view(-1), vecs, per)
    return st


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if case["op"] == "adamw":
        return _prepare_adamw(case, gen)
    st = {"case": dict(case)}
    if case["op"] == "quantize":
        # channels of different size, as a network's are
        spread = torch.exp2(torch.randint(-4, 5, (case["cols"],), generator=gen, device=DEV).float())
        rational = case["act"] == "rational"
        x = _normal(gen, (case["rows"], case["cols"]), 1.0, torch.float32)
        st["x"] = (x if rational else x * spread).to(TYPES[case["io"]])
        st["A"], st["B"] = _swish_like(gen, 8) if rational else (None, None)
        return st
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        st["a"], st["sa"] = _weights8(gen, m, k, False)
        st["b"], st["sb"] = _weights8(gen, n, k, case["tile"])
        st["bias"] = _normal(gen, (n,), 1.0, torch.float32) if case["bias"] else None
        st["r"] = _normal(gen, (m, n), 1.0, TYPES[case["out"]]) if case["residual"] else None
        return st
    io, c, rows = TYPES[case["io"]], case["c"], case["samples"] * case["positions"]
    shape = (case["samples"], case["positions"], c)
    st["f"] = _normal(gen, shape, 1.0, io, 0.2)
    st["weight"] = 1.0 + _normal(gen, (c,), 0.1, torch.float32)
    st["bias"] = _normal(gen, (c,), 0.1, torch.float32) if case["norm"] == "layer" else None
    st["scale"] = _normal(gen, (c,), 0.1, torch.float32, 0.5)
    post = case["post"] != "none"
    st["post_weight"] = 1.0 + _normal(gen, (c,), 0.1, torch.float32) if post else None
    st["post_bias"] = _normal(gen, (c,), 0.1, torch.float32) if case["post"] == "layer" else None
    st["gate"] = None
    if case["gate"] == "sample":      # stochastic depth: a sample's branch is left out or scaled up
        keep = torch.rand((case["samples"], 1, 1), generator=gen, device=DEV) < 0.9
        st["gate"] = torch.where(keep, 1.0 / 0.9, 0.0)
    elif case["gate"] == "channel":
        st["gate"] = _normal(gen, (case["samples"], 1, c), 0.5, io, 1.0)
    elif case["gate"] == "token":
        st["gate"] = _normal(gen, (*shape[:2], 1), 0.5, io, 1.0)
    elif case["gate"] == "element":
        st["gate"] = _normal(gen, shape, 0.5, io, 1.0)
    if case["way"] == "fwd":
        st["x"] = _normal(gen, shape, 1.5, io, 0.3)
    else:
        # the forward pass kept its result h and the statistics
        st["h"] = _normal(gen, shape, 1.8, io, 0.3)
        st["dh"], st["dz"] = _normal(gen, shape, 1e-2, io), _normal(gen, shape, 1e-2, io)
        stats = [*_moments(st["h"].double().view(rows, c), case["norm"])]
        if post:
            stats += [*_moments(st["f"].double().view(rows, c), case["post"])]
        st["stats"] = torch.stack(stats).float()
    return st


def _moments(v, kind):
    """(mean, 1 / sqrt(var + eps)) of each row; the root mean square's has mean 0."""
    mean = v.mean(dim=1) if kind == "layer" else torch.zeros_like(v[:, 0])
    return mean, 1.0 / torch.sqrt((v - mean[:, None]).square().mean(dim=1) + EPS)


# ---------------------------------------------------------------- the operators' plain forms

def _power_of_two_scale(amax):
    """The smallest 2^e, e >= -126, with amax <= 448 * 2^e; 1 for amax = 0."""
    mant, e = torch.frexp(amax)           # amax = mant 2^e, mant in [1/2, 1); 448 = 7/8 * 2^9
    e = (e - 9 + (mant > 0.875)).clamp_min(-126)
    return torch.where(amax == 0, torch.ones_like(amax), torch.exp2(e.to(amax.dtype)))


def _to_codes(v):
    """(e4m3 codes, scales) of blocks along the last dimension, rounded to nearest."""
    s = _power_of_two_scale(torch.where(v.isfinite(), v.abs(), 0.0).amax(dim=-1))
    return (v / s[..., None]).to(F8), s


def _quantized(x, tile):
    """(codes [rows, cols], scales [rows or row blocks, column blocks]) of fp32 x."""
    rows, cols = x.shape
    rb, cb = _ceil(rows, BLOCK) if tile else rows, _ceil(cols, BLOCK)
    v = torch.nn.functional.pad(x, (0, cb * BLOCK - cols, 0, (rb * BLOCK if tile else rows) - rows))
    v = v.view(rb, -1, cb, BLOCK)
    s = _power_of_two_scale(torch.where(v.isfinite(), v.abs(), 0.0).amax(dim=(1, 3)))
    q = (v / s[:, None, :, None]).to(F8).view(-1, cb * BLOCK)
    return q[:rows, :cols], s


def _rational(x, A, B):
    g = A.shape[0]
    v = x.view(-1, g, x.shape[-1] // g)
    a, b = [t.view(1, g, 1) for t in A.unbind(1)], [t.view(1, g, 1) for t in B.unbind(1)]
    P = ((((a[5] * v + a[4]) * v + a[3]) * v + a[2]) * v + a[1]) * v + a[0]
    Q = (((b[3] * v + b[2]) * v + b[1]) * v + b[0]) * v
    return (P / (1.0 + Q.abs())).view(x.shape)


def _plain_quantize(st):
    case, x = st["case"], st["x"].float()
    if case["act"] == "rational":
        x = _rational(x, st["A"], st["B"])
    out = []
    if case["outputs"] != "columns":
        out += _quantized(x, case["tile"])
    if case["outputs"] != "rows":
        out += _quantized(x.t(), case["tile"])
    return tuple(out)


def _values(codes, scale, tile, dtype):
    """The values that codes stand for."""
    s = scale.to(dtype).repeat_interleave(BLOCK, dim=1)[:, :codes.shape[1]]
    if tile:
        s = s.repeat_interleave(BLOCK, dim=0)[:codes.shape[0]]
    return codes.to(torch.float32).to(dtype) * s


def _plain_matmul(st):
    case = st["case"]
    c = _values(st["a"], st["sa"], False, torch.float32) @ _values(st["b"], st["sb"], case["tile"], torch.float32).t()
    if st["bias"] is not None:
        c = c + st["bias"]
    if st["r"] is not None:
        c = c + st["r"].float()
    return c.to(TYPES[case["out"]])


def _normalised(v, kind, weight, bias):
    mean, rstd = _moments(v, kind)
    h = (v - mean[:, None]) * rstd[:, None] * weight
    return (h if bias is None else h + bias), mean, rstd


def _rows_of_gate(st, dtype):
    """The gate at each element's row, broadcast: [samples, positions or 1, c or 1]."""
    return 1.0 if st["gate"] is None else st["gate"].to(dtype)


def _plain_residual(st):
    case = st["case"]
    shape = st["f"].shape
    c, io = shape[-1], st["f"].dtype
    post = case["post"] != "none"
    f = st["f"].float().view(-1, c)
    gate = _rows_of_gate(st, torch.float32)
    if case["way"] == "fwd":
        u, stats = f, ()
        if post:
            u, *stats = _normalised(f, case["post"], st["post_weight"], st["post_bias"])
        h = st["x"].float() + st["scale"] * gate * u.view(shape)
        z, mean, rstd = _normalised(h.view(-1, c), case["norm"], st["weight"], st["bias"])
        return h.to(io), z.view(shape).to(io), torch.stack([mean, rstd, *stats])
    stats = st["stats"][:, :, None]
    dz = st["dz"].float().view(-1, c)
    xh = (st["h"].float().view(-1, c) - stats[0]) * stats[1]
    dh = st["dh"].float().view(-1, c) + _norm_backward(dz * st["weight"], xh, stats[1], case["norm"])
    out = {"dx": dh.view(shape).to(io), "dweight": (dz * xh).sum(0)}
    if case["norm"] == "layer":
        out["dbias"] = dz.sum(0)
    u, fh = f, None
    if post:
        fh = (f - stats[2]) * stats[3]
        u = fh * st["post_weight"]
        if st["post_bias"] is not None:
            u = u + st["post_bias"]
    dh, u = dh.view(shape), u.view(shape)
    out["dscale"] = (dh * gate * u).sum(dim=(0, 1))
    if st["gate"] is not None:
        dg = dh * st["scale"] * u
        over = [d for d in (1, 2) if st["gate"].shape[d] == 1 and shape[d] > 1]
        out["dgate"] = (dg.sum(dim=over, keepdim=True) if over else dg).to(st["gate"].dtype)
    du = (dh * gate * st["scale"]).view(-1, c)
    if post:
        out["dpost_weight"] = (du * fh).sum(0)
        if case["post"] == "layer":
            out["dpost_bias"] = du.sum(0)
        du = _norm_backward(du * st["post_weight"], fh, stats[3], case["post"])
    out["df"] = du.view(shape).to(io)
    return out


def _norm_backward(t, xh, rstd, kind):
    t = t - xh * (t * xh).mean(dim=1, keepdim=True) - (t.mean(dim=1, keepdim=True) if kind == "layer" else 0.0)
    return t * rstd


BETA1, BETA2, ADAM_EPS, DECAY = 0.9, 0.999, 1e-8, 0.05


def _mix(h):
    """A 32-bit value from a 32-bit value (held in 64): xor-shifts and odd factors."""
    h = ((h ^ (h >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _random16(st, first_block, blocks):
    """Two numbers of 16 bits for each value of the blocks: the operator's random numbers are a function of
    (seed, step, block, place), its seed an input."""
    key = torch.tensor([st["seed"] & 0xFFFFFFFF], device=DEV)
    key = _mix((_mix(key) + st["step"]) & 0xFFFFFFFF)
    block = torch.arange(first_block, first_block + blocks, device=DEV)
    h = _mix((_mix((key + block) & 0xFFFFFFFF)[:, None] + torch.arange(BLOCK, device=DEV)) & 0xFFFFFFFF)
    return h & 0xFFFF, h >> 16


def _stochastic(v, random16):
    """(codes, scales) of non-negative or signed blocks [n, 128], rounded up with the probability of the
    remainder: 3 bits of mantissa are kept, and below 2^-6 multiples of 2^-9."""
    s = _power_of_two_scale(torch.where(v.isfinite(), v.abs(), 0.0).amax(dim=-1))
    y = v / s[:, None]
    a = y.abs()
    low = a < 2.0 ** -6
    bits = (a + low * 2.0 ** -6).view(torch.int32) + (random16 * 16 + 8).to(torch.int32)
    a = (bits & ~0xFFFFF).view(torch.float32) - low * 2.0 ** -6
    return torch.where(y < 0, -a, a), s


def _step(st, g, p, m, v):
    """(p, m, v) after the step, fp32."""
    t, lr = st["step"], st["lr"]
    if st["grad_scale"] is not None:
        g = g * st["grad_scale"]
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g * g
    d = v.sqrt() * (1.0 / math.sqrt(1.0 - BETA2 ** t)) + ADAM_EPS
    return p * (1.0 - lr * DECAY) - (lr / (1.0 - BETA1 ** t)) * (m / d), m, v


def _plain_adamw_part(st, k, first_block):
    g, p = st[k + "_grad"].float(), st[k + "_master"]
    out = {}
    if st["case"]["bits"] == 32:
        q, m, v = _step(st, g, p, st[k + "_m"], st[k + "_v"])
        st[k + "_m"].copy_(m)
        st[k + "_v"].copy_(v)
        out = {"m": st[k + "_m"], "v": st[k + "_v"]}
    else:
        m = (st[k + "_m"].float() * st[k + "_ms"][:, None]).view(-1)
        r = (st[k + "_r"].float() * st[k + "_rs"][:, None]).view(-1)
        q, m, v = _step(st, g, p, m, r * r)
        one, two = _random16(st, first_block, m.numel() // BLOCK)
        code, scale = _stochastic(m.view(-1, BLOCK), one)
        st[k + "_m"].copy_(code.to(F8))
        st[k + "_ms"].copy_(scale)
        r = v.sqrt().view(-1, BLOCK)
        code, scale = _stochastic(r, two)
        # the root of a moment that is not 0 is not rounded to 0: it divides
        code = torch.where(r > 0, code.clamp_min(2.0 ** -9), code)
        st[k + "_r"].copy_(code.to(F8))
        st[k + "_rs"].copy_(scale)
        out = {"m": st[k + "_m"], "ms": st[k + "_ms"], "r": st[k + "_r"], "rs": st[k + "_rs"]}
    p.copy_(q)
    return {k + "_" + name: t for name, t in {**out, "master": p}.items()}


def _plain_adamw(st):
    out = {**_plain_adamw_part(st, "w", 0), **_plain_adamw_part(st, "b", st["w_grad"].numel() // BLOCK)}
    st["w_param"].copy_(st["w_master"])
    return {**out, "w_param": st["w_param"]}


# ---------------------------------------------------------------- the library's operators

def _own_quantize(st):
    from gr_kan_rational_amd import grkan_fp8_quantize

    case = st["case"]
    return grkan_fp8_quantize(st["x"], outputs=case["outputs"], tile=case["tile"], act=case["act"], A=st["A"],
                              B=st["B"], n_groups=8)


def _own_matmul(st):
    from gr_kan_rational_amd import grkan_fp8_matmul

    return grkan_fp8_matmul(st["a"], st["sa"], st["b"], st["sb"], bias=st["bias"], residual=st["r"],
                            dtype=TYPES[st["case"]["out"]])


def _own_residual(st):
    from gr_kan_rational_amd import grkan_residual_norm_backward, grkan_residual_norm_forward

    case = st["case"]
    params = dict(norm=case["norm"], weight=st["weight"], bias=st["bias"], scale=st["scale"], gate=st["gate"],
                  post=case["post"], post_weight=st["post_weight"], post_bias=st["post_bias"])
    if case["way"] == "fwd":
        return grkan_residual_norm_forward(st["x"], st["f"], eps=EPS, **params)
    got = grkan_residual_norm_backward(st["f"], st["h"], st["dh"], st["dz"], st["stats"], **params)
    names = ("dx", "df", "dscale", "dgate", "dweight", "dbias", "dpost_weight", "dpost_bias")
    return {k: v for k, v in zip(names, got) if v is not None}


def _own_adamw(st):
    from gr_kan_rational_amd import grkan_adamw_step

    eight = st["case"]["bits"] == 8
    grkan_adamw_step(st["params"], st["grads"], st["avgs"], st["sqs"], step=st["step"], lr=st["lr"], beta1=BETA1,
                     beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY, masters=st["masters"],
                     avg_scales=st["avg_scales"] if eight else None, sq_scales=st["sq_scales"] if eight else None,
                     grad_scale=st["grad_scale"], seed=st["seed"])
    kept = ("m", "ms", "r", "rs", "master") if eight else ("m", "v", "master")
    return {**{k + "_" + name: st[k + "_" + name] for k in ("w", "b") for name in kept}, "w_param": st["w_param"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"quantize": _own_quantize, "matmul": _own_matmul, "residual": _own_residual,
                "adamw": _own_adamw}[op](state)
    return {"quantize": _plain_quantize, "matmul": _plain_matmul, "residual": _plain_residual,
            "adamw": _plain_adamw}[op](state)


# ---------------------------------------------------------------- the definitions in fp64

def _exact_scale(amax):
    s = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)).clamp_min(-126.0))
    s = torch.where(amax / (s / 2) <= E4M3_MAX, s / 2, s)      # a logarithm that came out too large
    s = torch.where(amax / s > E4M3_MAX, s * 2, s)             # or too small
    return torch.where(amax == 0, 1.0, s)


def _e4m3_step(a):
    """The distance of e4m3 values at a >= 0."""
    return torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3.0)


def _exact_quantized(x, tile):
    rows, cols = x.shape
    rb, cb = _ceil(rows, BLOCK) if tile else rows, _ceil(cols, BLOCK)
    v = x.new_zeros((rb * BLOCK if tile else rows, cb * BLOCK))
    v[:rows, :cols] = x
    s = _exact_scale(v.view(rb, -1, cb, BLOCK).abs().amax(dim=(1, 3)))
    y = x / s.repeat_interleave(BLOCK, 1)[:, :cols].repeat_interleave(BLOCK if tile else 1, 0)[:rows]
    step = _e4m3_step(y.abs())
    return torch.round(y / step) * step, s          # torch.round: halves to even


def _exact_quantize(case, st):
    x = st["x"].double()
    if case["act"] == "rational":
        c = x.shape[-1]
        a, b = st["A"].double().repeat_interleave(c // 8, 0), st["B"].double().repeat_interleave(c // 8, 0)
        P = sum(a[:, i] * x ** i for i in range(6))
        x = P / (1.0 + sum(b[:, j] * x ** (j + 1) for j in range(4)).abs())
    out = []
    if case["outputs"] != "columns":
        out += _exact_quantized(x, case["tile"])
    if case["outputs"] != "rows":
        out += _exact_quantized(x.t(), case["tile"])
    return tuple(out)


def _exact_matmul(case, st):
    c = torch.mm(_values(st["a"], st["sa"], False, torch.float64),
                 _values(st["b"], st["sb"], case["tile"], torch.float64).t())
    if st["bias"] is not None:
        c += st["bias"].double()
    if st["r"] is not None:
        c += st["r"].double()
    return c


def _exact_residual(case, st):
    """The forward by its formulas; the backward by autograd of the formulas in fp64, as d/d(x, f, ...) of
    sum(dh h + dz z) at the x that gives h."""
    shape, c = st["f"].shape, case["c"]
    post = case["post"] != "none"

    def leaf(t):
        return None if t is None else t.double().requires_grad_(case["way"] == "bwd")

    f, w, b, s, g = (leaf(st[k]) for k in ("f", "weight", "bias", "scale", "gate"))
    pw, pb = leaf(st["post_weight"]), leaf(st["post_bias"])

    def norm(v, kind, weight, bias):
        mean = v.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(v[..., :1])
        rstd = ((v - mean).square().mean(-1, keepdim=True) + EPS) ** -0.5
        y = (v - mean) * rstd * weight
        return (y if bias is None else y + bias), mean.reshape(-1), rstd.reshape(-1)

    u, stats = f, []
    if post:
        u, *stats = norm(f, case["post"], pw, pb)
    branch = s * u if g is None else s * g * u
    x = st["x"].double() if case["way"] == "fwd" else (st["h"].double() - branch).detach().requires_grad_()
    h = x + branch
    z, mean, rstd = norm(h, case["norm"], w, b)
    if case["way"] == "fwd":
        return h, z, torch.stack([mean, rstd, *stats])
    loss = (st["dh"].double() * h).sum() + (st["dz"].double() * z).sum()
    leaves = {"dx": x, "df": f, "dscale": s, "dgate": g, "dweight": w, "dbias": b, "dpost_weight": pw, "dpost_bias": pb}
    leaves = {k: v for k, v in leaves.items() if v is not None}
    return dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))


def _exact_adamw(case, st):
    t, lr, out, first = st["step"], st["lr"], {}, 0
    clip = 1.0 if st["grad_scale"] is None else st["grad_scale"].double()
    for k in ("w", "b"):
        g, p = st[k + "_grad"].double() * clip, st[k + "_master"].double()
        if case["bits"] == 32:
            m, v = st[k + "_m"].double(), st[k + "_v"].double()
        else:
            m = (st[k + "_m"].float().double() * st[k + "_ms"].double()[:, None]).view(-1)
            v = (st[k + "_r"].float().double() * st[k + "_rs"].double()[:, None]).view(-1).square()
        m = m + (1.0 - BETA1) * (g - m)
        v = v + (1.0 - BETA2) * (g * g - v)
        mh, vh = m / (1.0 - BETA1 ** t), v / (1.0 - BETA2 ** t)
        out[k + "_master"] = p - lr * (DECAY * p + mh / (torch.sqrt(vh) + ADAM_EPS))
        if case["bits"] == 32:
            out[k + "_m"], out[k + "_v"] = m, v
            continue
        blocks = m.numel() // BLOCK
        for name, value, random in zip("mr", (m, torch.sqrt(v)), _random16(st, first, blocks)):
            value = value.view(blocks, BLOCK)
            s = _exact_scale(value.abs().amax(dim=1))
            y = value.abs() / s[:, None]
            step = _e4m3_step(y)
            code = torch.floor(y / step + (random + 0.5) / 65536.0) * step
            if name == "r":
                code = torch.where(y > 0, code.clamp_min(2.0 ** -9), code)
            out[k + "_" + name], out[k + "_" + name + "s"] = code * value.sign(), s
        first += blocks
    return {**out, "w_param": out["w_master"].clone()}


def exact(case, seed):
    st = prepare(case, seed)
    return {"quantize": _exact_quantize, "matmul": _exact_matmul, "residual": _exact_residual,
            "adamw": _exact_adamw}[case["op"]](case, st)


# ---------------------------------------------------------------- the least work

def work(case):
    if case["op"] == "quantize":
        rows, cols = case["rows"], case["cols"]
        e, es = rows * cols, 4 if case["io"] == "f32" else 2
        scales = 0
        if case["outputs"] != "columns":
            scales += (_ceil(rows, BLOCK) if case["tile"] else rows) * _ceil(cols, BLOCK)
        if case["outputs"] != "rows":
            scales += (_ceil(cols, BLOCK) if case["tile"] else cols) * _ceil(rows, BLOCK)
        outs = 2 if case["outputs"] == "both" else 1
        return {"bytes": e * (es + outs) + 4 * scales, "flops": e * (2 * outs + (21 if case["act"] == "rational" else 0))}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        es, kb = 4 if case["out"] == "f32" else 2, _ceil(k, BLOCK)
        scales = m * kb + (_ceil(n, BLOCK) if case["tile"] else n) * kb
        return {"bytes": (m + n) * k + 4 * scales + m * n * es * (1 + case["residual"]) + 4 * n * case["bias"],
                "flops": 2 * m * n * k}
    if case["op"] == "residual":
        rows, c = case["samples"] * case["positions"], case["c"]
        e, es = rows * c, 4 if case["io"] == "f32" else 2
        gate = {"none": 0, "sample": 4 * case["samples"], "channel": case["samples"] * c * es, "token": rows * es,
                "element": e * es}[case["gate"]]
        stats = 8 * rows * (1 if case["post"] == "none" else 2)
        vectors = 4 * c * (2 + (case["norm"] == "layer") + {"none": 0, "rms": 1, "layer": 2}[case["post"]])
        if case["way"] == "fwd":
            return {"bytes": 4 * e * es + gate + stats + vectors, "flops": e * (10 if case["post"] == "none" else 18)}
        return {"bytes": 6 * e * es + 2 * gate + stats + 2 * vectors, "flops": e * (24 if case["post"] == "none" else 40)}
    mats, vecs = _shapes(case)
    w = case["blocks"] * sum(math.prod(s) for s in mats)
    b = case["blocks"] * sum(math.prod(s) for s in vecs)
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK      # both moments, read and written
    return {"bytes": w * (2 + 8 + 2 + state) + b * (4 + 8 + state), "flops": 15 * (w + b)}
