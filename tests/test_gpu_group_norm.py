"""GPU tests of the group norm with an activation (channels last) against its definition in fp64; the
bounds are derived in tests/block_ref.py."""
import math

import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ("none", "silu", "gelu", "rational")

# (samples, positions, channels, norm groups, activation groups)
SHAPES = [
    # one position: lanes of a wave, of several waves, one lane; ragged accesses
    (1, 1, 768, 1, 8), (5, 1, 192, 8, 8), (3, 1, 37, 1, 1), (2, 1, 10, 10, 10), (7, 1, 48, 3, 8), (4, 1, 4096, 1, 8),
    (300, 1, 96, 1, 8), (130, 1, 1, 1, 1), (6, 1, 1500, 5, 10), (2, 1, 7000, 1, 8), (1100, 1, 64, 4, 8),
    # one position, activation groups that end inside a lane's columns, or of few channels
    (20, 1, 1000, 1, 8), (9, 1, 528, 1, 8), (6, 1, 296, 1, 8), (5, 1, 180, 2, 6), (3, 1, 300, 1, 300),
    (4, 1, 640, 1, 128), (11, 1, 36, 2, 12),
    # one position, a group beyond one workgroup
    (3, 1, 1100, 1, 1100),
    (2, 1, 20001, 1, 1),
    # several positions, a group in one workgroup
    (2, 7, 32, 4, 8), (3, 197, 96, 1, 8), (2, 49, 320, 32, 8), (9, 5, 33, 3, 3), (1, 2, 8, 8, 8), (17, 3, 24, 2, 4),
    (8, 197, 192, 8, 8), (2, 2, 2048, 1, 8), (40, 16, 40, 8, 8),
    # a group beyond one workgroup
    (1, 3000, 64, 32, 8), (2, 4097, 40, 4, 8), (1, 900, 1000, 1, 8), (3, 70, 9000, 2, 8), (1, 20000, 5, 5, 1),
]


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


def coefficients(groups, gen):
    """Coefficients of a Swish fit (an even, positive denominator), each group's a little off it."""
    A = torch.tensor([0.0, 0.5, 0.249944, 0.0526866, 0.00555034, 0.000244433]).repeat(groups, 1)
    B = torch.tensor([0.0, 0.105373, 0.0, 0.000488866]).repeat(groups, 1)
    A = A * (1 + 0.1 * torch.rand(A.shape, generator=gen)) + 0.05
    B = B * (1 + 0.1 * torch.rand(B.shape, generator=gen))
    return A, B


def make(shape, dtype, act, seed, affine=True, mean=0.3):
    n, s, c, g, ng = shape
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((n, s, c), generator=gen) * 1.5 + mean).to(dtype)
    dy = (torch.randn((n, s, c), generator=gen) * 0.1).to(dtype)
    w = 1 + 0.2 * torch.randn(c, generator=gen) if affine else None
    b = 0.2 * torch.randn(c, generator=gen) if affine else None
    A, B = coefficients(ng, gen) if act == "rational" else (None, None)
    return x, dy, w, b, A, B


def gpu(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def name(shape):
    return "x".join(map(str, shape))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("io", DTYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=name)
def test_forward_and_backward(gk, shape, io, act):
    print(f"[group norm] {name(shape)} {io} {act}", flush=True)
    n, s, c, g, ng = shape
    x, dy, w, b, A, B = make(shape, DTYPES[io], act, 100 + n + s + c)
    X, DY, W, Bi, Ad, Bd = gpu(x, dy, w, b, A, B)
    y, mean, rstd = gk.grkan_group_norm_forward(X, g, W, Bi, 1e-5, act, Ad, Bd, ng)
    want = ref.norm_forward(x, g, w, b, 1e-5, act, A, B)
    for k, got in (("mean", mean), ("rstd", rstd), ("y", y)):
        ref.check(f"{name(shape)} {k}", got, *want[k])
    grads = gk.grkan_group_norm_backward(X, DY, mean, rstd, g, W, Bi, act, Ad, Bd, ng)
    want = ref.norm_backward(x, dy, mean.cpu(), rstd.cpu(), g, w, b, act, A, B)
    for k, got in zip(("dx", "dweight", "dbias", "dA", "dB"), grads):
        if k in want:
            ref.check(f"{name(shape)} {k}", got, *want[k])
        else:
            assert got is None
    again = gk.grkan_group_norm_backward(X, DY, mean, rstd, g, W, Bi, act, Ad, Bd, ng)
    for p, q in zip(grads, again):
        assert p is None or torch.equal(p, q), "two calls differ"


@pytest.mark.parametrize("shape", [(4, 1, 96, 1, 8), (3, 50, 96, 4, 8), (1, 3000, 64, 8, 8)], ids=name)
def test_without_weight_and_bias(gk, shape):
    n, s, c, g, ng = shape
    x, dy, _, _, _, _ = make(shape, torch.float32, "silu", 7, affine=False)
    X, DY = gpu(x, dy)
    y, mean, rstd = gk.grkan_group_norm_forward(X, g, act="silu")
    ref.check("y", y, *ref.norm_forward(x, g, None, None, 1e-5, "silu")["y"])
    dx, dw, db, dA, dB = gk.grkan_group_norm_backward(X, DY, mean, rstd, g, act="silu")
    want = ref.norm_backward(x, dy, mean.cpu(), rstd.cpu(), g, None, None, "silu")
    ref.check("dx", dx, *want["dx"])
    ref.check("dweight", dw, *want["dweight"])
    ref.check("dbias", db, *want["dbias"])


@pytest.mark.parametrize("act", ("none", "rational"))
@pytest.mark.parametrize("shape", [(6, 1, 96, 1, 8), (3, 50, 96, 4, 8), (2, 3000, 64, 8, 8)], ids=name)
@pytest.mark.parametrize("io", DTYPES)
def test_strided_and_unaligned_inputs(gk, shape, io, act):
    """Positions dropped, channels sliced at an odd offset, an output off its 16-byte boundary: the values
    of the dense tensors, and nothing written outside the output."""
    n, s, c, g, ng = shape
    x, dy, w, b, A, B = make(shape, DTYPES[io], act, 11)
    X, DY, W, Bi, Ad, Bd = gpu(x, dy, w, b, A, B)
    xw = torch.randn((n, s + 2, c + 5), device=DEV).to(DTYPES[io])
    xw[:, 1:-1, 3:-2] = X
    xs = xw[:, 1:-1, 3:-2]
    gw = torch.randn((n, s + 1, c + 1), device=DEV).to(DTYPES[io])
    gw[:, 1:, 1:] = DY
    gs = gw[:, 1:, 1:]
    buf = torch.full((n * s * c + 2,), 7.0, dtype=DTYPES[io], device=DEV)
    out = buf[1:-1].view(n, s, c)
    y0, m0, r0 = gk.grkan_group_norm_forward(X, g, W, Bi, 1e-5, act, Ad, Bd, ng)
    y1, m1, r1 = gk.grkan_group_norm_forward(xs, g, W, Bi, 1e-5, act, Ad, Bd, ng, out=out)
    assert torch.equal(y0, y1) and torch.equal(m0, m1) and torch.equal(r0, r1)
    assert float(buf[0]) == 7.0 and float(buf[-1]) == 7.0
    d0 = gk.grkan_group_norm_backward(X, DY, m0, r0, g, W, Bi, act, Ad, Bd, ng)
    d1 = gk.grkan_group_norm_backward(xs, gs, m0, r0, g, W, Bi, act, Ad, Bd, ng, dx=out)
    for p, q in zip(d0, d1):
        assert p is None or torch.equal(p, q)
    assert float(buf[0]) == 7.0 and float(buf[-1]) == 7.0


@pytest.mark.parametrize("shape", [(6, 1, 96, 1, 8), (3, 50, 96, 4, 8), (2, 3000, 64, 8, 8)], ids=name)
def test_in_place(gk, shape):
    n, s, c, g, ng = shape
    x, dy, w, b, A, B = make(shape, torch.float32, "rational", 12)
    X, DY, W, Bi, Ad, Bd = gpu(x, dy, w, b, A, B)
    y, mean, rstd = gk.grkan_group_norm_forward(X, g, W, Bi, 1e-5, "rational", Ad, Bd, ng)
    x2 = X.clone()
    gk.grkan_group_norm_forward(x2, g, W, Bi, 1e-5, "rational", Ad, Bd, ng, out=x2)
    assert torch.equal(y, x2)
    dx = gk.grkan_group_norm_backward(X, DY, mean, rstd, g, W, Bi, "rational", Ad, Bd, ng)[0]
    for which in (0, 1):
        xc, gc = X.clone(), DY.clone()
        got = gk.grkan_group_norm_backward(xc, gc, mean, rstd, g, W, Bi, "rational", Ad, Bd, ng,
                                           dx=xc if which == 0 else gc)[0]
        assert torch.equal(dx, got)


@pytest.mark.parametrize("shape", [(4, 1, 96, 4, 8), (4, 30, 96, 4, 8), (2, 3000, 64, 4, 8)], ids=name)
@pytest.mark.parametrize("bad", (float("nan"), float("inf"), -float("inf")))
def test_non_finite_values_stay_in_their_group(gk, shape, bad):
    n, s, c, g, ng = shape
    x, dy, w, b, _, _ = make(shape, torch.float32, "silu", 13)
    X, DY, W, Bi = gpu(x, dy, w, b)
    y0, _, _ = gk.grkan_group_norm_forward(X, g, W, Bi, 1e-5, "silu")
    X2 = X.clone()
    X2[1, s // 2, c // g + 1] = bad  # sample 1, group 1
    y1, _, _ = gk.grkan_group_norm_forward(X2, g, W, Bi, 1e-5, "silu")
    y0, y1 = y0.view(n, s, g, -1), y1.view(n, s, g, -1)
    assert torch.isnan(y1[1, :, 1]).all()
    keep = torch.ones((n, g), dtype=torch.bool, device=DEV)
    keep[1, 1] = False
    assert torch.equal(y0.transpose(1, 2)[keep], y1.transpose(1, 2)[keep])


@pytest.mark.parametrize("shape", [(3, 1, 256, 1, 8), (3, 60, 64, 2, 8), (1, 5000, 64, 2, 8)], ids=name)
def test_mean_far_from_zero_and_constant_groups(gk, shape):
    n, s, c, g, ng = shape
    x, _, w, b, _, _ = make(shape, torch.float32, "none", 14, mean=3000.0)
    x[0] = 5.0  # variance 0: rstd = 1 / sqrt(eps)
    X, W, Bi = gpu(x, w, b)
    y, mean, rstd = gk.grkan_group_norm_forward(X, g, W, Bi, 1e-5)
    want = ref.norm_forward(x, g, w, b, 1e-5, "none")
    for k, got in (("mean", mean), ("rstd", rstd), ("y", y)):
        ref.check(k, got, *want[k])


@pytest.mark.parametrize("shape", [(3, 1, 48, 1, 8), (2, 20, 48, 4, 8), (1, 2500, 48, 4, 8)], ids=name)
@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(gk, shape, act):
    """The loss sum(g y) along a random direction of all inputs: a central difference of the kernel's own
    forward.  Step 2^-7: truncation ~ step^2 of the third derivative, rounding ~ u |terms| / step."""
    n, s, c, g, ng = shape
    x, dy, w, b, A, B = make(shape, torch.float32, act, 15)
    X, DY, W, Bi, Ad, Bd = gpu(x, dy, w, b, A, B)
    y, mean, rstd = gk.grkan_group_norm_forward(X, g, W, Bi, 1e-5, act, Ad, Bd, ng)
    grads = gk.grkan_group_norm_backward(X, DY, mean, rstd, g, W, Bi, act, Ad, Bd, ng)
    gen = torch.Generator().manual_seed(16)
    ins = [X, W, Bi] + ([Ad, Bd] if act == "rational" else [])
    dirs = [torch.randn(t.shape, generator=gen).to(DEV) for t in ins]
    if act == "rational":
        dirs[-1] = dirs[-1] * Bd  # the denominator keeps its even, positive form
    h = 2.0 ** -7

    def loss(sign):
        v = [t + sign * h * d for t, d in zip(ins, dirs)]
        out = gk.grkan_group_norm_forward(v[0], g, v[1], v[2], 1e-5, act, *(v[3:] or (None, None)), ng)[0]
        return (out.double() * DY.double()).sum()

    num = (loss(1) - loss(-1)) / (2 * h)
    terms = [(gr.double() * d.double()) for gr, d in zip(grads, dirs)]
    ana = sum(t.sum() for t in terms)
    scale = math.sqrt(sum(float((t ** 2).sum()) for t in terms)) + float((y.double() * DY.double()).norm())
    assert abs(float(num - ana)) <= 2e-3 * scale


def test_no_elements(gk):
    W = torch.ones(32, device=DEV)
    y, mean, rstd = gk.grkan_group_norm_forward(torch.empty((3, 0, 32), device=DEV), 4, W, W, 1e-4)
    assert y.shape == (3, 0, 32) and float(mean.abs().max()) == 0.0
    assert torch.allclose(rstd, torch.full_like(rstd, 100.0))
    assert gk.grkan_group_norm_forward(torch.empty((0, 5, 32), device=DEV), 4, W, W)[0].shape == (0, 5, 32)
    A, B = (t.to(DEV) for t in coefficients(8, torch.Generator()))
    for shape in ((3, 0, 32), (0, 5, 32)):
        x = torch.empty(shape, device=DEV)
        st = torch.ones((shape[0], 4), device=DEV)
        out = gk.grkan_group_norm_backward(x, x, st, st, 4, W, W, "rational", A, B, 8)
        assert out[0].shape == shape
        for t in out[1:]:
            assert float(t.abs().max()) == 0.0


def test_another_stream(gk):
    """Everything, allocations included, on the stream given; the results are those of the current one."""
    x, dy, w, b, A, B = make((2, 3000, 64, 8, 8), torch.float32, "rational", 17)
    X, DY, W, Bi, Ad, Bd = gpu(x, dy, w, b, A, B)
    args = (W, Bi, 1e-5, "rational", Ad, Bd, 8)
    y, mean, rstd = gk.grkan_group_norm_forward(X, 8, *args)
    d = gk.grkan_group_norm_backward(X, DY, mean, rstd, 8, W, Bi, "rational", Ad, Bd, 8)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for stream in (st, st.cuda_stream):
        y1, m1, r1 = gk.grkan_group_norm_forward(X, 8, *args, stream=stream)
        d1 = gk.grkan_group_norm_backward(X, DY, m1, r1, 8, W, Bi, "rational", Ad, Bd, 8, stream=stream)
        st.synchronize()
        assert torch.equal(y, y1) and all(torch.equal(p, q) for p, q in zip(d, d1))


@pytest.mark.parametrize("way", ("tokens", "images", "map"))
def test_offsets_past_32_bits(gk, way):
    """More than 2^31 elements of bf16: the last rows have the values of a tensor of their own."""
    c = 1024
    rows = (1 << 31) // c + 5
    shape = {"tokens": (rows, 1, c), "images": (rows // 64 + 1, 64, c), "map": (1, rows, c)}[way]
    x = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
    flat = x.view(-1, c)
    tail = torch.randn((64, c), generator=torch.Generator().manual_seed(18)).to(torch.bfloat16)
    flat[-64:] = tail.to(DEV)
    g = 8 if way == "images" else 1
    y, mean, rstd = gk.grkan_group_norm_forward(x, g)
    dx = gk.grkan_group_norm_backward(x, y, mean, rstd, g, dx=y if way == "tokens" else None)[0]
    torch.cuda.synchronize()
    if way == "map":
        m, r = float(mean[0, 0]), float(rstd[0, 0])
        total = float(shape[1]) * c
        want_m = float(tail.double().sum()) / total
        want_r = 1 / math.sqrt(float((tail.double() ** 2).sum()) / total - want_m ** 2 + 1e-5)
        assert abs(m - want_m) <= 1e-6 * abs(want_m) + 1e-12 and abs(r - want_r) <= 1e-5 * want_r
        want = (tail.double() - m) * r
        ref.check("y", y.view(-1, c)[-64:], want, ref.rounding(want, torch.bfloat16) + 8 * ref.U * want.abs())
    else:
        small = tail.to(DEV).view((64, 1, c) if way == "tokens" else (1, 64, c))
        y1, m1, r1 = gk.grkan_group_norm_forward(small, g)
        d1 = gk.grkan_group_norm_backward(small, y1, m1, r1, g)[0]
        assert torch.equal(rstd[-m1.shape[0]:], r1) and torch.equal(mean[-m1.shape[0]:], m1)
        assert torch.equal(dx.view(-1, c)[-64:], d1.view(-1, c))


def test_autograd(gk):
    x, dy, w, b, A, B = make((4, 30, 96, 4, 8), torch.float32, "rational", 19)
    leaves = [t.to(DEV).requires_grad_() for t in (x, w, b, A, B)]
    X, W, Bi, Ad, Bd = leaves
    y = gk.GRKANGroupNorm.apply(X, 4, W, Bi, 1e-5, "rational", Ad, Bd, 8)
    y.backward(dy.to(DEV))
    _, mean, rstd = gk.grkan_group_norm_forward(X.detach(), 4, W.detach(), Bi.detach())
    want = gk.grkan_group_norm_backward(X.detach(), dy.to(DEV), mean, rstd, 4, W.detach(), Bi.detach(), "rational",
                                        Ad.detach(), Bd.detach(), 8)
    for leaf, g in zip(leaves, want):
        assert torch.equal(leaf.grad, g)
