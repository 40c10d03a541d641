"""GPU tests of the linear map with bias, activation and residual in its epilogue, and of its backward,
against the definitions in fp64; the bounds are derived in tests/block_ref.py."""
import math

import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
ACTS = ("none", "silu", "gelu", "rational")

# (rows, d_in, d_out, activation groups)
SHAPES = [
    # few rows
    (1, 768, 256, 8), (1, 1, 1, 1), (3, 37, 19, 1), (16, 64, 48, 8), (17, 200, 40, 8), (33, 129, 72, 8),
    (64, 512, 64, 8), (5, 1000, 1000, 10),
    # small tiles, odd widths, a rational with groups that end inside a chunk
    (65, 64, 64, 8), (100, 96, 200, 8), (197, 768, 384, 8), (130, 77, 51, 3), (257, 1001, 130, 2), (300, 64, 100, 10),
    # the k range split
    (70, 4096, 64, 8), (200, 3001, 40, 1), (5000, 48, 56, 7),
]
# the larger tiles (forward; dx; dW), whole and odd
LARGE = [(2050, 72, 4104, 8), (4100, 40, 4104, 8), (4099, 37, 4101, 1), (4100, 4104, 40, 8), (4097, 4099, 35, 5),
         (40, 4104, 4104, 8), (35, 4101, 4099, 1), (20000, 264, 520, 8)]


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


def make(shape, act, seed):
    rows, d_in, d_out, ng = shape
    gen = torch.Generator().manual_seed(seed)

    def normal(size, std):
        return (torch.randn(size, generator=gen) * std).to(DEV)

    x, W = normal((rows, d_in), 1.0).to(BF), normal((d_out, d_in), d_in ** -0.5).to(BF)
    bias, r = normal((d_out,), 0.3), normal((rows, d_out), 1.0).to(BF)
    dz, pre = normal((rows, d_out), 0.1).to(BF), normal((rows, d_out), 1.2).to(BF)
    A = normal((ng, 6), 0.5) if act == "rational" else None
    B = normal((ng, 4), 0.5) if act == "rational" else None
    return x, W, bias, r, dz, pre, A, B


def name(shape):
    return "x".join(map(str, shape))


def both_ways(gk, shape, act, seed):
    print(f"[linear] {name(shape)} {act}", flush=True)
    ng = shape[3]
    x, W, bias, r, dz, pre, A, B = make(shape, act, seed)
    z, h = gk.grkan_linear_act_forward(x, W, bias, act, A, B, ng, residual=r, keep=True)
    want = ref.linear_forward(x, W, bias, act, A, B, r)
    ref.check(f"{name(shape)} pre", h, *want["pre"])
    ref.check(f"{name(shape)} z", z, *want["z"])
    grads = gk.grkan_linear_act_backward(x, W, dz, pre, act, A, B, ng)
    want = ref.linear_backward(x, W, dz, pre, act, A, B)
    for k, got in zip(("dx", "dW", "dbias", "dA", "dB"), grads):
        if k in want:
            ref.check(f"{name(shape)} {k}", got, *want[k])
        else:
            assert got is None
    return (x, W, bias, r, dz, pre, A, B), z, h, grads


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", SHAPES, ids=name)
def test_forward_and_backward(gk, shape, act):
    (x, W, bias, r, dz, pre, A, B), z, h, grads = both_ways(gk, shape, act, 200 + sum(shape))
    z2, h2 = gk.grkan_linear_act_forward(x, W, bias, act, A, B, shape[3], residual=r, keep=True)
    assert torch.equal(z, z2) and torch.equal(h, h2)
    for p, q in zip(grads, gk.grkan_linear_act_backward(x, W, dz, pre, act, A, B, shape[3])):
        assert p is None or torch.equal(p, q), "two calls differ"


@pytest.mark.parametrize("act", ("gelu", "rational"))
@pytest.mark.parametrize("shape", LARGE, ids=name)
def test_larger_tiles(gk, shape, act):
    both_ways(gk, shape, act, 300 + sum(shape))


# 256-row tiles: one round, and whole rounds with the other rows in smaller tiles (forward; dx); dW in splits
@pytest.mark.parametrize("act", ("silu", "rational"))
@pytest.mark.parametrize("shape", [(4095, 2056, 3944, 8), (8449, 1032, 2040, 8), (8450, 2040, 1032, 8)], ids=name)
def test_largest_tiles(gk, shape, act):
    both_ways(gk, shape, act, 400 + sum(shape))


@pytest.mark.parametrize("shape", [(1, 96, 80, 8), (70, 96, 80, 8), (40, 33, 27, 1)], ids=name)
def test_optional_arguments(gk, shape):
    """No bias, no residual, no pre: each alone and all together."""
    x, W, bias, r, dz, pre, _, _ = make(shape, "silu", 31)
    for b, res, keep in ((None, None, False), (bias, None, False), (None, r, False), (None, None, True)):
        z, h = gk.grkan_linear_act_forward(x, W, b, "silu", residual=res, keep=keep)
        want = ref.linear_forward(x, W, b, "silu", residual=res)
        ref.check("z", z, *want["z"])
        assert (h is None) != keep
        if keep:
            ref.check("pre", h, *want["pre"])


@pytest.mark.parametrize("shape", [(6, 96, 80, 8), (140, 96, 80, 8), (140, 90, 77, 7)], ids=name)
@pytest.mark.parametrize("act", ("none", "rational"))
def test_strided_and_unaligned(gk, shape, act):
    """Rows of wider tensors, an odd element offset, outputs off their 16-byte boundary: the values of the
    dense tensors within their bounds, and nothing written outside the outputs."""
    rows, d_in, d_out, ng = shape
    x, W, bias, r, dz, pre, A, B = make(shape, act, 32)

    def wide(t, left, right):
        w = torch.randn((t.shape[0], left + t.shape[1] + right), device=DEV).to(BF)
        w[:, left:left + t.shape[1]] = t
        return w[:, left:left + t.shape[1]]

    def odd(size, dtype=BF):
        buf = torch.full((math.prod(size) + 2,), 7.0, dtype=dtype, device=DEV)
        return buf, buf[1:-1].view(size)

    want = ref.linear_forward(x, W, bias, act, A, B, r)
    grad = ref.linear_backward(x, W, dz, pre, act, A, B)
    for left, right in ((3, 2), (8, 8)):
        xs, rs, gs = wide(x, left, right), wide(r, left, right), wide(dz, left, right)
        bz, z = odd((rows, d_out))
        bp, h = odd((rows, d_out))
        gk.grkan_linear_act_forward(xs, W, bias, act, A, B, ng, residual=rs, out=z, pre=h)
        ref.check("z", z, *want["z"])
        ref.check("pre", h, *want["pre"])
        bx, dx = odd((rows, d_in))
        bw, dW = odd((d_out, d_in))
        out = gk.grkan_linear_act_backward(xs, W, gs, pre, act, A, B, ng, dx=dx, dW=dW)
        for k, got in zip(("dx", "dW", "dbias", "dA", "dB"), out):
            if k in grad:
                ref.check(k, got, *grad[k])
        for buf in (bz, bp, bx, bw):
            assert float(buf[0]) == 7.0 and float(buf[-1]) == 7.0
    bw, w2 = odd((d_out, d_in))
    w2.copy_(W)
    ref.check("z", gk.grkan_linear_act_forward(x, w2, bias, act, A, B, ng, residual=r)[0], *want["z"])


@pytest.mark.parametrize("rows", (1, 40, 300))
def test_in_place_on_the_residual(gk, rows):
    x, W, bias, r, _, _, A, B = make((rows, 96, 80, 8), "rational", 33)
    z = gk.grkan_linear_act_forward(x, W, bias, "rational", A, B, 8, residual=r)[0]
    r2 = r.clone()
    gk.grkan_linear_act_forward(x, W, bias, "rational", A, B, 8, residual=r2, out=r2)
    assert torch.equal(z, r2)


@pytest.mark.parametrize("rows", (4, 100))
@pytest.mark.parametrize("bad", (float("nan"), float("inf")))
def test_non_finite_rows_stay_in_their_row(gk, rows, bad):
    """A row of x with a NaN or infinity changes that row of z and dx alone (the zeros past K and past the
    last row must not meet it), and its bits past the tensor's end do not matter."""
    x, W, bias, r, dz, pre, _, _ = make((rows, 100, 72, 8), "silu", 34)
    z0 = gk.grkan_linear_act_forward(x, W, bias, "silu", residual=r)[0]
    x2 = x.clone()
    x2[1, 50] = bad
    z1 = gk.grkan_linear_act_forward(x2, W, bias, "silu", residual=r)[0]
    keep = torch.arange(rows, device=DEV) != 1
    assert torch.equal(z0[keep], z1[keep])
    assert not torch.isfinite(z1[1]).all()
    dx0, dW0 = gk.grkan_linear_act_backward(x, W, dz, pre, "silu")[:2]
    dz2 = dz.clone()
    dz2[1, 7] = bad
    dx1, dW1 = gk.grkan_linear_act_backward(x, W, dz2, pre, "silu")[:2]
    assert torch.equal(dx0[keep], dx1[keep])
    cols = torch.arange(72, device=DEV) != 7
    assert torch.equal(dW0[cols], dW1[cols])


@pytest.mark.parametrize("shape", [(4, 48, 40, 8), (130, 48, 40, 8)], ids=name)
@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(gk, shape, act):
    """The loss sum(g z) along a random direction of bias (and the coefficients): a central difference of
    the kernel's forward, whose z is bf16: half a unit of each z, times |g|, over the step, adds up in
    quadrature; 6 standard deviations, plus 1% for the third derivative at step 2^-3."""
    rows, d_in, d_out, ng = shape
    x, W, bias, _, dz, _, A, B = make(shape, act, 35)
    if act == "rational":  # a smooth unit: an even, positive denominator
        B = B.abs() * torch.tensor([0.0, 1.0, 0.0, 0.02], device=DEV)
    z, pre = gk.grkan_linear_act_forward(x, W, bias, act, A, B, ng, keep=True)
    _, _, db, dA, dB = gk.grkan_linear_act_backward(x, W, dz, pre, act, A, B, ng)
    gen = torch.Generator().manual_seed(36)
    pairs = [(bias, db)] + ([(A, dA), (B, dB)] if act == "rational" else [])
    dirs = [torch.randn(t.shape, generator=gen).to(DEV) * 0.3 for t, _ in pairs]
    if act == "rational":
        dirs[2] = dirs[2] * B
    step = 2.0 ** -3

    def loss(sign):
        v = [t + sign * step * d for (t, _), d in zip(pairs, dirs)]
        return (gk.grkan_linear_act_forward(x, W, v[0], act, *(v[1:] or (None, None)), ng)[0].double() * dz.double()).sum()

    num = float((loss(1) - loss(-1)) / (2 * step))
    terms = [(g.double() * d.double()) for (_, g), d in zip(pairs, dirs)]
    ana = float(sum(t.sum() for t in terms))
    noise = float((2.0 ** -9 * z.double().abs() * dz.double().abs()).norm()) / step
    size = math.sqrt(sum(float((t ** 2).sum()) for t in terms))
    assert abs(num - ana) <= 6 * noise + 0.01 * size


def test_no_rows(gk):
    _, W, bias, _, _, _, A, B = make((1, 33, 24, 8), "rational", 37)
    x, dz = torch.empty((0, 33), dtype=BF, device=DEV), torch.empty((0, 24), dtype=BF, device=DEV)
    z, pre = gk.grkan_linear_act_forward(x, W, bias, "rational", A, B, 8, keep=True)
    assert z.shape == (0, 24) and pre.shape == (0, 24)
    dx, *rest = gk.grkan_linear_act_backward(x, W, dz, pre, "rational", A, B, 8)
    assert dx.shape == (0, 33)
    for t in rest:
        assert float(t.float().abs().max()) == 0.0


def test_another_stream(gk):
    x, W, bias, r, dz, pre, A, B = make((70, 4096, 64, 8), "rational", 38)
    z, h = gk.grkan_linear_act_forward(x, W, bias, "rational", A, B, 8, residual=r, keep=True)
    d = gk.grkan_linear_act_backward(x, W, dz, pre, "rational", A, B, 8)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    z1, h1 = gk.grkan_linear_act_forward(x, W, bias, "rational", A, B, 8, residual=r, keep=True, stream=st)
    d1 = gk.grkan_linear_act_backward(x, W, dz, pre, "rational", A, B, 8, stream=st)
    st.synchronize()
    assert torch.equal(z, z1) and torch.equal(h, h1) and all(torch.equal(p, q) for p, q in zip(d, d1))


def test_offsets_past_32_bits(gk):
    """More than 2^31 elements of z, and of x: the last rows have the values of a product of their own."""
    gen = torch.Generator().manual_seed(39)
    tail = torch.randn((256, 64), generator=gen).to(BF).to(DEV)
    W = (torch.randn((4096, 64), generator=gen) / 8).to(BF).to(DEV)
    rows = (1 << 31) // 4096 + 300
    x = torch.zeros((rows, 64), dtype=BF, device=DEV)
    x[-256:] = tail
    z, _ = gk.grkan_linear_act_forward(x, W)
    want = ref.linear_forward(tail, W, None, "none")["z"]
    ref.check("z", z[-256:], *want)
    assert float(z[:1000].abs().max()) == 0.0
    W2 = W.t().contiguous()  # [64, 4096]
    z2, _ = gk.grkan_linear_act_forward(z, W2)
    ref.check("z2", z2[-256:], *ref.linear_forward(z[-256:], W2, None, "none")["z"])
    dx, dW = gk.grkan_linear_act_backward(x, W, z)[:2]
    want = ref.linear_backward(tail, W, z[-256:], None, "none")
    ref.check("dx", dx[-256:], *want["dx"])
    ref.check("dW", dW, *want["dW"])


def test_autograd(gk):
    x, W, bias, r, dz, _, A, B = make((100, 96, 80, 8), "rational", 40)
    leaves = [t.clone().requires_grad_() for t in (x, W, bias, A, B, r)]
    z = gk.GRKANLinearAct.apply(leaves[0], leaves[1], leaves[2], "rational", leaves[3], leaves[4], 8, leaves[5])
    z.backward(dz)
    _, pre = gk.grkan_linear_act_forward(x, W, bias, "rational", A, B, 8, keep=True)
    dx, dW, db, dA, dB = gk.grkan_linear_act_backward(x, W, dz, pre, "rational", A, B, 8)
    for leaf, g in zip(leaves, (dx, dW, db, dA, dB, dz)):
        assert torch.equal(leaf.grad, g)
