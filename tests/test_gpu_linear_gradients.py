"""GPU tests of the linear map's backward where its arithmetic or its dispatch can go wrong: the rational's
coefficient gradients next to the roots of its denominator's polynomial."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


def near_root(h0, scale):
    """fp32 (A, B) whose Q has terms of about `scale` at h0 and is itself about 0.3 there, and whose P has
    terms of one sign at h0."""
    s = 1.0 if h0 > 0 else -1.0
    a = torch.tensor([0.3 * s ** i / abs(h0) ** i for i in range(6)], dtype=torch.float64)
    b = torch.tensor([0.0, -1.25 * scale / h0 ** 2, 0.5 * scale / h0 ** 3, scale / h0 ** 4], dtype=torch.float64)
    a, b = a.float(), b.float()
    rest = sum(float(b[j]) * h0 ** (j + 1) for j in range(1, 4))
    b[0] = (0.3 - rest) / h0  # rounded to fp32: Q moves by up to 2^-24 of its terms, and is taken as it is
    return a, b


@pytest.mark.parametrize("d_out, groups", [(64, 2), (36, 6)], ids=("whole-chunks", "narrow-groups"))
@pytest.mark.parametrize("scale", (1e3, 3e4))
@pytest.mark.parametrize("h0", (3.0, -2.5, 1.4140625, 0.71875))
def test_coefficient_gradients_next_to_a_root_of_q(gk, h0, scale, d_out, groups):
    """Every pre of a group is the same bf16 value, so each sum is one term times the sum of dz and its
    relative error that of the term.  P's terms have one sign (12 u with the powers), Q is rounded once from
    fp64 (1 u of |Q| < D), D, its reciprocal and the products of a term cost 12 u more, and equal addends of
    one sign 64 u: under 100 u = 6e-6 of the value; 1e-5 is asked for.  (Q in fp32 would be off by a
    unit of its terms, 2^-24 scale, which moves D of about 1.3 by up to 1e-4 and 3e-3.)"""
    rows, d_in = 64, 16
    A, B = near_root(h0, scale)
    g = torch.arange(groups, dtype=torch.float32)[:, None]
    A = A[None] * (1.0 + 0.25 * g)  # another scale of P in each group, the terms' signs kept
    B = B[None].repeat(groups, 1)
    pre = torch.full((rows, d_out), h0, dtype=BF)
    assert float(pre[0, 0]) == h0
    dz = (0.5 + torch.rand((rows, d_out), generator=torch.Generator().manual_seed(5))).to(BF)
    x, W = torch.zeros((rows, d_in), dtype=BF), torch.zeros((d_out, d_in), dtype=BF)
    _, _, _, dA, dB = gk.grkan_linear_act_backward(*(t.to(DEV) for t in (x, W, dz, pre)), "rational", A.to(DEV),
                                                   B.to(DEV), groups)
    P = sum(A.double()[:, i] * h0 ** i for i in range(6))
    Q = sum(B.double()[:, j - 1] * h0 ** j for j in range(1, 5))
    D, s = 1 + Q.abs(), torch.sign(Q)
    total = dz.double().reshape(rows, groups, -1).sum((0, 2))
    for i in range(6):
        want = total * h0 ** i / D
        ref.check(f"dA{i}", dA[:, i], want, 1e-5 * want.abs())
    for j in range(1, 5):
        want = -total * s * P * h0 ** j / D ** 2
        ref.check(f"dB{j}", dB[:, j - 1], want, 1e-5 * want.abs())


@pytest.mark.parametrize("seed", range(4))
def test_coefficient_gradients_at_full_size(gk, seed):
    """Coefficients whose Q has real roots among the values, 25,216 x 768 in 8 groups: the rule of the
    activation's own gradients, 1e-4 of the sum or of a hundredth of its terms' norm, 1e-6 besides."""
    rows, d_out, groups = 25216, 768, 8
    gen = torch.Generator(device=DEV).manual_seed(50 + seed)
    pre = torch.randn((rows, d_out), generator=gen, device=DEV).to(BF)
    dz = (torch.randn((rows, d_out), generator=gen, device=DEV) * 1e-2).to(BF)
    A, B = (torch.randn((groups, k), generator=gen, device=DEV) * 0.5 for k in (6, 4))
    x, W = torch.zeros((rows, 8), dtype=BF, device=DEV), torch.zeros((d_out, 8), dtype=BF, device=DEV)
    _, _, _, dA, dB = gk.grkan_linear_act_backward(x, W, dz, pre, "rational", A, B, groups)
    h, g = (t.double().reshape(rows, groups, -1) for t in (pre, dz))
    P = sum(A.double()[:, i, None] * h ** i for i in range(6))
    Q = sum(B.double()[:, j - 1, None] * h ** j for j in range(1, 5))
    D, s = 1 + Q.abs(), torch.sign(Q)
    for k in range(10):
        t = g * h ** k / D if k < 6 else -g * s * P * h ** (k - 5) / D ** 2
        want, norm = t.sum((0, 2)), t.square().sum((0, 2)).sqrt()
        got = dA[:, k] if k < 6 else dB[:, k - 6]
        ref.check(f"coefficient {k}", got, want, 1e-4 * torch.maximum(want.abs(), 1e-2 * norm) + 1e-6)


def inputs(rows, d_in, d_out, act, groups, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(size, std):
        return torch.randn(size, generator=gen, device=DEV) * std

    x, W = normal((rows, d_in), 1.0).to(BF), normal((d_out, d_in), d_in ** -0.5).to(BF)
    dz, pre = normal((rows, d_out), 0.1).to(BF), normal((rows, d_out), 1.2).to(BF)
    A, B = (normal((groups, 6), 0.5), normal((groups, 4), 0.5)) if act == "rational" else (None, None)
    return x, W, dz, pre, A, B


def check_backward(gk, x, W, dz, pre, act, A, B, groups):
    got = gk.grkan_linear_act_backward(x, W, dz, pre, act, A, B, groups)
    want = ref.linear_backward(x, W, dz, pre, act, A, B)
    for k, g in zip(("dx", "dW", "dbias", "dA", "dB"), got):
        if k in want:
            ref.check(k, g, *want[k])


# 256-row tiles, or whole rounds of them with the other rows in smaller tiles, where aligned operands would
# be; for the third of these dx alone
@pytest.mark.parametrize("shape, act, groups", [((8449, 1033, 2041), "silu", 1), ((8450, 2041, 1033), "silu", 1),
                                                ((5297, 3839, 407), "silu", 1), ((50432, 777, 1501), "rational", 19),
                                                ((50432, 770, 1500), "none", 1)], ids=str)
def test_unaligned_widths_of_large_products(gk, shape, act, groups):
    """Odd widths: no row but the first of an operand begins on a 16-byte boundary."""
    print(f"[linear backward, unaligned] {shape} {act}", flush=True)
    x, W, dz, pre, A, B = inputs(*shape, act, groups, 60)
    check_backward(gk, x, W, dz, pre, act, A, B, groups)


def off_boundary(t, left, right):
    """The values of t in the columns of a wider tensor of NaN, `left` elements off its rows' starts."""
    wide = torch.full((t.shape[0], left + t.shape[1] + right), float("nan"), dtype=t.dtype, device=DEV)
    view = wide[:, left:left + t.shape[1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("which", ("x", "W", "dz", "dz-stride"))
@pytest.mark.parametrize("shape", [(8449, 1032, 2040), (8450, 2040, 1032)], ids=str)
def test_unaligned_operands_of_aligned_widths(gk, shape, which):
    """One operand at an odd address or with an odd row stride, its neighbours in memory NaN."""
    print(f"[linear backward, unaligned {which}] {shape}", flush=True)
    rows, d_in, d_out = shape
    x, W, dz, _, _, _ = inputs(*shape, "none", 1, 61)
    if which == "W":
        buf = torch.full((d_out * d_in + 16,), float("nan"), dtype=BF, device=DEV)
        w2 = buf[7:7 + d_out * d_in].view(d_out, d_in)
        w2.copy_(W)
        W = w2
    elif which == "x":
        x = off_boundary(x, 3, 5)
    elif which == "dz":
        dz = off_boundary(dz, 1, 7)
    else:
        dz = off_boundary(dz, 0, 3)
    check_backward(gk, x, W, dz, None, "none", None, None, 1)


@pytest.mark.parametrize("act", ("none", "silu", "rational"))
def test_skipped_gradients(gk, act):
    """Each subset of dx, dW and dbias left out: None there, the other results unchanged."""
    x, W, dz, pre, A, B = inputs(300, 96, 80, act, 8, 62)
    names = ("dx", "dW", "dbias")
    full = gk.grkan_linear_act_backward(x, W, dz, pre, act, A, B, 8)
    for bits in range(1, 8):
        skip = [n for i, n in enumerate(names) if bits >> i & 1]
        got = gk.grkan_linear_act_backward(x, W, dz, pre, act, A, B, 8, skip=skip)
        for n, p, q in zip((*names, "dA", "dB"), full, got):
            assert q is None if n in skip else (p is q is None or torch.equal(p, q)), (skip, n)


@pytest.mark.parametrize("shape, groups", [((40, 1, 96), 1), ((3, 50, 96), 4), ((2, 3000, 64), 4)], ids=str)
@pytest.mark.parametrize("act", ("silu", "rational"))
def test_skipped_gradients_of_the_norm(gk, shape, groups, act):
    gen = torch.Generator(device=DEV).manual_seed(63)
    x, dy = (torch.randn(shape, generator=gen, device=DEV) for _ in range(2))
    A, B = (torch.randn((8, k), generator=gen, device=DEV) * 0.5 for k in (6, 4)) if act == "rational" else (None, None)
    _, mean, rstd = gk.grkan_group_norm_forward(x, groups, act=act, A=A, B=B)
    args = (x, dy, mean, rstd, groups, None, None, act, A, B, 8)
    full = gk.grkan_group_norm_backward(*args)
    for skip in (("dweight",), ("dbias",), ("dweight", "dbias")):
        got = gk.grkan_group_norm_backward(*args, skip=skip)
        for n, p, q in zip(("dx", "dweight", "dbias", "dA", "dB"), full, got):
            assert q is None if n in skip else (p is q is None or torch.equal(p, q)), (skip, n)
