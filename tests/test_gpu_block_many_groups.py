"""GPU tests of the block operators at sizes for which one workgroup an output would pass the 2^32 threads of a
launch."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
GROUPS = 430_000  # 10 coefficients each, in workgroups of 1,024 threads: 4.4e9


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


def coefficients(gen):
    A = torch.randn((GROUPS, 6), generator=gen, device=DEV) * 0.5
    B = torch.randn((GROUPS, 4), generator=gen, device=DEV) * 0.5
    return A, B


@pytest.mark.parametrize("norm_groups", (1, GROUPS // 10))
def test_one_rational_per_channel_behind_a_norm(gk, norm_groups):
    print(f"[group norm] 2 x {GROUPS} in {norm_groups}, one rational a channel", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(90)
    x, dy = (torch.randn((2, GROUPS), generator=gen, device=DEV) for _ in range(2))
    A, B = coefficients(gen)
    y, mean, rstd = gk.grkan_group_norm_forward(x, norm_groups, act="rational", A=A, B=B, n_groups=GROUPS)
    one = torch.ones(GROUPS, device=DEV)
    want = ref.norm_forward(x, norm_groups, one, 0 * one, 1e-5, "rational", A, B)
    ref.check("y", y, *want["y"])
    got = gk.grkan_group_norm_backward(x, dy, mean, rstd, norm_groups, None, None, "rational", A, B, GROUPS)
    h = ((x.double().view(2, norm_groups, -1) - mean.double()[..., None]) * rstd.double()[..., None]).view(2, -1)
    check_coefficients(h, dy, A, B, got[3], got[4], 64)


def check_coefficients(h, dy, A, B, dA, dB, ulps):
    """One or a few terms a sum: each within `ulps` units of its terms' magnitudes, where Q is not within that of
    zero (its sign, and with it dB, is then that of the fp32 h's Q)."""
    h, g, A, B = h.double(), dy.double(), A.double(), B.double()
    P, mP = (sum(f(A[:, i] * h ** i) for i in range(6)) for f in (torch.clone, torch.abs))
    Q, mQ = (sum(f(B[:, j - 1] * h ** j) for j in range(1, 5)) for f in (torch.clone, torch.abs))
    D, s = 1 + Q.abs(), torch.sign(Q)
    u = ulps * 2.0 ** -24
    sure = (Q.abs() > u * mQ).all(0)
    assert float(sure.double().mean()) > 0.99
    for k in range(10):
        if k < 6:
            t, m = g * h ** k / D, g.abs() * h.abs() ** k / D * (1 + mQ / D)
        else:
            t = -g * s * P * h ** (k - 5) / D ** 2
            m = g.abs() * h.abs() ** (k - 5) / D ** 2 * (mP + 2 * P.abs() * mQ / D)
        got = dA[:, k] if k < 6 else dB[:, k - 6]
        bound = u * m.sum(0) + 1e-30
        ref.check(f"coefficient {k}", got[sure], t.sum(0)[sure], bound[sure])


def test_one_rational_per_column_of_a_linear_map(gk):
    print(f"[linear backward] 3 x 8 -> {GROUPS}, one rational a column", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(91)
    x, W = (torch.randn(s, generator=gen, device=DEV).to(BF) for s in ((3, 8), (GROUPS, 8)))
    dz, pre = (torch.randn((3, GROUPS), generator=gen, device=DEV).to(BF) for _ in range(2))
    A, B = coefficients(gen)
    _, _, _, dA, dB = gk.grkan_linear_act_backward(x, W, dz, pre, "rational", A, B, GROUPS)
    check_coefficients(pre, dz, A, B, dA, dB, 64)


def test_no_rows_of_a_large_weight(gk):
    """dW of 2^32 elements without rows: zeros throughout."""
    d = 1 << 16
    print(f"[linear backward] 0 x {d} -> {d}", flush=True)
    W = torch.empty((d, d), dtype=BF, device=DEV)
    dW = torch.full((d, d), 7.0, dtype=BF, device=DEV)
    x, dz = (torch.empty((0, d), dtype=BF, device=DEV) for _ in range(2))
    gk.grkan_linear_act_backward(x, W, dz, dW=dW)
    assert not bool(dW.view(torch.int16).any())
