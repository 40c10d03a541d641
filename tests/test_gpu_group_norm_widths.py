"""GPU tests of the group norm at channel counts whose groups end inside accesses of nearly as many columns as
a workgroup takes: their sums need the most LDS."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


@pytest.mark.parametrize("n, s, c, g", [(2, 1024, 2044, 4), (64, 197, 2046, 1), (2, 197, 2047, 1), (8, 512, 4080, 16),
                                        (8, 512, 4080, 40), (8, 512, 6080, 64), (4, 512, 6112, 32),
                                        (16, 1024, 4094, 2), (8, 1300, 1995, 57)])
def test_forward_and_backward(gk, n, s, c, g):
    print(f"[group norm] {n} x {s} x {c} in {g}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(80 + c + g)
    x = (torch.randn((n, s, c), generator=gen, device=DEV) * 1.5 + 0.3).bfloat16()
    dy = (torch.randn((n, s, c), generator=gen, device=DEV) * 0.1).bfloat16()
    w = 1 + 0.2 * torch.randn(c, generator=gen, device=DEV)
    b = 0.2 * torch.randn(c, generator=gen, device=DEV)
    y, mean, rstd = gk.grkan_group_norm_forward(x, g, w, b, act="silu")
    want = ref.norm_forward(x, g, w, b, 1e-5, "silu")
    for k, got in (("mean", mean), ("rstd", rstd), ("y", y)):
        ref.check(k, got, *want[k])
    got = gk.grkan_group_norm_backward(x, dy, mean, rstd, g, w, b, "silu")
    want = ref.norm_backward(x, dy, mean, rstd, g, w, b, "silu")
    for k, t in zip(("dx", "dweight", "dbias"), got):
        ref.check(k, t, *want[k])
