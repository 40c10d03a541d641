"""GPU tests of the 8-bit product's two kinds of sums, of their bounds and of the calls that choose."""
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


@pytest.mark.parametrize("shape", [(3, 40, 256), (100, 130, 200), (700, 400, 520), (130, 80, 12000)], ids=str)
def test_sums_that_cancel(gk, shape):
    """Large products cancel in every 8 values of k; what is left is 2^-14 of them.  fp32 sums have it exactly (every
    partial sum is a multiple of 2^-6 below 2^18); cut sums lose it, within their bound."""
    m, n, k = shape
    a, b = torch.zeros((m, k), device=DEV), torch.zeros((n, k), device=DEV)
    a[:, 0::8], a[:, 1::8], a[:, 2::8] = 256.0, 256.0, 0.125
    b[:, 0::8], b[:, 1::8], b[:, 2::8] = 128.0, -128.0, 0.125
    held = ref.ceil(k, 16) * 16
    q = [torch.zeros((t.shape[0], held), device=DEV).to(F8) for t in (a, b)]
    for c, t in zip(q, (a, b)):
        c.view(torch.uint8)[:, :k] = t.to(F8).view(torch.uint8)
    q = [c[:, :k] for c in q]
    s = [torch.ones((t.shape[0], ref.ceil(k, 128)), device=DEV) for t in (a, b)]
    want = torch.full((m, n), 2.0 ** -6 * ((k + 5) // 8), device=DEV)
    for dtype in (BF, torch.float32):
        assert torch.equal(gk.grkan_fp8_matmul(q[0], s[0], q[1], s[1], dtype=dtype), want.to(dtype))
    assert torch.equal(gk.grkan_fp8_matmul(q[0], s[0], q[1], s[1], dtype=torch.float32, sums="fast"), want)
    cut = gk.grkan_fp8_matmul(q[0], s[0], q[1], s[1], sums="fast")
    ref.check("cut", cut, *ref.matmul(q[0], s[0], q[1], s[1], False))


def test_linear_with_either_sums(gk):
    """The layer's three products take the kind of sums: each result is that of the products by themselves."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn((70, 200), generator=gen, device=DEV).to(BF).requires_grad_()
    W = (torch.randn((90, 200), generator=gen, device=DEV) * 0.1).to(BF).requires_grad_()
    dy = torch.randn((70, 90), generator=gen, device=DEV).to(BF)
    for sums in ("fp32", "fast", None):
        y = gk.GRKANFp8Linear.apply(x, W, *((None, "none", None, None, 8, sums) if sums else ()))
        sums = sums or "fp32"
        dx, dW = torch.autograd.grad(y, (x, W), dy)
        q, s, qt, st = gk.grkan_fp8_quantize(x.detach(), "both")
        wq, ws, wt, wst = gk.grkan_fp8_quantize(W.detach(), "both", tile=True)
        g, gs, gt, gst = gk.grkan_fp8_quantize(dy, "both")
        assert torch.equal(y, gk.grkan_fp8_matmul(q, s, wq, ws, sums=sums))
        assert torch.equal(dx, gk.grkan_fp8_matmul(g, gs, wt, wst, sums=sums))
        assert torch.equal(dW, gk.grkan_fp8_matmul(gt, gst, qt, st, sums=sums))


def test_stack_with_either_sums(gk):
    from gr_kan_rational_amd.mixer import GRKANStack

    torch.manual_seed(3)
    one = GRKANStack(2, 64, 128, products="fp8", sums="fast", device=DEV)
    two = GRKANStack(2, 64, 128, products="fp8", device=DEV)
    two.load_state_dict(one.state_dict())
    x = torch.randn((3, 20, 64), device=DEV).to(BF)
    a, b = one(x).detach().double(), two(x).detach().double()
    # one product's cut sums are 5e-5 of its norm off; requantised and rounded to bf16 a value may move by a step of e4m3
    assert 0 < float((a - b).norm()) <= 2.0 ** -4 * float(b.norm())
