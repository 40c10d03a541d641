"""GPU tests of the channel mixer: the block operators together, against the same block in fp64, and the
example's training loop."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = torch.device("cuda:0")


def rational(h, A, B):
    g = A.shape[0]
    v = h.reshape(-1, g, h.shape[-1] // g)
    P = sum(A[:, i].view(1, g, 1) * v ** i for i in range(6))
    Q = sum(B[:, j].view(1, g, 1) * v ** (j + 1) for j in range(4))
    return (P / (1 + Q.abs())).reshape(h.shape)


def reference(m, x):
    """The mixer in fp64 autograd, its parameters as leaves."""
    p = {k: v.detach().double().requires_grad_() for k, v in m.named_parameters()}
    xd = x.detach().double().requires_grad_()
    g, c = m.norm_groups or 1, x.shape[-1]
    v = xd.reshape(x.shape[0], -1, g, c // g) if m.norm_groups else xd.reshape(-1, 1, g, c // g)
    mean = v.mean((1, 3), keepdim=True)
    var = (v - mean).square().mean((1, 3), keepdim=True)
    h = ((v - mean) / torch.sqrt(var + 1e-5)).reshape(x.shape) * p["norm_weight"] + p["norm_bias"]
    h = rational(h, p["A1"], p["B1"]) @ p["W1"].t() + p["b1"]
    return xd + rational(h, p["A2"], p["B2"]) @ p["W2"].t() + p["b2"], xd, p


@pytest.mark.parametrize("norm_groups, shape", [(0, (3, 50, 96)), (0, (1, 96)), (4, (3, 50, 96))])
def test_mixer_against_fp64(norm_groups, shape):
    """Values and every gradient within 2% in norm: three bf16 tensors lie between input and output, five
    on the way back, each within 2^-8 of its values, and the gradients add them up in quadrature."""
    from gr_kan_rational_amd.mixer import GRKANMixer

    torch.manual_seed(1)
    m = GRKANMixer(96, 256, norm_groups=norm_groups, device=DEV)
    with torch.no_grad():  # away from the identity and the even denominators' zeros
        for k, v in m.named_parameters():
            if v.dtype == torch.float32:
                v += 0.05 * torch.rand_like(v)
    x = torch.randn(shape, device=DEV).to(torch.bfloat16).requires_grad_()
    dy = torch.randn(shape, device=DEV).to(torch.bfloat16)
    y = m(x)
    y.backward(dy)
    want, xd, p = reference(m, x)
    want.backward(dy.double())

    def close(what, got, ref):
        got, ref = got.detach().double(), ref.detach()
        assert float((got - ref).norm()) <= 0.02 * float(ref.norm()), what

    close("y", y, want)
    close("dx", x.grad, xd.grad)
    for k, v in m.named_parameters():
        close(k, v.grad, p[k].grad)


def test_training_example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    from train_mixer import train

    losses = train(steps=40, tokens=1024, dim=64, hidden=128, quiet=True)
    assert losses[-1] < 0.5 * losses[0]
