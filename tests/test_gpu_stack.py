"""GPU tests of the deep stack: the operators of a training step together, against the same stack in fp64, with
products in both types, and the example."""
import os
import sys

import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = torch.device("cuda:0")
BF = torch.bfloat16


def rational(h, A, B):
    g = A.shape[0]
    v = h.reshape(-1, g, h.shape[-1] // g)
    P = sum(A[:, i].view(1, g, 1) * v ** i for i in range(6))
    Q = sum(B[:, j].view(1, g, 1) * v ** (j + 1) for j in range(4))
    return (P / (1 + Q.abs())).reshape(h.shape)


def norm(v, kind, w=None, b=None):
    mean = v.mean(-1, keepdim=True) if kind == "layer" else 0.0
    y = (v - mean) * ((v - mean).square().mean(-1, keepdim=True) + 1e-5) ** -0.5
    y = y if w is None else y * w
    return y if b is None else y + b


def reference(stack, x, gates):
    """(z, x and the parameters as fp64 leaves)."""
    p = {k: v.detach().double().requires_grad_() for k, v in stack.named_parameters()}
    xd = x.detach().double().requires_grad_()
    h, depth = xd, len(stack.blocks)
    z = norm(h, "layer", p["blocks.0.norm_weight"], p["blocks.0.norm_bias"])
    for i in range(depth):
        m = {k: p[f"blocks.{i}.{k}"] for k in stack.blocks[i].keys()}
        f = rational(rational(z, m["A1"], m["B1"]) @ m["W1"].t() + m["b1"], m["A2"], m["B2"]) @ m["W2"].t() + m["b2"]
        if stack.post != "none":
            f = norm(f, stack.post, m["post_weight"], m.get("post_bias"))
        gate = 1.0 if gates[i] is None else gates[i].double()
        h = h + m["scale"] * gate * f
        after = f"blocks.{i + 1}." if i + 1 < depth else ""
        z = norm(h, "layer", p[after + "norm_weight"], p[after + "norm_bias"])
    return z, xd, p


def make(products, post, drop=0.0):
    from gr_kan_rational_amd.mixer import GRKANStack

    torch.manual_seed(3)
    s = GRKANStack(3, 96, 256, products=products, post=post, scale=0.5, drop=drop, device=DEV)
    with torch.no_grad():  # away from the identity and the even denominators' zeros
        for v in s.parameters():
            if v.dtype == torch.float32:
                v += 0.05 * torch.rand_like(v)
    return s, torch.randn(4, 30, 96, device=DEV).to(BF), torch.randn(4, 30, 96, device=DEV).to(BF)


# What each product adds to a branch in norm.  bf16: five tensors rounded to 2^-8 of their values at most lie on
# the way forward and twice as many on the way back, adding in quadrature: 2%, as for one mixer.  8 bits: an
# operand's values are off by 2^-4 at most, 2^-4 / sqrt 3 in the mean (3.6%), two operands a product 5.1%, two
# products in a row 7.2%; the gradients pass four more and, through F', the values of both: 15%; three mixers in a
# row add theirs in quadrature, a factor sqrt 3.
BOUNDS = {"bf16": (0.02, 0.04), "fp8": (0.072 * 3 ** 0.5, 0.15 * 3 ** 0.5)}


@pytest.mark.parametrize("post", ("none", "layer", "rms"))
@pytest.mark.parametrize("products", ("bf16", "fp8"))
def test_stack_against_fp64(products, post):
    s, x, dy = make(products, post)
    x.requires_grad_()
    y = s(x)
    y.backward(dy)
    want, xd, p = reference(s, x, [None] * 3)
    want.backward(dy.double())
    forward, backward = BOUNDS[products]

    def close(what, got, ref, tol):
        err = float((got.detach().double() - ref.detach()).norm()) / float(ref.detach().norm())
        assert err <= tol, f"{what}: {err}"

    close("z", y, want, forward)
    close("dx", x.grad, xd.grad, backward)
    for k, v in s.named_parameters():
        # (the denominators' gradients are sums that nearly cancel)
        if not k.endswith(("B1", "B2")):
            close(k, v.grad, p[k].grad, backward)


def test_stochastic_depth():
    """A sample whose branches are all left out passes as it is; the others' gates are 1 / (1 - rate)."""
    s, x, _ = make("bf16", "none", drop=0.5)
    gates = [torch.tensor([0.0, 1.0, 2.0, 0.0], device=DEV).view(4, 1, 1)] * 3
    s.gates = lambda x: gates
    y = s(x)
    want, _, _ = reference(s, x, gates)
    want = want.detach()
    assert float((y.detach().double() - want).norm()) <= 0.02 * float(want.norm())
    plain = norm(x.double(), "layer", s.norm_weight.double(), s.norm_bias.double())
    for i in (0, 3):
        assert float((y[i].detach().double() - plain[i].detach()).norm()) <= 2 ** -7 * float(plain[i].detach().norm())
    del s.gates
    torch.manual_seed(5)
    got = torch.stack(s.train().gates(torch.zeros(20000, 1, 1, device=DEV))).view(3, -1)
    for k, rate in enumerate((0.0, 0.25, 0.5)):
        kept = got[k] > 0
        assert torch.allclose(got[k][kept], torch.tensor(1 / (1 - rate), device=DEV))
        assert abs(float(kept.double().mean()) - (1 - rate)) <= 5 * (rate * (1 - rate) / 20000) ** 0.5 + 1e-12
    assert s.eval().gates(x) == [None] * 3


def test_no_mixer():
    from gr_kan_rational_amd.mixer import GRKANStack

    s = GRKANStack(0, 64, 64, device=DEV)
    x = torch.randn(5, 64, device=DEV).to(BF)
    assert torch.allclose(s(x).float(), norm(x.float(), "layer"), atol=2 ** -7, rtol=2 ** -7)


def test_a_captured_step():
    """Forward, backward and the optimizer's step captured once: each replay does what the eager step does."""
    import gr_kan_rational_amd as gk

    def build():
        s, x, dy = make("fp8", "rms")
        params = list(s.parameters())
        states = [gk.grkan_adamw_state(p, 8) for p in params]
        masters = [p.detach().float() if p.dtype == BF else None for p in params]
        return s, x, dy, params, states, masters

    def step(s, x, dy, params, states, masters, count):
        grads = torch.autograd.grad(s(x), params, dy)
        with torch.no_grad():
            gk.grkan_adamw_step([p.detach() for p in params], [g.contiguous() for g in grads], [t[0] for t in states],
                                [t[1] for t in states], step=count, lr=1e-2, masters=masters,
                                avg_scales=[t[2] for t in states], sq_scales=[t[3] for t in states], seed=9)

    eager, captured = build(), build()
    counts = [torch.tensor([1], device=DEV) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # (as a capture wants it, once outside)
        step(*captured, counts[1])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*captured, counts[1])
    step(*eager, counts[0])
    for k in range(2, 5):
        for c in counts:
            c.fill_(k)
        x = torch.randn(4, 30, 96, device=DEV).to(BF)
        eager[1].copy_(x), captured[1].copy_(x)
        step(*eager, counts[0])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager[3], captured[3]):
            assert torch.equal(a, b)


@pytest.mark.parametrize("products, bits", (("fp8", 8), ("bf16", 32)))
def test_training_example(products, bits):
    """Runs to its end with finite losses."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    from train_stack import train

    losses = train(steps=5, samples=8, positions=16, depth=2, dim=64, hidden=128, products=products, bits=bits, quiet=True)
    assert len(losses) == 5 and all(0.0 < v < 1e3 for v in losses)
