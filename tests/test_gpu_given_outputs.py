"""GPU tests that a call which writes into tensors that it was given is noticed as a modification in place."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


def bf(*shape):
    return torch.ones(shape, dtype=BF, device=DEV)


def f32(*shape):
    return torch.ones(shape, device=DEV)


def calls(gk):
    """(name, names of the outputs, shapes and types for them, call of them)."""
    from gr_kan_rational_amd import binding as b

    x, W, A, B = bf(20, 64), bf(64, 64), f32(8, 6), f32(8, 4)
    mean, rstd, stats, C = f32(20, 1), f32(20, 1), f32(2, 20), bf(64, 64, 8)
    q, s = gk.grkan_fp8_quantize(x)
    wq, ws = gk.grkan_fp8_quantize(W, tile=True)
    grads = dict(dx=bf(20, 64), dA=f32(8, 6), dB=f32(8, 4))
    return [
        ("forward", dict(out=bf(20, 64)), lambda **k: gk.grkan_forward(x, A, B, **k)),
        ("backward", grads, lambda **k: gk.grkan_backward(x, x, A, B, **k)),
        ("noalloc", grads, lambda **k: b.grkan_backward_noalloc(x, x, A, B, **k)),
        ("probe", dict(out=bf(20, 64)), lambda **k: b.grkan_stream_probe(x, x, **k)),
        ("layer", dict(out=bf(20, 64)), lambda **k: b.grkan_layer_forward(x, A, B, W, **k)),
        ("layer_ws", dict(out=bf(20, 64)), lambda **k: b.grkan_layer_forward_ws(x, A, B, W, **k)),
        ("linear", dict(out=bf(20, 64)), lambda **k: b.grkan_linear_forward(x, W, **k)),
        ("layer_backward", dict(grads, dW=f32(64, 64)), lambda **k: b.grkan_layer_backward(x, bf(20, 64), A, B, W, **k)),
        ("chebykan", dict(out=bf(20, 64)), lambda **k: b.grkan_chebykan_forward(x, C, **k)),
        ("chebykan_backward", dict(dx=bf(20, 64), dC=f32(64, 64, 8)),
         lambda **k: b.grkan_chebykan_backward(x, bf(20, 64), C, **k)),
        ("group_norm", dict(out=bf(20, 64), mean=f32(20, 1), rstd=f32(20, 1)),
         lambda **k: gk.grkan_group_norm_forward(x, 1, **k)),
        ("group_norm_backward", dict(grads, dweight=f32(64), dbias=f32(64)),
         lambda **k: gk.grkan_group_norm_backward(x, x, mean, rstd, 1, act="rational", A=A, B=B, **k)),
        ("linear_act", dict(out=bf(20, 64), pre=bf(20, 64)),
         lambda **k: gk.grkan_linear_act_forward(x, W, act="rational", A=A, B=B, **k)),
        ("linear_act_backward", dict(grads, dW=bf(64, 64), dbias=f32(64)),
         lambda **k: gk.grkan_linear_act_backward(x, W, bf(20, 64), bf(20, 64), "rational", A, B, **k)),
        ("fp8_matmul", dict(out=bf(20, 64)), lambda **k: gk.grkan_fp8_matmul(q, s, wq, ws, **k)),
        ("residual", dict(out=bf(20, 64), normed=bf(20, 64), stats=f32(2, 20)),
         lambda **k: gk.grkan_residual_norm_forward(x, x, **k)),
        ("residual_backward", dict(dx=bf(20, 64), df=bf(20, 64)),
         lambda **k: gk.grkan_residual_norm_backward(x, x, x, None, stats, **k)),
    ]


NAMES = ["forward", "backward", "noalloc", "probe", "layer", "layer_ws", "linear", "layer_backward", "chebykan",
         "chebykan_backward", "group_norm", "group_norm_backward", "linear_act", "linear_act_backward", "fp8_matmul",
         "residual", "residual_backward"]


@pytest.mark.parametrize("at", range(len(NAMES)), ids=NAMES)
def test_given_outputs_count_as_modified(gk, at):
    name, outputs, call = calls(gk)[at]
    assert name == NAMES[at]
    before = {k: t._version for k, t in outputs.items()}
    call(**outputs)
    assert {k: t._version for k, t in outputs.items()} == {k: v + 1 for k, v in before.items()}


def test_a_backward_notices(gk):
    """h = x + f written over x, which a product before it has kept."""
    x, W = bf(20, 64), torch.nn.Parameter(bf(64, 64))
    y = gk.GRKANLinearAct.apply(x, W)
    gk.grkan_residual_norm_forward(x, torch.ones_like(x), out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
