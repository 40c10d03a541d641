"""CPU checks of the block operators' autograd functions: what they ask of the operators, which a recorder
stands in for here."""
import pytest
import torch

from gr_kan_rational_amd import block

BF = torch.bfloat16


@pytest.fixture
def linear(monkeypatch):
    """Calls of the linear map, as dicts; its values by torch."""
    calls = []

    def forward(x, W, bias=None, act="none", A=None, B=None, n_groups=8, residual=None, keep=False):
        calls.append({"way": "forward", "keep": keep})
        pre = torch.nn.functional.linear(x, W)
        z = pre if residual is None else pre + residual
        return z.clone(), pre.clone() if keep else None

    def backward(x, W, dz, pre=None, act="none", A=None, B=None, n_groups=8, **kw):
        assert act == "none" or pre is not None
        calls.append({"way": "backward", **kw})
        skip = kw.get("skip", ())
        out = [t if n not in skip else None for n, t in (("dx", dz @ W), ("dW", dz.t() @ x), ("dbias", dz.float().sum(0)))]
        return (*out, torch.zeros_like(A), torch.zeros_like(B)) if act == "rational" else (*out, None, None)

    monkeypatch.setattr(block, "grkan_linear_act_forward", forward)
    monkeypatch.setattr(block, "grkan_linear_act_backward", backward)
    return calls


def linear_inputs(**grads):
    shapes = {"x": (5, 16), "W": (24, 16), "bias": (24,), "A": (8, 6), "B": (8, 4), "residual": (5, 24)}
    out = {}
    for k, s in shapes.items():
        t = torch.randn(s, generator=torch.Generator().manual_seed(len(out)))
        out[k] = (t if k in ("bias", "A", "B") else t.to(BF)).requires_grad_(grads.get(k, False))
    return out


def apply(t, act):
    rational = act == "rational"
    return block.GRKANLinearAct.apply(t["x"], t["W"], t["bias"], act, t["A"] if rational else None,
                                      t["B"] if rational else None, 8, t["residual"])


@pytest.mark.parametrize("act", ("silu", "rational", "none"))
@pytest.mark.parametrize("needs", ("x", "W", "bias", "A"))
def test_the_product_is_kept_for_a_backward_that_reads_it(linear, act, needs):
    t = linear_inputs(**{needs: True})
    apply(t, act)
    asked = act != "none" and (needs != "A" or act == "rational")
    assert linear[-1]["keep"] is asked


@pytest.mark.parametrize("act", ("silu", "rational", "none"))
def test_the_product_is_not_kept_without_gradients(linear, act):
    t = linear_inputs(x=True, W=True, bias=True, A=True, B=True, residual=True)
    with torch.no_grad():
        z = apply(t, act)
    assert linear == [{"way": "forward", "keep": False}] and not z.requires_grad
    t = linear_inputs()
    z = apply(t, act)
    assert linear[-1]["keep"] is False and not z.requires_grad


@pytest.mark.parametrize("act", ("silu", "none"))
def test_the_residuals_gradient_alone(linear, act):
    t = linear_inputs(residual=True)
    z = apply(t, act)
    assert linear[-1]["keep"] is False
    dz = torch.randn(z.shape).to(BF)
    z.backward(dz)
    assert torch.equal(t["residual"].grad, dz) and len(linear) == 1


@pytest.mark.parametrize("act", ("silu", "rational", "none"))
@pytest.mark.parametrize("needs", ("x", "W", "bias"))
def test_the_linear_backward_forms_what_is_asked_for(linear, act, needs):
    t = linear_inputs(**{needs: True})
    apply(t, act).float().sum().backward()
    grad = {"x": "dx", "W": "dW", "bias": "dbias"}
    assert sorted(linear[-1]["skip"]) == sorted(grad[k] for k in grad if k != needs)
    assert t[needs].grad is not None


def test_a_missing_bias_has_no_gradient(linear):
    t = linear_inputs(x=True, W=True)
    t["bias"] = None
    apply(t, "silu").float().sum().backward()
    assert linear[-1]["skip"] == ["dbias"]


@pytest.mark.parametrize("needs, skip", [(("x",), ["dweight", "dbias"]), (("x", "w"), ["dbias"]), (("b",), ["dweight"]),
                                         (("x", "w", "b"), [])])
def test_the_norms_backward_forms_what_is_asked_for(monkeypatch, needs, skip):
    calls = []
    monkeypatch.setattr(block, "grkan_group_norm_forward",
                        lambda x, g, *a: (x.clone(), torch.zeros(x.shape[0], g), torch.ones(x.shape[0], g)))

    def backward(x, dy, *a, skip=()):
        calls.append(skip)
        c = x.shape[-1]
        return (dy.clone(), *(None if n in skip else torch.ones(c) for n in ("dweight", "dbias")), None, None)

    monkeypatch.setattr(block, "grkan_group_norm_backward", backward)
    t = {"x": torch.randn(4, 32), "w": torch.ones(32), "b": torch.zeros(32)}
    for k in needs:
        t[k].requires_grad_()
    block.GRKANGroupNorm.apply(t["x"], 4, t["w"], t["b"]).sum().backward()
    assert calls == [skip]
    assert all((t[k].grad is not None) == (k in needs) for k in t)


def test_skip_names_and_outputs_are_checked():
    with pytest.raises(ValueError, match="skip"):
        block._skipped(("dA",), ("dx", "dW", "dbias"))
    with pytest.raises(ValueError, match="given and skipped"):
        block._wanted(("dx",), "dx", torch.zeros(3), (3,), torch.float32, torch.device("cpu"))
    assert block._wanted(["dx"], "dx", None, (3,), torch.float32, torch.device("cpu")) is None


def test_the_norms_arguments_may_be_left_out(monkeypatch):
    monkeypatch.setattr(block, "grkan_group_norm_forward",
                        lambda x, g, *a: (x.clone(), torch.zeros(x.shape[0], g), torch.ones(x.shape[0], g)))
    monkeypatch.setattr(block, "grkan_group_norm_backward",
                        lambda x, dy, *a, skip=(): (dy.clone(), *(None if n in skip else torch.ones(32)
                                                                  for n in ("dweight", "dbias")), None, None))
    x, w = torch.randn(4, 32, requires_grad=True), torch.ones(32, requires_grad=True)
    block.GRKANGroupNorm.apply(x, 4).sum().backward()
    block.GRKANGroupNorm.apply(x, 4, w).sum().backward()
    assert x.grad is not None and w.grad is not None


def test_a_second_derivative_is_refused(linear, monkeypatch):
    """The backward's results have no graph of their own: differentiating them raises, where it would leave
    their part of the second derivative out."""
    t = linear_inputs(x=True, W=True)
    z = apply(t, "silu").float()
    gx, = torch.autograd.grad((z ** 2).sum(), t["x"], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (gx.float() ** 2).sum().backward()
    monkeypatch.setattr(block, "grkan_group_norm_forward",
                        lambda x, g, *a: (x.clone(), torch.zeros(x.shape[0], g), torch.ones(x.shape[0], g)))
    monkeypatch.setattr(block, "grkan_group_norm_backward",
                        lambda x, dy, *a, skip=(): (dy.clone(), None, None, None, None))
    x = torch.randn(4, 32, requires_grad=True)
    gx, = torch.autograd.grad((block.GRKANGroupNorm.apply(x, 4) ** 2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (gx ** 2).sum().backward()
