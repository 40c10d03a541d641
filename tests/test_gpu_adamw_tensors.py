"""GPU tests of what the AdamW step and its optimizer do with a program's tensors."""
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


@pytest.mark.parametrize("bits", (32, 8))
def test_a_step_between_forward_and_backward_is_noticed(gk, bits):
    """As torch's own optimizers: the backward of a forward from before the step raises, one from after it works; the
    states count as modified too."""
    x = torch.ones((5, 64), device=DEV, dtype=BF, requires_grad=True)
    W = torch.nn.Parameter(torch.full((32, 64), 0.5, device=DEV, dtype=BF))
    opt = gk.GRKANAdamW([W], lr=0.1, bits=bits)
    gk.GRKANLinearAct.apply(x, W).sum().backward()
    late = gk.GRKANLinearAct.apply(x, W).sum()
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        late.backward()
    gk.GRKANLinearAct.apply(x, W).sum().backward()
    before = {k: v._version for k, v in opt.state[W].items() if isinstance(v, torch.Tensor)}
    assert set(before) == {"avg", "sq", "master", *(("avg_scale", "sq_scale") if bits == 8 else ())}
    version = W._version
    opt.step()
    assert W._version == version + 1 and all(opt.state[W][k]._version == v + 1 for k, v in before.items())
