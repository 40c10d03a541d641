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


@pytest.mark.parametrize("bits", (32, 8))
def test_a_parameter_written_between_steps_is_not_undone(gk, bits):
    """Loaded, clamped, set through .data, in some elements or all: what was written is stepped, the others go on from
    their masters' low bits; a model loaded beside its optimizer's state changes nothing."""
    def start():
        gen = torch.Generator().manual_seed(1)
        p = torch.nn.Parameter((torch.randn(40, 25, generator=gen) * 0.5).to(DEV).to(BF))
        p.grad = torch.randn(40, 25, generator=gen).to(DEV).to(BF)
        return p, gk.GRKANAdamW([p], lr=1e-3, weight_decay=0.0, bits=bits, seed=4)

    def clamp(p):
        p.clamp_(-0.4, 0.4)

    def data(p):
        p.data[3:5] = 2.0

    def load(p):
        p.copy_(torch.linspace(-1, 1, 1000, device=DEV).view(40, 25))

    def nan(p):
        p[7] = torch.nan

    for write in (clamp, data, load, nan):
        (p, opt), (q, same) = start(), start()
        for _ in range(3):
            opt.step()
            same.step()
        with torch.no_grad():
            write(p)
        changed = p != q
        assert changed.any()
        master = same.state[q]["master"]
        with torch.no_grad():   # what the step should start from
            master[changed] = p[changed].float()
            q.copy_(master.to(BF))
        opt.step()
        same.step()
        assert torch.equal(torch.nan_to_num(p, 9.0), torch.nan_to_num(q, 9.0))
        assert torch.equal(torch.nan_to_num(opt.state[p]["master"], 9.0), torch.nan_to_num(master, 9.0))
        still = ~changed
        assert write is load or (master[still] != q[still].float()).any()   # (low bits are there to lose)
    (p, opt), (q, same) = start(), start()
    opt.step()
    same.step()
    r, other = start()
    other.load_state_dict(opt.state_dict())
    with torch.no_grad():
        r.copy_(p)
    same.step()
    other.step()
    assert torch.equal(q, r) and torch.equal(same.state[q]["master"], other.state[r]["master"])


@pytest.mark.parametrize("bits", (32, 8))
def test_a_broken_master_is_replaced(gk, bits):
    """A parameter set anew where its master has become NaN or infinite: the parameter counts.  Odd sizes, unaligned."""
    for offset, n in ((0, 256), (1, 131)):
        w = torch.linspace(-1, 1, n, device=DEV)
        param, master = (torch.zeros(n + offset, dtype=t, device=DEV)[offset:] for t in (BF, torch.float32))
        param.copy_(w)
        master.copy_(w)
        master[5], master[130] = torch.nan, torch.inf
        g = torch.zeros_like(param)
        avg, sq, ms, rs = gk.grkan_adamw_state(param, bits)
        gk.grkan_adamw_step([param], [g], [avg], [sq], step=1, lr=0.1, weight_decay=0.0, masters=[master],
                            avg_scales=None if ms is None else [ms], sq_scales=None if rs is None else [rs])
        want = w.clone()
        want[5], want[130] = w[5].to(BF).float(), w[130].to(BF).float()
        assert torch.equal(master, want) and torch.equal(param, want.to(BF))
