"""CPU checks of the operators of include/grkan_train.h, beside tests/test_train_cpu.py: what the library and the binding
refuse, and what the binding does around a call."""
import pytest
import torch

from gr_kan_rational_amd import train
from test_train_cpu import A8, BF16, F32, INVALID, NONE, UNSUPPORTED, T, adamw, lib, matmul, p, quantize  # noqa: F401


def test_kind_of_sums(lib):  # noqa: F811
    """One of two names; in the C ABI a flag beside b_tile, which does not hide other values of it."""
    assert open(__file__.replace("tests/test_train_checks_cpu.py", "include/grkan_train.h")).read().count(
        f"#define GRKAN_FP8_SUMS_CUT {train.GRKAN_FP8_SUMS_CUT}\n") == 1
    for tile in (18, 19, 15, 32, -1, -16):
        assert matmul(lib, tile=tile) == INVALID
    assert matmul(lib, tile=17, c=None) == INVALID and matmul(lib, tile=16, m=0, a=None, sa=None, c=None, out=F32) == 0
    f8, s = torch.zeros(4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(4, 1)
    with pytest.raises(ValueError, match="sums"):
        train.grkan_fp8_matmul(f8, s, f8, s, sums="fp16")
    from gr_kan_rational_amd.mixer import GRKANStack

    with pytest.raises(ValueError, match="sums"):
        GRKANStack(1, 16, 16, products="fp8", sums="bf16")


def test_optimizer_checks_its_numbers():
    w = torch.nn.Parameter(torch.zeros(4))
    for kw in (dict(betas=(0.9, 1.0)), dict(betas=(-0.1, 0.9)), dict(betas=(0.9,)), dict(betas=(float("nan"), 0.9)),
               dict(eps=-1e-8), dict(eps=float("nan")), dict(weight_decay=-0.1), dict(weight_decay=float("nan"))):
        with pytest.raises(ValueError, match=next(iter(kw))):
            train.GRKANAdamW([w], **kw)
    train.GRKANAdamW([w], betas=[0, 0.5], eps=0.0, weight_decay=0)


def test_a_refused_step_is_not_counted(monkeypatch):
    """Parameters that the step has taken count it, those behind a refusal do not, and a second try goes on from there."""
    a, b = (torch.nn.Parameter(torch.zeros(4)) for _ in range(2))
    a.grad, b.grad = torch.ones(4), torch.ones(4)
    opt = train.GRKANAdamW([{"params": [a]}, {"params": [b], "weight_decay": 0.5}])
    seen, refuse = [], [True]

    def step(params, *args, step, weight_decay, **kw):
        if weight_decay == 0.5 and refuse[0]:
            raise ValueError("refused")
        seen.append((params[0].data_ptr(), step))

    monkeypatch.setattr(train, "grkan_adamw_step", step)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    with pytest.raises(ValueError, match="refused"):
        opt.step()
    assert opt.state[a]["step"] == 1 and opt.state[b]["step"] == 0
    refuse[0] = False
    opt.step()
    assert opt.state[a]["step"] == 2 and opt.state[b]["step"] == 1
    assert seen == [(a.data_ptr(), 1), (a.data_ptr(), 2), (b.data_ptr(), 1)]


def test_quantiser_sizes(lib):  # noqa: F811
    """The header's limit, 2^24 blocks of 64 rows x 128 columns, is the one that is kept: a size below it passes to the
    next check (no x)."""
    for rows, cols, want in (((1 << 30) - 64, 128, INVALID), ((1 << 30) - 63, 128, UNSUPPORTED), (1 << 28, 129, INVALID),
                             ((1 << 29) - 64, 129, INVALID), (1 << 29, 129, UNSUPPORTED), (64, 1 << 22, INVALID)):
        ld = -(-rows // 16) * 16
        assert quantize(lib, x=None, A=None, B=None, act=NONE, rows=rows, cols=cols, ldx=cols, ldq=-(-cols // 16) * 16,
                        ls=rows, ldqt=ld, lst=cols, io=BF16) == want, (rows, cols)


def test_adamw_scalars_lie_apart(lib):  # noqa: F811
    """A scalar on the device that the step itself would write, by any of its tensors, in a first or a later launch."""
    many = [{k: p(100 + 8 * i + j) for j, k in enumerate(("param", "grad", "master", "avg", "sq"))} for i in range(60)]
    for name in ("lr_ptr", "step_ptr", "grad_scale"):
        for at in (p(1), p(1, 1992), p(3, 16), p(3, 3992), p(4), p(5, 800)):
            assert adamw(lib, [T], hyper={name: at}) == INVALID, (name, at)
        assert adamw(lib, many, hyper={name: p(100 + 8 * 59)}) == INVALID
        for at in (p(4), p(5, 8), p(6), p(7, 16)):
            assert adamw(lib, [dict(T, **A8)], 8, hyper={name: at}) == INVALID, (name, at)


def test_linear_refuses_rows_that_its_backward_would(monkeypatch):
    """W's gradient is a product over the rows, of which one takes 2^22: refused in the forward, unless W asks for
    none."""
    def reached(*args, **kw):
        raise InterruptedError

    monkeypatch.setattr(train, "grkan_fp8_quantize", reached)
    BF = torch.bfloat16
    x, few = torch.empty((3, (1 << 22) // 3 + 1, 8), dtype=BF), torch.empty((1 << 22, 8), dtype=BF)
    W = torch.empty((16, 8), dtype=BF, requires_grad=True)
    with pytest.raises(ValueError, match="rows"):
        train.GRKANFp8Linear.apply(x, W)
    for a, b in ((few, W), (x, W.detach())):
        with pytest.raises(InterruptedError):
            train.GRKANFp8Linear.apply(a, b)
    with torch.no_grad(), pytest.raises(InterruptedError):
        train.GRKANFp8Linear.apply(x, W)
