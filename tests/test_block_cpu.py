"""CPU checks of the block operators: the header and the library agree, invalid arguments are refused before
any HIP call (the pointers below are never dereferenced), and the binding refuses what the library cannot
see."""
import ctypes
import os
import re

import pytest
import torch

from gr_kan_rational_amd import block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "grkan_block.h")
OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1
NONE, SILU, GELU, RATIONAL = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from gr_kan_rational_amd import binding

    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return block._library()


def p(k, offset=0):
    """A made-up address, 16 GB apart from the others'."""
    return ctypes.c_void_p((k << 34) + offset)


def test_header_declares_and_library_exports(lib):
    names = re.findall(r"GRKAN_API\s+[\w\s\*]*?\b(grkan_\w+)\s*\(", open(HEADER).read())
    assert sorted(names) == sorted(f"grkan_{op}_{way}{size}" for op in ("group_norm", "linear_act")
                                   for way in ("forward", "backward") for size in ("", "_workspace_size"))
    for n in names:
        assert hasattr(lib, n)
    text = open(HEADER).read()
    for k, v in (("NONE", NONE), ("SILU", SILU), ("GELU", GELU), ("RATIONAL", RATIONAL)):
        assert re.search(rf"GRKAN_ACT_{k} = {v}\b", text) and getattr(block, f"GRKAN_ACT_{k}") == v


# ---------------------------------------------------------------- group norm

NORM = dict(x=p(1), y=p(2), mean=p(3), rstd=p(4), weight=p(5), bias=p(6), A=p(7), B=p(8), n=4, s=10, c=64, xs=640,
            xr=64, groups=4, ng=8, eps=1e-5, act=RATIONAL, io=F32, ws=p(9), wsn=1 << 30)


def norm(lib, **kw):
    a = dict(NORM, **kw)
    return lib.grkan_group_norm_forward(*[a[k] for k in ("x", "y", "mean", "rstd", "weight", "bias", "A", "B", "n",
                                                         "s", "c", "xs", "xr", "groups", "ng", "eps", "act", "io",
                                                         "ws", "wsn")], None)


NORM_BAD = [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
    (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(act=SILU), INVALID),  # coefficients without the rational
    (dict(act=4), INVALID), (dict(act=-1), INVALID), (dict(io=2), INVALID), (dict(n=-1), INVALID),
    (dict(s=-1), INVALID), (dict(c=0), INVALID), (dict(groups=0), INVALID), (dict(groups=5), INVALID),
    (dict(ng=0), INVALID), (dict(ng=7), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(xr=63), INVALID), (dict(xs=-1), INVALID), (dict(xs=1 << 62), INVALID),
    (dict(x=p(1, 2)), UNSUPPORTED), (dict(y=p(2, 1)), UNSUPPORTED), (dict(mean=p(3, 2)), UNSUPPORTED),
    (dict(weight=p(5, 1)), UNSUPPORTED), (dict(A=p(7, 2)), UNSUPPORTED),
    (dict(c=1 << 24, xs=10 << 24, xr=1 << 24), UNSUPPORTED), (dict(s=1 << 31, xs=1 << 40), UNSUPPORTED),
    (dict(n=1 << 30), UNSUPPORTED),
    (dict(y=p(1, 4)), INVALID), (dict(y=p(5)), INVALID), (dict(mean=p(4)), INVALID), (dict(mean=p(1)), INVALID),
    (dict(y=p(1), xs=641), INVALID),  # in place on a strided x
]


@pytest.mark.parametrize("kw, status", NORM_BAD, ids=[str(k) for k, _ in NORM_BAD])
def test_group_norm_forward_refuses(lib, kw, status):
    assert norm(lib, **kw) == status


def test_group_norm_workspace(lib):
    size = lib.grkan_group_norm_forward_workspace_size
    assert size(4, 10, 64, 4, 8, RATIONAL, F32) == 0           # held on chip
    need = size(1, 65536, 128, 32, 8, SILU, F32)               # split: needs a workspace
    assert need > 0
    big = dict(n=1, s=65536, c=128, xs=65536 * 128, xr=128, groups=32, act=SILU, A=None, B=None)
    assert norm(lib, **big, wsn=need - 1) == INVALID
    assert norm(lib, **big, ws=None) == INVALID
    assert norm(lib, **big, ws=p(9, 64)) == UNSUPPORTED
    assert norm(lib, **big, ws=p(1)) == INVALID
    for bad in ((-1, 1, 64, 1, 8, SILU, F32), (1, 1, 64, 3, 8, SILU, F32), (1, 1, 64, 1, 8, 9, F32)):
        assert size(*bad) == 0
    assert norm(lib, n=0, x=None, y=None, mean=None, rstd=None) == OK


GRAD = dict(x=p(1), dy=p(2), mean=p(3), rstd=p(4), weight=p(5), bias=p(6), A=p(7), B=p(8), dx=p(10), dw=p(11),
            db=p(12), dA=p(13), dB=p(14), n=4, s=10, c=64, xs=640, xr=64, ds=640, dr=64, groups=4, ng=8,
            act=RATIONAL, io=F32, ws=p(9), wsn=1 << 30)


def grad(lib, **kw):
    a = dict(GRAD, **kw)
    return lib.grkan_group_norm_backward(*[a[k] for k in ("x", "dy", "mean", "rstd", "weight", "bias", "A", "B", "dx",
                                                          "dw", "db", "dA", "dB", "n", "s", "c", "xs", "xr", "ds",
                                                          "dr", "groups", "ng", "act", "io", "ws", "wsn")], None)


GRAD_BAD = [
    (dict(x=None), INVALID), (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(mean=None), INVALID),
    (dict(rstd=None), INVALID), (dict(dA=None), INVALID), (dict(dB=None), INVALID),
    (dict(act=SILU, A=None, B=None), INVALID),  # dA, dB without the rational
    (dict(dr=32), INVALID), (dict(ds=-4), INVALID), (dict(ws=None), INVALID), (dict(wsn=16), INVALID),
    (dict(dy=p(2, 1)), UNSUPPORTED), (dict(dx=p(10, 3)), UNSUPPORTED), (dict(dw=p(11, 2)), UNSUPPORTED),
    (dict(dw=p(12)), INVALID), (dict(dw=p(5)), INVALID), (dict(dx=p(1, 4)), INVALID), (dict(dA=p(7)), INVALID),
    (dict(dx=p(2), ds=1000), INVALID), (dict(ws=p(10)), INVALID), (dict(ws=p(9, 128)), UNSUPPORTED),
]


@pytest.mark.parametrize("kw, status", GRAD_BAD, ids=[str(k) for k, _ in GRAD_BAD])
def test_group_norm_backward_refuses(lib, kw, status):
    assert grad(lib, **kw) == status


# ---------------------------------------------------------------- linear map

LIN = dict(x=p(1), W=p(2), bias=p(3), r=p(4), A=p(5), B=p(6), z=p(7), pre=p(8), rows=100, d_in=64, d_out=48, ldx=64,
           ldr=48, ng=8, act=RATIONAL, ws=p(9), wsn=1 << 30)


def lin(lib, **kw):
    a = dict(LIN, **kw)
    return lib.grkan_linear_act_forward(*[a[k] for k in ("x", "W", "bias", "r", "A", "B", "z", "pre", "rows", "d_in",
                                                         "d_out", "ldx", "ldr", "ng", "act", "ws", "wsn")], None)


LIN_BAD = [
    (dict(x=None), INVALID), (dict(W=None), INVALID), (dict(z=None), INVALID), (dict(A=None), INVALID),
    (dict(act=GELU), INVALID), (dict(act=17), INVALID), (dict(rows=-1), INVALID), (dict(d_in=0), INVALID),
    (dict(d_out=0), INVALID), (dict(ng=7), INVALID), (dict(ng=0), INVALID), (dict(ldx=63), INVALID),
    (dict(ldr=47), INVALID), (dict(rows=1 << 31), UNSUPPORTED), (dict(d_in=(1 << 22) + 8, ldx=1 << 23), UNSUPPORTED),
    (dict(ldx=(1 << 22) + 2), UNSUPPORTED), (dict(x=p(1, 1)), UNSUPPORTED), (dict(z=p(7, 1)), UNSUPPORTED),
    (dict(bias=p(3, 2)), UNSUPPORTED), (dict(pre=p(8, 1)), UNSUPPORTED),
    (dict(rows=1 << 30, d_out=1 << 12, ldr=1 << 12), UNSUPPORTED),
    (dict(z=p(1)), INVALID), (dict(z=p(8)), INVALID), (dict(pre=p(4)), INVALID), (dict(z=p(4, 2)), INVALID),
    (dict(z=p(4), ldr=56), INVALID),  # in place on a strided residual
]


@pytest.mark.parametrize("kw, status", LIN_BAD, ids=[str(k) for k, _ in LIN_BAD])
def test_linear_forward_refuses(lib, kw, status):
    assert lin(lib, **kw) == status


def test_linear_workspace(lib):
    assert lin(lib, rows=0, x=None, z=None) == OK
    need = lib.grkan_linear_act_forward_workspace_size(200, 4096, 64, 8, SILU)  # k is split
    assert need > 0
    kw = dict(rows=200, d_in=4096, d_out=64, ldx=4096, ldr=64, act=SILU, A=None, B=None)
    assert lin(lib, **kw, wsn=need - 1) == INVALID and lin(lib, **kw, ws=None) == INVALID
    assert lin(lib, **kw, ws=p(9, 16)) == UNSUPPORTED
    assert lib.grkan_linear_act_forward_workspace_size(1, 4096, 64, 8, SILU) == 0
    assert lib.grkan_linear_act_backward_workspace_size(0, 64, 64, 8, SILU) == 0


LGRAD = dict(x=p(1), W=p(2), dz=p(3), pre=p(4), A=p(5), B=p(6), dx=p(10), dW=p(11), db=p(12), dA=p(13), dB=p(14),
             rows=100, d_in=64, d_out=48, ldx=64, lddz=48, ng=8, act=RATIONAL, ws=p(9), wsn=1 << 30)


def lgrad(lib, **kw):
    a = dict(LGRAD, **kw)
    return lib.grkan_linear_act_backward(*[a[k] for k in ("x", "W", "dz", "pre", "A", "B", "dx", "dW", "db", "dA",
                                                          "dB", "rows", "d_in", "d_out", "ldx", "lddz", "ng", "act",
                                                          "ws", "wsn")], None)


LGRAD_BAD = [
    (dict(x=None), INVALID), (dict(W=None), INVALID), (dict(dz=None), INVALID), (dict(pre=None), INVALID),
    (dict(dA=None), INVALID), (dict(act=SILU, A=None, B=None), INVALID), (dict(lddz=40), INVALID),
    (dict(ws=None), INVALID), (dict(wsn=100), INVALID), (dict(ws=p(9, 32)), UNSUPPORTED),
    (dict(dx=p(10, 1)), UNSUPPORTED), (dict(dW=p(11, 1)), UNSUPPORTED), (dict(db=p(12, 2)), UNSUPPORTED),
    (dict(dx=p(1)), INVALID), (dict(dx=p(3)), INVALID), (dict(dW=p(2)), INVALID), (dict(dW=p(10)), INVALID),
    (dict(db=p(9)), INVALID), (dict(lddz=1 << 23), UNSUPPORTED),
]


@pytest.mark.parametrize("kw, status", LGRAD_BAD, ids=[str(k) for k, _ in LGRAD_BAD])
def test_linear_backward_refuses(lib, kw, status):
    assert lgrad(lib, **kw) == status


# ---------------------------------------------------------------- the binding

BF = torch.bfloat16


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="GPU device"):
        block.grkan_group_norm_forward(x, 4)
    with pytest.raises(ValueError, match="GPU device"):
        block.grkan_group_norm_backward(x, x, x, x, 4)
    with pytest.raises(ValueError, match="GPU device"):
        block.grkan_linear_act_forward(x.to(BF), torch.zeros(8, 64, dtype=BF))
    with pytest.raises(ValueError, match="GPU device"):
        block.grkan_linear_act_backward(x.to(BF), torch.zeros(8, 64, dtype=BF), torch.zeros(4, 8, dtype=BF))
    with pytest.raises(TypeError):
        block.grkan_group_norm_forward(x.half(), 4)
    with pytest.raises(ValueError, match="act"):
        block.grkan_group_norm_forward(x, 4, act="relu")


def test_binding_reads_strides():
    t = torch.zeros(5, 12, 40)
    assert block._samples(t, "x") == (5, 12, 40, 480, 40)
    assert block._samples(t[:, 1:], "x") == (5, 11, 40, 480, 40)
    assert block._samples(t[:, :, 8:], "x") == (5, 12, 32, 480, 40)
    assert block._samples(t[:, ::2], "x") == (5, 6, 40, 480, 80)
    assert block._samples(t.view(5, 3, 4, 40)[..., :8], "x") == (5, 12, 8, 480, 40)
    assert block._samples(t[:, 0], "x")[:3] == (5, 1, 40)
    assert block._samples(t[0:1, 0, :], "x")[:3] == (1, 1, 40)
    for bad in (t.transpose(1, 2), t.view(5, 3, 4, 40)[:, :, :2], t[0, 0]):
        with pytest.raises(ValueError):
            block._samples(bad, "x")
    dev = torch.device("cpu")
    b = torch.zeros(6, 40, dtype=BF)
    assert block._rows(b, "x", dev) == (6, 40, 40)
    assert block._rows(b[:, 3:20], "x", dev) == (6, 17, 40)
    assert block._rows(b[::2], "x", dev) == (3, 40, 80)
    assert block._rows(b[0], "x", dev) == (1, 40, 40)
    for bad in (b.t(), b[:1].expand(6, 40), torch.zeros(3, 4, 40, dtype=BF)[:, :2]):
        with pytest.raises(ValueError):
            block._rows(bad, "x", dev)
    with pytest.raises(TypeError):
        block._rows(b.float(), "x", dev)


def test_binding_checks_coefficients():
    dev = torch.device("cpu")
    A, B = torch.zeros(8, 6), torch.zeros(8, 4)
    assert block._act_coefs(RATIONAL, A, B, 8, 64, dev)[2] == 8
    with pytest.raises(ValueError):
        block._act_coefs(RATIONAL, None, B, 8, 64, dev)
    with pytest.raises(ValueError):
        block._act_coefs(RATIONAL, A, B, 7, 64, dev)
    with pytest.raises(ValueError):
        block._act_coefs(RATIONAL, A[:4], B, 8, 64, dev)
    assert block._act_coefs(SILU, A, B, 8, 64, dev) == (None, None, 1)
    for bad in (torch.zeros(63), torch.zeros(64, dtype=torch.float64), torch.zeros(128)[::2]):
        with pytest.raises(ValueError):
            block._channel_vector(bad, "weight", 64, dev)


@pytest.mark.parametrize("rows", ((1 << 31) - 1, (1 << 31) - 64, (1 << 31) - 256))
def test_rows_whose_tiles_pass_32_bits_are_refused(lib, rows):
    """Row numbers of the last tile, 256 past the last row at most, have to fit 32 bits."""
    one = dict(rows=rows, d_in=1, d_out=1, ldx=1, act=SILU, A=None, B=None)
    assert lin(lib, **one, r=None) == UNSUPPORTED
    assert lgrad(lib, **one, lddz=1, dA=None, dB=None) == UNSUPPORTED
    assert lib.grkan_linear_act_forward_workspace_size(rows, 1, 1, 1, SILU) == 0
    assert lib.grkan_linear_act_backward_workspace_size(rows, 1, 1, 1, SILU) == 0
    assert lib.grkan_linear_act_backward_workspace_size((1 << 31) - 257, 1, 1, 1, SILU) > 0
