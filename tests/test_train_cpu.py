"""CPU checks of the operators of include/grkan_train.h: the header and the library agree, invalid arguments are
refused before any HIP call (the pointers below are never dereferenced), the binding refuses what the library
cannot see, and the numbers that the 8-bit states' rounding draws are even."""
import ctypes
import os
import re

import pytest
import torch

import train_ref as ref
from gr_kan_rational_amd import train

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "grkan_train.h")
OK, INVALID, UNSUPPORTED = 0, 1, 2
F32, BF16 = 0, 1
NONE, SILU, RATIONAL = 0, 1, 3
LAYER, RMS = 1, 2


@pytest.fixture(scope="module")
def lib():
    from gr_kan_rational_amd import binding

    if not os.path.exists(binding.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return train._library()


def p(k, offset=0):
    """A made-up address, 16 GB apart from the others'."""
    return ctypes.c_void_p((k << 34) + offset)


def test_header_declares_and_library_exports(lib):
    names = re.findall(r"GRKAN_API\s+[\w\s\*]*?\b(grkan_\w+)\s*\(", open(HEADER).read())
    assert sorted(names) == ["grkan_adamw_step", "grkan_fp8_matmul", "grkan_fp8_matmul_workspace_size",
                             "grkan_fp8_quantize", "grkan_residual_norm_backward",
                             "grkan_residual_norm_backward_workspace_size", "grkan_residual_norm_forward"]
    for n in names:
        assert hasattr(lib, n)
    text = open(HEADER).read()
    for k, v in (("NONE", 0), ("LAYER", LAYER), ("RMS", RMS)):
        assert re.search(rf"GRKAN_NORM_{k} = {v}\b", text) and getattr(train, f"GRKAN_NORM_{k}") == v
    # the structures' sizes: pointers, a count, an enumeration; five doubles, a step, three pointers, a seed
    assert ctypes.sizeof(train.grkan_adamw_tensor_t) == 72 and ctypes.sizeof(train.grkan_adamw_t) == 80


# ---------------------------------------------------------------- quantiser

Q = dict(x=p(1), A=p(2), B=p(3), q=p(4), s=p(5), qt=p(6), st=p(7), rows=100, cols=64, ldx=64, ldq=64, ls=100, ldqt=112,
         lst=64, tile=0, ng=8, act=RATIONAL, io=BF16)


def quantize(lib, **kw):
    a = dict(Q, **kw)
    return lib.grkan_fp8_quantize(*[a[k] for k in ("x", "A", "B", "q", "s", "qt", "st", "rows", "cols", "ldx", "ldq",
                                                   "ls", "ldqt", "lst", "tile", "ng", "act", "io")], None)


Q_BAD = [
    (dict(x=None), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(act=NONE), INVALID),
    (dict(act=SILU, A=None, B=None), INVALID), (dict(act=9), INVALID), (dict(io=2), INVALID), (dict(rows=-1), INVALID),
    (dict(cols=0), INVALID), (dict(ldx=63), INVALID), (dict(ng=0), INVALID), (dict(ng=7), INVALID),
    (dict(tile=2), INVALID), (dict(tile=-1), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID),
    (dict(qt=None), INVALID), (dict(st=None), INVALID), (dict(q=None, s=None, qt=None, st=None), INVALID),
    (dict(ldq=48), INVALID), (dict(ls=99), INVALID), (dict(ldqt=96), INVALID), (dict(lst=63), INVALID),
    (dict(ldq=72), UNSUPPORTED), (dict(ldqt=104), UNSUPPORTED), (dict(q=p(4, 8)), UNSUPPORTED),
    (dict(qt=p(6, 1)), UNSUPPORTED), (dict(s=p(5, 2)), UNSUPPORTED), (dict(x=p(1, 1)), UNSUPPORTED),
    (dict(rows=(1 << 31) - 1), UNSUPPORTED), (dict(ldx=(1 << 22) + 2), UNSUPPORTED),
    (dict(rows=1 << 30, cols=1 << 12, ldx=1 << 12), UNSUPPORTED),
    (dict(q=p(1)), INVALID), (dict(q=p(6)), INVALID), (dict(s=p(7)), INVALID), (dict(st=p(2)), INVALID),
    (dict(qt=p(4, 16)), INVALID),
]


@pytest.mark.parametrize("kw, status", Q_BAD, ids=[str(k) for k, _ in Q_BAD])
def test_quantize_refuses(lib, kw, status):
    assert quantize(lib, **kw) == status


def test_quantize_of_no_rows(lib):
    assert quantize(lib, rows=0, x=None, q=None, s=None, qt=None, st=None) == OK


# ---------------------------------------------------------------- product

G = dict(a=p(1), sa=p(2), b=p(3), sb=p(4), bias=p(5), r=p(6), c=p(7), m=100, n=48, k=300, lda=304, sar=1, sab=100,
         ldb=320, sbr=3, sbb=1, tile=0, ldr=48, out=BF16, ws=p(9), wsn=1 << 30)


def matmul(lib, **kw):
    a = dict(G, **kw)
    return lib.grkan_fp8_matmul(*[a[k] for k in ("a", "sa", "b", "sb", "bias", "r", "c", "m", "n", "k", "lda", "sar",
                                                 "sab", "ldb", "sbr", "sbb", "tile", "ldr", "out", "ws", "wsn")], None)


G_BAD = [
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(sa=None), INVALID), (dict(sb=None), INVALID),
    (dict(c=None), INVALID), (dict(m=-1), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(out=2), INVALID),
    (dict(tile=2), INVALID), (dict(lda=288), INVALID), (dict(ldb=288), INVALID), (dict(ldr=47), INVALID),
    (dict(sar=-1), INVALID), (dict(sbb=-1), INVALID), (dict(lda=308), UNSUPPORTED), (dict(ldb=328), UNSUPPORTED),
    (dict(a=p(1, 8)), UNSUPPORTED), (dict(b=p(3, 4)), UNSUPPORTED), (dict(sa=p(2, 2)), UNSUPPORTED),
    (dict(bias=p(5, 1)), UNSUPPORTED), (dict(c=p(7, 1)), UNSUPPORTED), (dict(r=p(6, 2), out=F32), UNSUPPORTED),
    (dict(m=(1 << 31) - 1), UNSUPPORTED), (dict(n=(1 << 22) + 1, ldr=(1 << 22) + 1), UNSUPPORTED),
    (dict(lda=(1 << 22) + 16), UNSUPPORTED), (dict(sar=1 << 31), UNSUPPORTED),
    (dict(m=1 << 30, n=1 << 12, ldr=1 << 12), UNSUPPORTED),
    (dict(c=p(1)), INVALID), (dict(c=p(5)), INVALID), (dict(c=p(6, 2)), INVALID), (dict(c=p(6), ldr=56), INVALID),
]


@pytest.mark.parametrize("kw, status", G_BAD, ids=[str(k) for k, _ in G_BAD])
def test_matmul_refuses(lib, kw, status):
    assert matmul(lib, **kw) == status


def test_matmul_workspace(lib):
    assert matmul(lib, m=0, a=None, sa=None, c=None) == OK
    size = lib.grkan_fp8_matmul_workspace_size
    assert size(0, 10, 10) == 0 and size(-1, 10, 10) == 0 and size(10, 0, 10) == 0 and size(10, 10, 0) == 0
    need = size(200, 64, 65536)
    if need:
        kw = dict(m=200, n=64, k=65536, lda=65536, ldb=65536, ldr=64)
        assert matmul(lib, **kw, wsn=need - 1) == INVALID and matmul(lib, **kw, ws=None) == INVALID
        assert matmul(lib, **kw, ws=p(9, 64)) == UNSUPPORTED and matmul(lib, **kw, ws=p(3)) == INVALID


# ---------------------------------------------------------------- residual path

R = dict(x=p(1), f=p(2), w=p(3), b=p(4), s=p(5), gate=p(6), pw=p(7), pb=p(8), h=p(9), z=p(10), stats=p(11), rows=24,
         c=64, ldx=64, ldf=64, gates=4, gc=64, eps=1e-5, norm=LAYER, post=RMS, io=BF16, gio=BF16)


def residual(lib, **kw):
    a = dict(R, **kw)
    return lib.grkan_residual_norm_forward(*[a[k] for k in ("x", "f", "w", "b", "s", "gate", "pw", "pb", "h", "z",
                                                            "stats", "rows", "c", "ldx", "ldf", "gates", "gc", "eps",
                                                            "norm", "post", "io", "gio")], None)


R_BAD = [
    (dict(x=None), INVALID), (dict(f=None), INVALID), (dict(h=None), INVALID), (dict(z=None), INVALID),
    (dict(stats=None), INVALID), (dict(rows=-1), INVALID), (dict(c=0), INVALID), (dict(norm=0), INVALID),
    (dict(norm=3), INVALID), (dict(post=3), INVALID), (dict(post=0), INVALID),  # post_weight without a post norm
    (dict(io=2), INVALID), (dict(gio=2), INVALID), (dict(io=F32, gio=BF16), INVALID), (dict(gates=5), INVALID),
    (dict(gates=0), INVALID), (dict(gates=-4), INVALID), (dict(gc=2), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(ldx=63), INVALID), (dict(ldf=63), INVALID),
    (dict(c=16385, ldx=16385, ldf=16385, gc=1), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(ldx=(1 << 31) + 2), UNSUPPORTED), (dict(x=p(1, 1)), UNSUPPORTED), (dict(z=p(10, 1)), UNSUPPORTED),
    (dict(w=p(3, 2)), UNSUPPORTED), (dict(stats=p(11, 2)), UNSUPPORTED), (dict(gate=p(6, 1)), UNSUPPORTED),
    (dict(gate=p(6, 2), gio=F32), UNSUPPORTED), (dict(h=p(1, 2)), INVALID), (dict(h=p(1), ldx=80), INVALID),
    (dict(z=p(1)), INVALID), (dict(z=p(2)), INVALID), (dict(h=p(2)), INVALID), (dict(z=p(9)), INVALID),
    (dict(stats=p(6)), INVALID), (dict(h=p(6)), INVALID),
]


@pytest.mark.parametrize("kw, status", R_BAD, ids=[str(k) for k, _ in R_BAD])
def test_residual_forward_refuses(lib, kw, status):
    assert residual(lib, **kw) == status


D = dict(f=p(1), h=p(2), dh=p(3), dz=p(4), stats=p(5), w=p(6), s=p(7), gate=p(8), pw=p(9), pb=p(10), dx=p(11), df=p(12),
         ds=p(13), dg=p(14), dw=p(15), db=p(16), dpw=p(17), dpb=p(18), rows=24, c=64, ldf=64, ldh=64, ldz=64, gates=4,
         gc=64, norm=LAYER, post=RMS, io=BF16, gio=BF16, ws=p(19), wsn=1 << 30)


def residual_grad(lib, **kw):
    a = dict(D, **kw)
    return lib.grkan_residual_norm_backward(*[a[k] for k in ("f", "h", "dh", "dz", "stats", "w", "s", "gate", "pw", "pb",
                                                             "dx", "df", "ds", "dg", "dw", "db", "dpw", "dpb", "rows",
                                                             "c", "ldf", "ldh", "ldz", "gates", "gc", "norm", "post",
                                                             "io", "gio", "ws", "wsn")], None)


D_BAD = [
    (dict(f=None), INVALID), (dict(h=None), INVALID), (dict(stats=None), INVALID), (dict(dh=None, dz=None), INVALID),
    (dict(gate=None), INVALID),  # dgate without a gate
    (dict(post=0), INVALID), (dict(post=0, pw=None, pb=None), INVALID), (dict(gates=5), INVALID), (dict(gc=3), INVALID),
    (dict(ldf=60), INVALID), (dict(ldh=60), INVALID), (dict(ldz=60), INVALID), (dict(ws=None), INVALID),
    (dict(wsn=64), INVALID), (dict(ws=p(19, 32)), UNSUPPORTED), (dict(dx=p(11, 1)), UNSUPPORTED),
    (dict(dw=p(15, 2)), UNSUPPORTED), (dict(dg=p(14, 1)), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(dx=p(4)), INVALID), (dict(df=p(3)), INVALID), (dict(dx=p(3), ldh=80), INVALID), (dict(dx=p(3, 8)), INVALID),
    (dict(dx=p(12)), INVALID), (dict(dx=p(1)), INVALID), (dict(df=p(2)), INVALID), (dict(ds=p(15)), INVALID),
    (dict(dg=p(8)), INVALID), (dict(ws=p(13)), INVALID),
]


@pytest.mark.parametrize("kw, status", D_BAD, ids=[str(k) for k, _ in D_BAD])
def test_residual_backward_refuses(lib, kw, status):
    assert residual_grad(lib, **kw) == status


def test_residual_of_no_rows(lib):
    assert residual(lib, rows=0, x=None, f=None, h=None, z=None, stats=None) == OK
    size = lib.grkan_residual_norm_backward_workspace_size
    assert size(0, 64, 0, 1, RMS, BF16) == 0 and size(24, 64, 5, 64, RMS, BF16) == 0
    assert size(24, 64, 0, 1, 7, BF16) == 0 and size(24, 64, 0, 1, 0, BF16) > 0


# ---------------------------------------------------------------- AdamW

T = dict(param=p(1), grad=p(2), master=p(3), avg=p(4), sq=p(5), n=1000, io=BF16)
H = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1)


def adamw(lib, tensors, bits=32, hyper=None, count=None):
    table = (train.grkan_adamw_tensor_t * max(1, len(tensors)))()
    for row, t in zip(table, tensors):
        for k, v in dict(T, **t).items():
            setattr(row, k, v)
    h = train.grkan_adamw_t(**dict(H, **(hyper or {})))
    return lib.grkan_adamw_step(ctypes.addressof(table), len(tensors) if count is None else count, ctypes.byref(h), bits, None)


A_BAD = [
    (dict(param=None), INVALID), (dict(grad=None), INVALID), (dict(avg=None), INVALID), (dict(sq=None), INVALID),
    (dict(n=-1), INVALID), (dict(io=2), INVALID), (dict(avg_scale=p(6)), INVALID), (dict(param=p(1, 1)), UNSUPPORTED),
    (dict(master=p(3, 2)), UNSUPPORTED), (dict(avg=p(4, 2)), UNSUPPORTED), (dict(n=1 << 40), UNSUPPORTED),
    (dict(param=p(2)), INVALID), (dict(avg=p(5, 400)), INVALID), (dict(master=p(4, 16)), INVALID),
]
A8 = dict(avg_scale=p(6), sq_scale=p(7))
A8_BAD = [(dict(avg_scale=None), INVALID), (dict(sq_scale=None), INVALID), (dict(avg=p(4, 8)), UNSUPPORTED),
          (dict(sq=p(5, 4)), UNSUPPORTED), (dict(avg_scale=p(6, 2)), UNSUPPORTED), (dict(sq=p(4, 1008)), INVALID),
          (dict(sq_scale=p(6, 28)), INVALID)]


@pytest.mark.parametrize("kw, status", A_BAD, ids=[str(k) for k, _ in A_BAD])
def test_adamw_refuses(lib, kw, status):
    assert adamw(lib, [kw]) == status


@pytest.mark.parametrize("kw, status", A8_BAD, ids=[str(k) for k, _ in A8_BAD])
def test_adamw8_refuses(lib, kw, status):
    assert adamw(lib, [dict(A8, **kw)], 8) == status


def test_adamw_hyper_parameters(lib):
    for bad in (dict(lr=-1.0), dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.5), dict(eps=-1.0),
                dict(weight_decay=-1.0), dict(step=0), dict(beta2=float("nan"))):
        assert adamw(lib, [T], hyper=bad) == INVALID
    assert adamw(lib, [T], bits=16) == INVALID and adamw(lib, [], count=-1) == INVALID
    assert adamw(lib, [T], hyper=dict(lr_ptr=p(20, 2))) == UNSUPPORTED
    assert adamw(lib, [T], hyper=dict(step_ptr=p(20, 4))) == UNSUPPORTED
    assert adamw(lib, []) == OK and adamw(lib, [dict(n=0)] * 100) == OK


def test_adamw_refuses_the_same_tensor_twice(lib):
    """In one launch, in the second launch, and as another's state; nothing is launched before all is checked."""
    def far(i, **kw):
        return dict({k: p(100 + 8 * i + j) for j, k in enumerate(("param", "grad", "master", "avg", "sq"))}, **kw)

    many = [far(i) for i in range(60)]
    assert adamw(lib, [T, T]) == INVALID
    assert adamw(lib, [*many, far(59)]) == INVALID
    assert adamw(lib, [far(0), far(1, avg=p(100, 100))]) == INVALID


# ---------------------------------------------------------------- the binding

BF = torch.bfloat16


def test_binding_refuses_host_tensors_and_types():
    x, f8 = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.ones(4, 1)
    for call in (lambda: train.grkan_fp8_quantize(x), lambda: train.grkan_fp8_matmul(f8, s, f8, s),
                 lambda: train.grkan_residual_norm_forward(x, x), lambda: train.grkan_residual_norm_backward(x, x, x, x, x),
                 lambda: train.grkan_adamw_step([x], [x], [x], [x], step=1, lr=0.1)):
        with pytest.raises(ValueError, match="GPU device"):
            call()
    with pytest.raises(TypeError):
        train.grkan_fp8_quantize(x.half())
    with pytest.raises(ValueError, match="outputs"):
        train.grkan_fp8_quantize(x, "row")
    with pytest.raises(ValueError, match="act"):
        train.grkan_fp8_quantize(x, act="silu")
    with pytest.raises(ValueError, match="norm"):
        train.grkan_residual_norm_forward(x, x, norm="none")
    with pytest.raises(ValueError, match="list"):
        train.grkan_adamw_step([x], [], [x], [x], step=1, lr=0.1)
    with pytest.raises(ValueError, match="together"):
        train.grkan_adamw_step([x], [x], [x], [x], step=1, lr=0.1, avg_scales=[x])
    with pytest.raises(TypeError, match="bfloat16"):
        train.GRKANFp8Linear.apply(x, x)
    train.grkan_adamw_step([], [], [], [], step=1, lr=0.1)


def test_binding_reads_gates():
    dev = torch.device("cpu")
    lead, c = (3, 5), 64

    def gate(*shape, dtype=torch.float32):
        return train._gate(torch.zeros(shape, dtype=dtype), lead, 15, c, BF, dev)

    assert train._gate(None, lead, 15, c, BF, dev) == (0, 1, F32)
    assert gate(3, 5, 64) == (15, 64, F32) and gate(3, 1, 64, dtype=BF) == (3, 64, BF16)
    assert gate(3, 1, 1) == (3, 1, F32) and gate(1, 1, 1) == (1, 1, F32) and gate(1, 1, 64) == (1, 64, F32)
    for bad in ((1, 5, 64), (3, 64), (3, 5, 2), (2, 5, 1), (64,)):
        with pytest.raises(ValueError):
            gate(*bad)
    with pytest.raises(ValueError):
        gate(3, 5, 64, dtype=torch.float16)
    assert train._gate(torch.zeros(1, 1, 1), (1, 1), 1, c, BF, dev)[:2] == (1, 1)


def test_binding_reads_operands():
    dev = torch.device("cpu")
    buf = torch.zeros(6, 64, dtype=torch.uint8)
    t = buf.view(torch.float8_e4m3fn)
    if t.data_ptr() % 16 == 0:
        assert train._operand8(t, "a", dev) == (6, 64, 64) and train._operand8(t[:, :40], "a", dev) == (6, 40, 64)
        assert train._operand8(t[:1, :40], "a", dev) == (1, 40, 48)
        with pytest.raises(ValueError, match="16 bytes"):
            train._operand8(t[:, 8:], "a", dev)
    with pytest.raises(ValueError):
        train._operand8(t.t(), "a", dev)
    with pytest.raises(TypeError):
        train._operand8(buf, "a", dev)
    s = torch.ones(6, 1)
    assert train._scale8(s, "s", (6,), 64, dev) == (1, 1)
    for bad in (s[:5], torch.ones(6, 2), s.double(), torch.ones(6)):
        with pytest.raises(ValueError):
            train._scale8(bad, "s", (6,), 64, dev)


def test_optimizer_refuses():
    w = torch.nn.Parameter(torch.zeros(4))
    with pytest.raises(ValueError, match="bits"):
        train.GRKANAdamW([w], bits=16)
    with pytest.raises(ValueError, match="lr"):
        train.GRKANAdamW([w], lr=-1.0)
    with pytest.raises(ValueError, match="bits"):
        train.grkan_adamw_state(w, 4)


def test_random_numbers_are_even():
    """The rounding's numbers over seeds, steps, blocks and places: each of the 32 bits is set in half of them, and
    the two 16-bit numbers of a value, and those of neighbours, do not go together (all within 5 standard errors)."""
    draws = torch.cat([ref.random32(seed, step, 1000 * seed, 64).reshape(-1) for seed in range(8) for step in (1, 2, 77)])
    n = draws.numel()
    for bit in range(32):
        assert abs(((draws >> bit) & 1).double().mean() - 0.5) < 5 * 0.5 / n ** 0.5
    lo, hi = (draws & 0xFFFF).double() / 65536 - 0.5, (draws >> 16).double() / 65536 - 0.5
    for a, b in ((lo, hi), (lo[1:], lo[:-1]), (hi[1:], hi[:-1]), (lo[128:], lo[:-128]), (lo[64 * 128:], lo[:-64 * 128])):
        assert abs((a * b).mean()) < 5 / 12 / n ** 0.5
    for v in (lo, hi):
        assert abs(v.mean()) < 5 * 12 ** -0.5 / n ** 0.5
        counts = torch.histc(v, 64, -0.5, 0.5)
        assert (counts - n / 64).abs().max() < 5 * (n / 64) ** 0.5


def test_stack_gates_of_one_row():
    """x without leading dimensions is one sample."""
    from gr_kan_rational_amd.mixer import GRKANStack

    s = GRKANStack(2, 16, 16, drop=0.5).train()
    assert [tuple(g.shape) for g in s.gates(torch.zeros(16))] == [(1,), (1,)]
    assert [tuple(g.shape) for g in s.gates(torch.zeros(3, 5, 16))] == [(3, 1, 1)] * 2


def test_binding_reads_gates_of_no_rows(lib):
    cpu = torch.device("cpu")
    for lead, gate, want in (((0, 5), (0, 1, 1), 0), ((0, 5), (1, 1, 24), 1), ((3, 0), (3, 1, 1), 3)):
        assert train._gate(torch.ones(gate), lead, 0, 24, torch.float32, cpu)[:2] == (want, gate[-1])
    assert residual_grad(lib, rows=0, gates=1 << 31) == UNSUPPORTED
