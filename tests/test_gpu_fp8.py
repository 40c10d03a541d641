"""GPU tests of the 8-bit quantiser and matrix product against their definitions in fp64; the bounds are derived
in tests/train_ref.py."""
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


def normal(shape, seed, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(DEV).to(dtype)


def spread(shape, seed, dtype=torch.float32):
    """Values over 40 binades, one scale a column and a row."""
    gen = torch.Generator().manual_seed(seed + 1)
    x = normal(shape, seed).double()
    x *= (2.0 ** torch.randint(-10, 11, (shape[-1],), generator=gen)).to(DEV)
    x *= (2.0 ** torch.randint(-10, 11, (x.numel() // shape[-1],), generator=gen)).to(DEV).view(*shape[:-1], 1)
    return x.to(dtype)


def same_codes(q, s, want):
    v, sc = want
    assert s.shape == sc.shape and torch.equal(s.double(), sc), f"scales: {int((s.double() != sc).sum())} differ"
    got = q.float().double()
    assert got.shape == v.shape and torch.equal(torch.nan_to_num(got, 1e9), torch.nan_to_num(v, 1e9)), "codes"


# ---------------------------------------------------------------- quantiser

SHAPES = [(1, 1), (1, 768), (3, 17), (128, 128), (129, 127), (16, 256), (200, 333), (257, 768), (1000, 64), (7, 2056)]


@pytest.mark.parametrize("dtype", (torch.float32, BF))
@pytest.mark.parametrize("tile", (False, True))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize(gk, shape, tile, dtype):
    """Codes and scales equal the definition's, in both layouts and alone."""
    print(f"[quantize] {shape} {tile} {dtype}", flush=True)
    x = spread(shape, sum(shape), dtype)
    rows, cols = ref.quantized(x, tile), ref.quantized(x.t(), tile)
    q, s, qt, st = gk.grkan_fp8_quantize(x, "both", tile=tile)
    same_codes(q, s, rows)
    same_codes(qt, st, cols)
    same_codes(*gk.grkan_fp8_quantize(x, tile=tile), rows)
    same_codes(*gk.grkan_fp8_quantize(x, "columns", tile=tile), cols)
    assert q.stride(0) % 16 == 0 and qt.stride(0) % 16 == 0
    for t in (q, qt):  # the bytes up to the next multiple of 16
        pad = torch.as_strided(t.view(torch.uint8), (t.shape[0], t.stride(0)), (t.stride(0), 1))[:, t.shape[1]:]
        assert not pad.any()


@pytest.mark.parametrize("outputs", ("rows", "columns", "both"))
def test_quantize_special_values(gk, outputs):
    """NaN and infinities become NaN and do not enter their block's scale; zeros, subnormals, the largest numbers
    and values that round to 448 or to even."""
    x = normal((130, 260), 3)
    x[0] = 0.0
    x[1, :128] = torch.nan
    x[2, 5], x[2, 6], x[2, 200] = torch.inf, -torch.inf, torch.nan
    x[3] = 1e-42
    x[4, 0] = 3.4e38
    x[5, :128], x[5, 0] = torch.linspace(-448, 448, 128), 448.0
    x[6, :128], x[6, 0] = torch.arange(128) * 0.5 + 16, 448.0    # halves of e4m3 steps
    x[7, :128], x[7, 0] = 1.0, 448.00003
    got = gk.grkan_fp8_quantize(x, outputs)
    if outputs != "columns":
        same_codes(got[0], got[1], ref.quantized(x))
    if outputs != "rows":
        same_codes(got[-2], got[-1], ref.quantized(x.t()))


@pytest.mark.parametrize("outputs", ("rows", "columns", "both"))
@pytest.mark.parametrize("dtype", (torch.float32, BF))
@pytest.mark.parametrize("shape, groups", [((65, 768), 8), ((3, 40), 5), ((130, 24), 24), ((200, 104), 8)], ids=str)
def test_quantize_rational(gk, shape, groups, dtype, outputs):
    """F(x) in fp32 is within its bound of the exact value: the scale and the codes are those of a value that near,
    so every code is within half a step of the exact value at the larger of the two scales, plus that bound."""
    x = normal(shape, 5, 1.5, dtype)
    A, B = normal((groups, 6), 6, 0.5), normal((groups, 4), 7, 0.5)
    y, ey, _, _, _ = ref.activation(x.double(), torch.zeros_like(x.double()), "rational", A, B)
    got = gk.grkan_fp8_quantize(x, outputs, act="rational", A=A, B=B, n_groups=groups)
    for q, s, v, e in ((got[0], got[1], y, ey), (got[-2], got[-1], y.t(), ey.t())):
        if q.shape != v.shape or (outputs == "rows" and v is not y) or (outputs == "columns" and v is y):
            continue
        amax = torch.nn.functional.pad(v.abs(), (0, -v.shape[1] % 128)).view(v.shape[0], -1, 128).amax(2)
        emax = torch.nn.functional.pad(e, (0, -v.shape[1] % 128)).view(v.shape[0], -1, 128).amax(2)
        assert ((s >= ref.scale_of((amax - emax).clamp_min(0))) & (s <= ref.scale_of(amax + emax))).all()
        sv = s.double().repeat_interleave(128, 1)[:, :v.shape[1]]
        step = ref.binade((v.abs() / sv).clamp_min(2.0 ** -6)) / 8 * sv
        ref.check("F(x)", ref.values(q, s), v, step / 2 + e)


def test_quantize_strided(gk):
    """Rows of a wider tensor, an odd offset, three dimensions: the dense tensor's results; both directions of
    no rows."""
    x = spread((6, 20, 96), 8, BF)
    want = gk.grkan_fp8_quantize(x, "both")
    wide = torch.full((6, 20, 131), 9.0, dtype=BF, device=DEV)
    wide[..., 3:99] = x
    for a, b in zip(want, gk.grkan_fp8_quantize(wide[..., 3:99], "both")):
        assert torch.equal(a.float(), b.float())
    q, s, qt, st = gk.grkan_fp8_quantize(x[:0], "both")
    assert q.shape == (0, 96) and s.shape == (0, 1) and qt.shape == (96, 0) and st.shape == (96, 0)


# ---------------------------------------------------------------- product

# (m, n, k)
PRODUCTS = [(1, 1, 1), (1, 768, 256), (1, 40, 1000), (5, 130, 129), (16, 64, 128), (17, 96, 384), (33, 200, 16),
            (64, 64, 127), (65, 65, 300), (100, 700, 64), (197, 384, 768), (257, 129, 257), (300, 520, 200),
            (64, 48, 4096), (40, 72, 3001)]


def operands(shape, tile, seed):
    m, n, k = shape

    def one(rows, seed, tiled):
        gen = torch.Generator().manual_seed(seed)
        x = torch.randn((rows, k), generator=gen) * 2.0 ** torch.randint(-4, 5, (k,), generator=gen)
        q = torch.full((rows, ref.ceil(k, 16) * 16), 0x7F, dtype=torch.uint8)  # NaN past the end
        q[:, :k] = ref.to_e4m3((x * 20).double().clamp(-448, 448)).to(F8).view(torch.uint8)
        s = torch.rand((ref.ceil(rows, 128) if tiled else rows, ref.ceil(k, 128)), generator=gen) + 0.5
        return q.to(DEV).view(F8)[:, :k], s.to(DEV)

    return one(m, seed, False), one(n, seed + 1, tile)


@pytest.mark.parametrize("dtype", (BF, torch.float32))
@pytest.mark.parametrize("tile", (True, False))
@pytest.mark.parametrize("shape", PRODUCTS, ids=str)
def test_matmul(gk, shape, tile, dtype):
    print(f"[matmul] {shape} {tile} {dtype}", flush=True)
    m, n, k = shape
    (a, sa), (b, sb) = operands(shape, tile, 10 + sum(shape))
    bias, r = normal((n,), 11), normal((m, n), 12, 3.0, dtype)
    for bi, re in ((None, None), (bias, None), (None, r), (bias, r)):
        want = ref.matmul(a, sa, b, sb, tile, bi, re, dtype)
        got = gk.grkan_fp8_matmul(a, sa, b, sb, bias=bi, residual=re, dtype=dtype)
        assert got.dtype == dtype
        ref.check(f"{shape}", got, *want)
        assert torch.equal(got, gk.grkan_fp8_matmul(a, sa, b, sb, bias=bi, residual=re, dtype=dtype)), "two calls differ"


# tiles of 64; of 256 rows, whole and odd, one block of k and several, the last rows apart; k split, its end inside a block
LARGE = [(700, 1100, 200), (513, 1025, 333), (9000, 2304, 1000),
         (4096, 4096, 128), (4100, 2100, 300), (8200, 2056, 100), (2049, 4107, 777), (300, 264, 20000), (520, 100, 30001)]


@pytest.mark.parametrize("dtype, tile", ((BF, True), (BF, False), (torch.float32, False)))
@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_matmul_large(gk, shape, dtype, tile):
    test_matmul(gk, shape, tile, dtype)


def test_matmul_layouts(gk):
    """Scales side by side in either order or expanded from one, operands in wider tensors, outputs off their
    16-byte boundary, in place on the residual: the same bits as dense ones; nothing outside the output."""
    m, n, k = 150, 200, 400
    (a, sa), (b, sb) = operands((m, n, k), True, 21)
    r = normal((m, n), 22, 1.0, BF)
    want = gk.grkan_fp8_matmul(a, sa, b, sb, residual=r)
    assert torch.equal(want, gk.grkan_fp8_matmul(a, sa.t().contiguous().t(), b, sb.t().contiguous().t(), residual=r))
    wide = torch.zeros((m, 608), dtype=torch.uint8, device=DEV).view(F8)
    wide.view(torch.uint8)[:, 96:96 + k] = a.view(torch.uint8)
    assert torch.equal(want, gk.grkan_fp8_matmul(wide[:, 96:96 + k], sa, b, sb, residual=r))
    r2 = r.clone()
    assert torch.equal(want, gk.grkan_fp8_matmul(a, sa, b, sb, residual=r2, out=r2))
    buf = torch.full((m * n + 2,), 7.0, dtype=BF, device=DEV)
    gk.grkan_fp8_matmul(a, sa, b, sb, residual=r, out=buf[1:-1].view(m, n))
    assert torch.equal(want, buf[1:-1].view(m, n)) and float(buf[0]) == 7.0 and float(buf[-1]) == 7.0
    one = torch.tensor([[0.25]], device=DEV)
    sa1, sb1 = one.expand(m, 4), one.expand(n, 4)
    ref.check("one scale", gk.grkan_fp8_matmul(a, sa1, b, sb1), *ref.matmul(a, sa1, b, sb1, False))
    assert gk.grkan_fp8_matmul(a[:0], sa[:0], b, sb).shape == (0, n)


def test_matmul_special_values(gk):
    """A NaN stays in its row or column; large and small scales meet without loss."""
    (a, sa), (b, sb) = operands((70, 90, 256), False, 31)
    a = a.clone()
    a.view(torch.uint8)[3, 200] = 0x7F
    for dtype in (BF, torch.float32):
        c = gk.grkan_fp8_matmul(a, sa, b, sb, dtype=dtype)
        assert c[3].isnan().all() and c[:3].isfinite().all() and c[4:].isfinite().all()
    a.view(torch.uint8)[3, 200] = 0
    want = gk.grkan_fp8_matmul(a, sa, b, sb, dtype=torch.float32)
    got = gk.grkan_fp8_matmul(a, sa * 2.0 ** 100, b, sb * 2.0 ** -100, dtype=torch.float32)
    assert torch.equal(want, got)


# ---------------------------------------------------------------- together

def rational64(x, A, B):
    return ref.activation(x, torch.zeros_like(x), "rational", A, B)[0]


@pytest.mark.parametrize("act", ("none", "rational"))
def test_linear_gradients(gk, act):
    """y = F(x) W^T + b and its gradients against fp64 with the operands the products see (the quantised ones):
    what is left is the products' rounding and bf16, 2^-8 a value; dx through F' once more."""
    rows, d_in, d_out, groups = 300, 256, 200, 8
    x = normal((3, 100, d_in), 41, 1.0, BF).requires_grad_()
    W = normal((d_out, d_in), 42, d_in ** -0.5, BF).requires_grad_()
    b = normal((d_out,), 43).requires_grad_()
    A = normal((groups, 6), 44, 0.5).requires_grad_() if act == "rational" else None
    B = normal((groups, 4), 45, 0.5).requires_grad_() if act == "rational" else None
    dy = normal((3, 100, d_out), 46, 0.1, BF)
    y = gk.GRKANFp8Linear.apply(x, W, b, act, A, B, groups)
    y.backward(dy)
    xd = x.detach().double().view(rows, d_in)
    fx = xd if act == "none" else rational64(xd, A.detach(), B.detach())
    g = dy.double().view(rows, d_out)

    def q(t, tile=False):
        v, s = ref.quantized(t, tile)
        s = s.repeat_interleave(128, 1)[:, :t.shape[1]]
        return v * (s.repeat_interleave(128, 0)[:t.shape[0]] if tile else s)

    wq = q(W.detach(), True)

    def close(what, got, want, tol):
        err = float((got.detach().double() - want).norm())
        assert err <= tol * float(want.norm()), f"{what}: {err / float(want.norm())}"

    close("y", y.view(rows, d_out), q(fx) @ wq.t() + b.detach().double(), 2 ** -8)
    close("dbias", b.grad, g.sum(0), 1e-6)
    # (F in fp32 may move a value over a rounding's border: one e4m3 step of 2^-4 in a few of 76,800)
    close("dW", W.grad, q(g.t().contiguous()) @ q(fx.t().contiguous()).t(), 2 ** -8)
    dfx = (q(g) @ wq).requires_grad_(False)
    if act == "none":
        close("dx", x.grad.view(rows, d_in), dfx, 2 ** -8)
    else:
        xx = xd.clone().requires_grad_()
        Ad, Bd = A.detach().double().requires_grad_(), B.detach().double().requires_grad_()
        v = xx.view(rows, groups, -1)
        P = sum(Ad[:, i].view(1, groups, 1) * v ** i for i in range(6))
        Q = sum(Bd[:, j].view(1, groups, 1) * v ** (j + 1) for j in range(4))
        (P / (1 + Q.abs())).view(rows, d_in).backward(dfx)
        close("dx", x.grad.view(rows, d_in), xx.grad, 2 ** -7)
        # The coefficients' sums cancel, so they are held to the bound of their terms: each moves by its factor times
        # the bound of dfx, a product in bf16 (tests/train_ref.py); the sums themselves are fp32's.
        _, edfx = ref.matmul(*gk.grkan_fp8_quantize(dy.view(rows, d_out)),
                             *gk.grkan_fp8_quantize(W.detach(), "columns", tile=True), True)
        v, D = xd.view(rows, groups, -1), (1 + Q.abs()).detach()
        edfx, P, d = edfx.view(v.shape), P.detach(), dfx.view(v.shape).abs()
        for name, got, want, factors in (("dA", A.grad, Ad.grad, [v ** i / D for i in range(6)]),
                                         ("dB", B.grad, Bd.grad, [P * v ** j / D ** 2 for j in range(1, 5)])):
            bound = torch.stack([((edfx + ref.SUM * d) * t.abs()).sum((0, 2)) for t in factors], 1)
            ref.check(name, got, want, bound)


def test_linear_asks_for_what_is_needed(gk):
    x, W = normal((40, 64), 51, 1.0, BF), normal((32, 64), 52, 1.0, BF)
    for rx, rw in ((True, False), (False, True), (False, False)):
        xx, ww = x.clone().requires_grad_(rx), W.clone().requires_grad_(rw)
        y = gk.GRKANFp8Linear.apply(xx, ww)
        if rx or rw:
            y.backward(torch.ones_like(y))
        assert (xx.grad is not None) == rx and (ww.grad is not None) == rw


def test_streams_and_graphs(gk):
    """On another stream, and captured once and replayed with new inputs: the eager results' bits."""
    x, W = normal((197, 256), 61, 1.0, BF), normal((384, 256), 62, 0.06, BF)
    wq, ws = gk.grkan_fp8_quantize(W, tile=True)

    def call(stream=None):
        q, s, qt, st = gk.grkan_fp8_quantize(x, "both", stream=stream)
        return [gk.grkan_fp8_matmul(q, s, wq, ws, stream=stream),
                gk.grkan_fp8_matmul(qt, st, qt, st, dtype=torch.float32, stream=stream)]

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in (63, 64, 65):
        x.copy_(normal((197, 256), seed, 1.0, BF))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(call(), out):
            assert torch.equal(a, b)


@pytest.mark.parametrize("act", ("none", "rational"))
def test_linear_of_no_rows(gk, act):
    x = normal((0, 7, 64), 71, 1.0, BF).requires_grad_()
    W = normal((32, 64), 72, 1.0, BF).requires_grad_()
    b = normal((32,), 73).requires_grad_()
    A, B = (normal((8, k), 74).requires_grad_() if act == "rational" else None for k in (6, 4))
    y = gk.GRKANFp8Linear.apply(x, W, b, act, A, B)
    assert y.shape == (0, 7, 32)
    y.backward(torch.empty_like(y))
    for t in (x, W, b, A, B):
        assert t is None or (t.grad.shape == t.shape and not t.grad.count_nonzero())


@pytest.mark.parametrize("d_in, d_out, groups", ((128, 40, 8), (37, 45, 37)))
def test_linear_of_strided_rows(gk, d_in, d_out, groups):
    """Rows that are parts of longer ones, and W a part of a larger one, give what dense copies give."""
    wide, Wide = normal((70, d_in + 64), 75, 1.0, BF), normal((d_out, d_in + 32), 76, 0.1, BF)
    A, B, b = normal((groups, 6), 77, 0.5), normal((groups, 4), 78, 0.5), normal((d_out,), 79)
    dy = normal((70, d_out), 80, 0.1, BF)
    got = []
    for dense in (False, True):
        x, W = wide[:, 64:], Wide[:, 16:16 + d_in]
        if dense:
            x, W = x.contiguous(), W.contiguous()
        leaves = [t.detach().requires_grad_() for t in (x, W, b, A, B)]
        y = gk.GRKANFp8Linear.apply(leaves[0], leaves[1], leaves[2], "rational", leaves[3], leaves[4], groups)
        got.append([y, *torch.autograd.grad(y, leaves, dy.t().contiguous().t() if not dense else dy)])
    for one, two in zip(*got):
        assert torch.equal(one, two)


def test_far_rows(gk):
    """Offsets past 2^32 bytes and elements: the last rows as if they were alone."""
    rows, k, n, last = (1 << 20) + 300, 4096, 4096, 300
    x = torch.empty((rows, k), dtype=BF, device=DEV)
    x[:-last] = 1.0
    x[-last:] = normal((last, k), 81, 1.0, BF)
    q, s, qt, st = gk.grkan_fp8_quantize(x, "both")
    del x
    tail = normal((last, k), 81, 1.0, BF)
    want = gk.grkan_fp8_quantize(tail, "both")
    assert torch.equal(q[-last:].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s[-last:], want[1])
    # (the tail begins at a block of rows)
    assert torch.equal(qt[:, -last:].view(torch.uint8), want[2].view(torch.uint8)) and torch.equal(st[:, -3:], want[3])
    del qt, st
    b, sb = gk.grkan_fp8_quantize(normal((n, k), 82, k ** -0.5, BF), tile=True)
    c = gk.grkan_fp8_matmul(q, s, b, sb)
    got, bound = ref.matmul(want[0], want[1], b, sb, True)
    ref.check("tail", c[-last:], got, bound)
    one = gk.grkan_fp8_matmul(q[:300], s[:300], b, sb)
    assert float((c[:300].double() - one.double()).abs().max()) <= 2.0 ** -7 * float(one.double().abs().max())
