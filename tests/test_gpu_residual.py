"""GPU tests of the residual path with its norms, forward and backward, against the definitions in fp64; the bounds
are derived in tests/train_ref.py."""
import itertools

import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
NAMES = ("dx", "df", "dscale", "dgate", "dweight", "dbias", "dpost_weight", "dpost_bias")


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


def make(shape, dtype, norm, post, gate, seed, gate_dtype=None):
    gen = torch.Generator().manual_seed(seed)
    c = shape[-1]

    def normal(size, std=1.0, mean=0.0, dt=torch.float32):
        return (torch.randn(size, generator=gen) * std + mean).to(DEV).to(dt)

    x, f = normal(shape, 1.5, 0.3, dtype), normal(shape, 1.0, 0.2, dtype)
    p = dict(norm=norm, weight=normal((c,), 0.2, 1.0), bias=normal((c,), 0.3) if norm == "layer" else None,
             scale=normal((c,), 0.3, 0.5), post=post, gate=None)
    p["post_weight"] = normal((c,), 0.2, 1.0) if post != "none" else None
    p["post_bias"] = normal((c,), 0.3) if post == "layer" else None
    if gate is not None:
        p["gate"] = normal(tuple(s if keep else 1 for s, keep in zip(shape, gate)), 0.5, 1.0, gate_dtype or dtype)
    return x, f, p, normal(shape, 1e-2, 0.0, dtype), normal(shape, 1e-2, 0.0, dtype)


def both_ways(gk, shape, dtype, norm, post, gate, seed, gate_dtype=None):
    print(f"[residual] {shape} {dtype} {norm} {post} {gate}", flush=True)
    x, f, p, dh, dz = make(shape, dtype, norm, post, gate, seed, gate_dtype)
    order = [p[k] for k in ("norm", "weight", "bias", "scale", "gate", "post", "post_weight", "post_bias")]
    h, z, stats = gk.grkan_residual_norm_forward(x, f, **p)
    want = ref.residual_forward(x, f, *order)
    for name, got in (("h", h), ("z", z), ("stats", stats)):
        ref.check(f"{name}", got, *want[name])
    for a, b in zip((h, z, stats), gk.grkan_residual_norm_forward(x, f, **p)):
        assert torch.equal(a, b), "two calls differ"
    got = gk.grkan_residual_norm_backward(f, h, dh, dz, stats, **p)
    want = ref.residual_backward(f, h, dh, dz, stats, *order)
    for name, t in zip(NAMES, got):
        if t is not None:
            ref.check(name, t, *want[name])
        else:
            assert name not in want
    for a, b in zip(got, gk.grkan_residual_norm_backward(f, h, dh, dz, stats, **p)):
        assert a is None or torch.equal(a, b), "two calls differ"
    return (x, f, p, dh, dz), (h, z, stats), got


NONE, SAMPLE, TOKEN, CHANNEL, ELEMENT = None, (1, 0, 0), (1, 1, 0), (1, 0, 1), (1, 1, 1)


@pytest.mark.parametrize("dtype", (torch.float32, BF))
@pytest.mark.parametrize("gate", (NONE, SAMPLE, TOKEN, CHANNEL, ELEMENT), ids=str)
@pytest.mark.parametrize("norm, post", list(itertools.product(("layer", "rms"), ("none", "layer", "rms"))))
def test_kinds(gk, norm, post, gate, dtype):
    both_ways(gk, (5, 13, 96), dtype, norm, post, gate, 1)


# one token, one channel, odd widths, each number of accesses and waves a row, few long and many short samples
SHAPES = [(1, 1, 768), (1, 1, 1), (3, 2, 1), (2, 3, 5), (4, 7, 37), (2, 50, 256), (3, 30, 257), (3, 11, 777), (2, 9, 1024),
          (2, 5, 1028), (3, 4, 2050), (2, 4, 3000), (2, 3, 4096), (2, 3, 4100), (1, 3, 8192), (1, 2, 8193), (1, 2, 16384),
          (1, 700, 64), (300, 2, 64), (40, 197, 192), (2, 3000, 40)]


@pytest.mark.parametrize("gate", (SAMPLE, CHANNEL), ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(gk, shape, gate):
    both_ways(gk, shape, BF, "layer", "rms", gate, 2)
    both_ways(gk, shape, torch.float32, "rms", "none", gate, 3)


@pytest.mark.parametrize("gate", (SAMPLE, TOKEN, CHANNEL, ELEMENT), ids=str)
def test_float32_gates_of_bf16_rows(gk, gate):
    both_ways(gk, (4, 9, 100), BF, "rms", "layer", gate, 4, torch.float32)


def test_four_dimensions(gk):
    both_ways(gk, (2, 3, 5, 64), torch.float32, "layer", "none", (1, 1, 0, 1), 5)


def test_optional_arguments(gk):
    """Each vector absent, one of the two gradients absent, gradients left out."""
    x, f, p, dh, dz = make((3, 7, 64), torch.float32, "layer", "layer", CHANNEL, 6)
    for gone in ("weight", "bias", "scale", "post_weight", "post_bias", "gate"):
        q = dict(p, **{gone: None})
        order = [q[k] for k in ("norm", "weight", "bias", "scale", "gate", "post", "post_weight", "post_bias")]
        h, z, stats = gk.grkan_residual_norm_forward(x, f, **q)
        want = ref.residual_forward(x, f, *order)
        for name, got in (("h", h), ("z", z), ("stats", stats)):
            ref.check(name, got, *want[name])
        for a, b in ((dh, dz), (None, dz), (dh, None)):
            want = ref.residual_backward(f, h, a, b, stats, *order)
            for name, got in zip(NAMES, gk.grkan_residual_norm_backward(f, h, a, b, stats, **q)):
                if name in want:
                    ref.check(f"{name} without {gone}", got, *want[name])
    every = gk.grkan_residual_norm_backward(f, h, dh, dz, stats, **dict(p, gate=None))
    for name in NAMES:
        got = gk.grkan_residual_norm_backward(f, h, dh, dz, stats, **dict(p, gate=None), skip=(name,))
        for k, a, b in zip(NAMES, every, got):
            assert b is None if k == name else (a is None or torch.equal(a, b))


def test_layouts(gk):
    """Rows of wider tensors, odd offsets, outputs off their boundary, in place: the dense tensors' values."""
    (x, f, p, dh, dz), (h, z, stats), grads = both_ways(gk, (4, 6, 96), BF, "layer", "rms", CHANNEL, 7)

    def wide(t, left):
        w = torch.full((*t.shape[:-1], left + t.shape[-1] + 5), 3.0, dtype=t.dtype, device=DEV)
        w[..., left:left + t.shape[-1]] = t
        return w[..., left:left + t.shape[-1]]

    order = [p[k] for k in ("norm", "weight", "bias", "scale", "gate", "post", "post_weight", "post_bias")]
    want, grad = ref.residual_forward(x, f, *order), ref.residual_backward(f, h, dh, dz, stats, *order)
    for left in (3, 4):
        got = gk.grkan_residual_norm_forward(wide(x, left), wide(f, left), **p)
        for name, t in zip(("h", "z", "stats"), got):
            ref.check(name, t, *want[name])
        got = gk.grkan_residual_norm_backward(wide(f, left), h, wide(dh, left), wide(dz, left), stats, **p)
        for name, t in zip(NAMES, got):
            if t is not None:
                ref.check(name, t, *grad[name])
    x2 = x.clone()
    h2, z2, _ = gk.grkan_residual_norm_forward(x2, f, out=x2, **p)
    assert h2.data_ptr() == x2.data_ptr() and torch.equal(h2, h) and torch.equal(z2, z)
    a, b = dh.clone(), dz.clone()
    got = gk.grkan_residual_norm_backward(f, h, a, b, stats, dx=a, df=b, **p)
    for u, v in zip(grads, got):
        assert u is None or torch.equal(u, v)
    buf = torch.full((x.numel() + 2,), 7.0, dtype=BF, device=DEV)
    zo = buf[1:-1].view(x.shape)
    ref.check("z", gk.grkan_residual_norm_forward(x, f, normed=zo, **p)[1], *want["z"])
    assert float(buf[0]) == 7.0 and float(buf[-1]) == 7.0


def test_nan_stays_in_its_row(gk):
    x, f, p, dh, dz = make((3, 5, 96), torch.float32, "layer", "rms", SAMPLE, 8)
    x[1, 2, 7], f[2, 0, 3] = torch.nan, torch.inf
    h, z, stats = gk.grkan_residual_norm_forward(x, f, **p)
    bad = torch.zeros((3, 5), dtype=torch.bool, device=DEV)
    bad[1, 2] = bad[2, 0] = True
    assert z[bad].isnan().all() and z[~bad].isfinite().all() and h[~bad].isfinite().all()


def test_no_rows(gk):
    x, f, p, dh, dz = make((0, 4, 32), BF, "layer", "layer", None, 9)
    h, z, stats = gk.grkan_residual_norm_forward(x, f, **p)
    assert h.shape == x.shape and stats.shape == (4, 0)
    for name, t in zip(NAMES, gk.grkan_residual_norm_backward(f, h, dh, dz, stats, **p)):
        assert t is None or t.numel() == 0 or not t.any(), name


def test_far_rows(gk):
    """Rows whose offsets pass 2^32 bytes: the last rows' values, and the sums over all."""
    rows, c = (1 << 32) // 2048 + 77, 1024
    x, f = (torch.zeros((rows, c), dtype=BF, device=DEV) for _ in range(2))
    x[-3:], f[-3:] = 1.0, torch.arange(c, device=DEV).to(BF) / 512
    h, z, stats = gk.grkan_residual_norm_forward(x, f, norm="rms")
    want = ref.residual_forward(x[-3:], f[-3:], "rms", None, None, None, None, "none", None, None)
    ref.check("z", z[-3:], *want["z"])
    assert not z[:100].any()
    dz = torch.zeros_like(x)
    dz[-3:] = 0.5
    got = gk.grkan_residual_norm_backward(f, h, None, dz, stats, norm="rms")
    want = ref.residual_backward(f[-3:], h[-3:], None, dz[-3:], stats[:, -3:], "rms", None, None, None, None, "none", None,
                                 None)
    ref.check("dx", got[0][-3:], *want["dx"])
    ref.check("dweight", got[4], *want["dweight"])


def test_autograd(gk):
    """The function's gradients are the backward's; a captured forward and backward replays them."""
    x, f, p, dh, dz = make((4, 10, 128), BF, "layer", "rms", CHANNEL, 10)
    names = ("weight", "bias", "scale", "gate", "post_weight")
    leaves = [t.requires_grad_() for t in (x, f, *(p[k] for k in names))]
    args = (p["norm"], p["weight"], p["bias"], p["scale"], p["gate"], p["post"], p["post_weight"], None)
    p["post_bias"] = None

    def run():
        h, z = gk.GRKANResidualNorm.apply(x, f, *args)
        return torch.autograd.grad((h, z), leaves, (dh, dz))

    got = run()
    plain = {k: v.detach() if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    h, z, stats = gk.grkan_residual_norm_forward(x.detach(), f.detach(), **plain)
    want = dict(zip(NAMES, gk.grkan_residual_norm_backward(f.detach(), h, dh, dz, stats, **plain)))
    for name, t in zip(("dx", "df", "dweight", "dbias", "dscale", "dgate", "dpost_weight"), got):
        assert torch.equal(t, want[name]), name
    only, = torch.autograd.grad(gk.GRKANResidualNorm.apply(x, f, *args)[1], [f], dz)  # z alone
    part = gk.grkan_residual_norm_backward(f.detach(), h, None, dz, stats, **plain)
    assert torch.equal(only, part[1])
    del got, only
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in (11, 12, 13):
        with torch.no_grad():
            new = make((4, 10, 128), BF, "layer", "rms", CHANNEL, seed)
            x.copy_(new[0]), f.copy_(new[1]), dh.copy_(new[3])
        graph.replay()
        torch.cuda.synchronize()
        h, z, stats = gk.grkan_residual_norm_forward(x.detach(), f.detach(), **plain)
        want = dict(zip(NAMES, gk.grkan_residual_norm_backward(f.detach(), h, dh, dz, stats, **plain)))
        for name, t in zip(("dx", "df", "dweight", "dbias", "dscale", "dgate", "dpost_weight"), out):
            assert torch.equal(t, want[name]), name


@pytest.mark.parametrize("dtype, gate_dtype", ((torch.float32, torch.float32), (BF, BF), (BF, torch.float32)))
def test_no_rows_of_a_gate(gk, dtype, gate_dtype):
    """A gate over no rows has a gradient of zeros, whatever lay where it is written."""
    for shape, lead in (((0, 5, 24), (1, 1)), ((3, 0, 24), (3, 1)), ((0, 24), (1,)), ((0, 5, 24), (0, 1))):
        for wide in (1, 24):
            x = torch.empty(shape, dtype=dtype, device=DEV)
            gate = torch.ones((*lead, wide), dtype=gate_dtype, device=DEV)
            stats = torch.empty((4, 0), device=DEV)
            [torch.full((128,), 7.1, device=DEV) for _ in range(200)]  # (freed: the next small tensors have their memory)
            got = gk.grkan_residual_norm_backward(x, x, x, x, stats, gate=gate, post="rms",
                                                  post_weight=torch.ones(24, device=DEV))
            for name, t in zip(NAMES, got):
                assert t is None or not t.count_nonzero(), (name, shape, lead)
            assert got[3].shape == gate.shape
