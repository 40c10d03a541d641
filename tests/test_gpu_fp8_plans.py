"""GPU tests of the 8-bit product in every way that it is laid out (tests/product_cases.py), against fp64: bias and
residual, apart and in place, odd sizes throughout."""
import pytest
import torch

import product_cases as cases
import train_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16
F8 = torch.float8_e4m3fn
KINDS = {"f32": (torch.float32, "fp32"), "sums": (BF, "fp32"), "cut": (BF, "fast")}


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


def codes(gen, rows, k, tile):
    """Random codes over 9 binades, NaN past the end of each row, and scales in [0.5, 1.5)."""
    held = ref.ceil(k, 16) * 16
    q = torch.full((rows, held), 0x7F, dtype=torch.uint8, device=DEV)
    q[:, :k] = torch.randint(16, 88, (rows, k), generator=gen, device=DEV, dtype=torch.uint8)
    q[:, :k] += torch.randint(0, 2, (rows, k), generator=gen, device=DEV, dtype=torch.uint8) * 128
    s = torch.rand((ref.ceil(rows, 128) if tile else rows, ref.ceil(k, 128)), generator=gen, device=DEV) + 0.5
    return q.view(F8)[:, :k], s


def expected(a, sa, b, sb, tile, bias, residual, kind):
    """(value, bound): fp32 sums' bound, of a bf16 result its rounding besides; cut sums' as they stand in train_ref."""
    if kind == "cut":
        return ref.matmul(a, sa, b, sb, tile, bias, residual, BF)
    v, err = ref.matmul(a, sa, b, sb, tile, bias, residual, torch.float32)
    return v, err if kind == "f32" else err + ref.rounding(v.abs() + err, BF)


def check(gk, shape, kind, tile):
    print(f"[product] {shape} {kind} {tile}", flush=True)
    m, n, k = shape
    dtype, sums = KINDS[kind]
    gen = torch.Generator(device=DEV).manual_seed(sum(shape))
    (a, sa), (b, sb) = codes(gen, m, k, False), codes(gen, n, k, tile)
    bias = torch.randn(n, generator=gen, device=DEV)
    r = (torch.randn((m, n), generator=gen, device=DEV) * 3).to(dtype)
    got = gk.grkan_fp8_matmul(a, sa, b, sb, bias=bias, residual=r, dtype=dtype, sums=sums)
    # (of many rows the first and last and every 37th: some of each tile and of each lane's)
    at = torch.arange(m, device=DEV)
    at = at[(at < 200) | (at >= m - 200) | (at % 37 == 0)]
    ref.check(f"{shape}", got[at], *expected(a.view(torch.uint8)[at].view(F8), sa[at], b, sb, tile, bias, r[at], kind))
    gk.grkan_fp8_matmul(a, sa, b, sb, bias=bias, residual=r, dtype=dtype, sums=sums, out=r)
    assert torch.equal(got, r), "in place"


@pytest.mark.parametrize("tile", (True, False))
@pytest.mark.parametrize("kind", tuple(KINDS))
@pytest.mark.parametrize("shape", cases.EVERY, ids=str)
def test_every_plan(gk, shape, kind, tile):
    check(gk, shape, kind, tile)


@pytest.mark.parametrize("shape", cases.CUT_TILES, ids=str)
def test_every_plan_of_cut_tiles(gk, shape):
    check(gk, shape, "cut", True)
