"""GPU test of the quantiser on many rows of few columns."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.mark.parametrize("outputs", ("rows", "both"))
def test_many_rows(outputs):
    """2^28 + 4,099 rows of 16: rows that repeat each 4,096 (and a part of them) give the codes of 4,096 alone."""
    import gr_kan_rational_amd as gk

    gk.load_library()
    few, times, rest, cols = 1 << 12, 1 << 16, (1 << 12) + 3, 16
    part = torch.randn((few, cols), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(BF)
    rows = few * times + rest
    x = torch.empty((rows, cols), dtype=BF, device=DEV)
    x[:few * times].view(times, few, cols).copy_(part)
    x[few * times:few * (times + 1)], x[few * (times + 1):] = part, part[:rest - few]
    want = gk.grkan_fp8_quantize(part, outputs)
    got = gk.grkan_fp8_quantize(x, outputs)

    def whole(t):
        return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t

    for w, g in zip(want[:2], got[:2]):
        w, g = whole(w), whole(g)
        assert torch.equal(g[few * times:few * (times + 1)], w) and torch.equal(g[few * (times + 1):], w[:rest - few])
        g = g[:few * times].unflatten(0, (times, few))
        assert all(torch.equal(g[at], w) for at in range(0, times, 4099)) and torch.equal(g[-1], w)
        assert (g.sum((1, 2), dtype=torch.float64) == w.sum(dtype=torch.float64)).all()
    if outputs == "both":   # (the last rows are no whole block of their columns)
        for w, g, block in ((want[2], got[2], few), (want[3], got[3], few // 128)):
            w, g = whole(w), whole(g)
            for at in (0, 1, times // 2, times):
                assert torch.equal(g[:, at * block:(at + 1) * block], w)
