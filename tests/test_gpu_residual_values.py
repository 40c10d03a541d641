"""GPU tests of what NaN and infinities do in the residual path."""
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


@pytest.mark.parametrize("c", (96, 1030, 5000))
@pytest.mark.parametrize("dtype", (torch.float32, BF))
@pytest.mark.parametrize("norm", ("layer", "rms"))
def test_h_and_z_of_a_row_that_is_not_finite(gk, norm, dtype, c):
    """Without a post norm h is its formula channel by channel: what the same call gives for finite rows, but at the
    NaN or infinity itself.  z: NaN throughout, 0 beside an infinity of an rms norm; other rows as they were."""
    gen = torch.Generator(device=DEV).manual_seed(c)
    x, f = (torch.randn((7, c), generator=gen, device=DEV).to(dtype) for _ in range(2))
    scale, weight = (torch.rand(c, generator=gen, device=DEV) + 0.5 for _ in range(2))
    gate = torch.rand((7, 1), generator=gen, device=DEV) + 0.5
    h0, z0, stats0 = gk.grkan_residual_norm_forward(x, f, norm, weight, scale=scale, gate=gate)
    x[1, 5], f[2, c - 1], f[3, 0], x[5, 7] = torch.nan, torch.nan, torch.inf, -torch.inf
    h, z, stats = gk.grkan_residual_norm_forward(x, f, norm, weight, scale=scale, gate=gate)
    at = torch.zeros((7, c), dtype=torch.bool, device=DEV)
    at[1, 5] = at[2, c - 1] = at[3, 0] = at[5, 7] = True
    assert torch.equal(h[~at], h0[~at])
    assert h[1, 5].isnan() and h[2, c - 1].isnan() and float(h[3, 0]) == torch.inf and float(h[5, 7]) == -torch.inf
    good = [0, 4, 6]
    assert torch.equal(z[good], z0[good]) and torch.equal(stats[:, good], stats0[:, good])
    assert z[1:3].isnan().all()
    if norm == "layer":
        assert z[[3, 5]].isnan().all()
    else:
        assert z[3, 0].isnan() and not z[3, 1:].any() and z[5, 7].isnan() and z[5].count_nonzero() == 1
        assert not stats[1, [3, 5]].any()


def test_h_behind_a_post_norm(gk):
    """Statistics that become NaN reach every channel of the row; an infinity of an rms norm leaves f's other channels
    zero."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, f = (torch.randn((4, 200), generator=gen, device=DEV) for _ in range(2))
    f[1, 5], f[2, 9] = torch.nan, torch.inf
    h = gk.grkan_residual_norm_forward(x, f, "rms", post="layer")[0]
    assert h[1:3].isnan().all() and h[[0, 3]].isfinite().all()
    h = gk.grkan_residual_norm_forward(x, f, "rms", post="rms")[0]
    rest = torch.arange(200, device=DEV) != 9
    assert h[1].isnan().all() and h[2, 9].isnan() and torch.equal(h[2, rest], x[2, rest])
