"""GPU tests of the group norm's statistics where a few positions are far larger than the others, as a
sequence's first token often is."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


@pytest.mark.parametrize("size", (1e2, 1e4, 1e6))
@pytest.mark.parametrize("shape, groups", [((1, 20000, 64), 8), ((2, 5000, 36), 3), ((8, 4096, 320), 32),
                                           ((1, 65536, 128), 32), ((3, 400, 2500), 1), ((4, 60, 96), 4)], ids=str)
@pytest.mark.parametrize("io", (torch.float32, torch.bfloat16), ids=("f32", "bf16"))
def test_statistics_with_a_large_first_position(gk, shape, groups, io, size):
    """mean and rstd within the bounds of sums of any order (64 units of the sum of magnitudes)."""
    gen = torch.Generator(device=DEV).manual_seed(100)
    x = torch.randn(shape, generator=gen, device=DEV)
    x[:, 0] = size * (1 + 0.1 * x[:, 0])
    x = x.to(io)
    y, mean, rstd = gk.grkan_group_norm_forward(x, groups)
    one = torch.ones(shape[-1], device=DEV)
    want = ref.norm_forward(x, groups, one, 0 * one, 1e-5, "none")
    for k, got in (("mean", mean), ("rstd", rstd), ("y", y)):
        ref.check(f"{shape} {k}", got, *want[k])
