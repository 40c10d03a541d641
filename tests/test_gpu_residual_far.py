"""GPU test of the residual path's backward with more gate values than a launch has threads."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


def test_more_gates_than_threads():
    """2^23 rows of 1,024 channels with a gate for each two rows, 2^32 gate values: rows that repeat each 4,096 give
    gradients that repeat, those of 4,096 rows alone (two rows of a gate are added by one wave in both)."""
    import gr_kan_rational_amd as gk

    gk.load_library()
    rows, few, c = 1 << 23, 1 << 12, 1024
    gen = torch.Generator(device=DEV).manual_seed(1)
    part = torch.randn((few // 2, 2, c), generator=gen, device=DEV).to(BF)
    gates = torch.randn((few // 2, 1, c), generator=gen, device=DEV).to(BF)
    skip = ("dx", "df", "dscale", "dweight")

    def grad(times):
        v, gate = part.repeat(times, 1, 1), gates.repeat(times, 1, 1)
        stats = torch.ones((2, few * times), device=DEV)
        stats[0] = 0.0
        return gk.grkan_residual_norm_backward(v, v, None, v, stats, "rms", gate=gate, skip=skip)[3]

    want, got = grad(1), grad(rows // few)
    assert want.count_nonzero() > want.numel() // 2
    got = got.view(rows // few, *want.shape)
    for at in range(0, rows // few, 64):   # (a comparison of all at once takes as much memory again)
        assert torch.equal(got[at:at + 64], want.expand(64, *want.shape)), f"from part {at} on"
