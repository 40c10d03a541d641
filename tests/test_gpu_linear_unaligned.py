"""GPU tests of the linear map's forward on operands off 16-byte boundaries where its plan, and with it the
workspace it takes, differs from that of aligned operands."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def gk():
    import gr_kan_rational_amd as g

    g.load_library()
    return g


# more k splits than aligned operands would get: 3 against 2, 2 against 1, and 3 against 2 by address alone
@pytest.mark.parametrize("rows, d_in, d_out, offset", [(130, 2265, 24786, 0), (1003, 6203, 12387, 0),
                                                       (130, 1688, 24608, 1)])
def test_workspace_is_enough(gk, rows, d_in, d_out, offset):
    """The call with a workspace of its own making, and with one of exactly the advertised bytes."""
    from gr_kan_rational_amd import block

    print(f"[linear, unaligned] {rows} x {d_in} -> {d_out} at {offset}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(70)
    wide = torch.randn((rows, d_in + 8 * offset), generator=gen, device=DEV).to(BF)
    x = wide[:, offset:offset + d_in]
    W = (torch.randn((d_out, d_in), generator=gen, device=DEV) * d_in ** -0.5).to(BF)
    want = ref.linear_forward(x, W, None, "silu")["z"]
    z = gk.grkan_linear_act_forward(x, W, act="silu")[0]
    ref.check("z", z, *want)
    need = block._library().grkan_linear_act_forward_workspace_size(rows, d_in, d_out, 1, block.GRKAN_ACT_SILU)
    guard = torch.full((need + 4096,), 7, dtype=torch.uint8, device=DEV)
    z2 = gk.grkan_linear_act_forward(x, W, act="silu", workspace=guard[:need])[0]
    assert torch.equal(z, z2) and bool((guard[need:] == 7).all())
