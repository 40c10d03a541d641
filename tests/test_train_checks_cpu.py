"""CPU checks of the operators of include/grkan_train.h, beside tests/test_train_cpu.py: what the library and the binding
refuse, and what the binding does around a call."""
import pytest
import torch

from gr_kan_rational_amd import train
from test_train_cpu import F32, INVALID, lib, matmul  # noqa: F401


def test_kind_of_sums(lib):  # noqa: F811
    """One of two names; in the C ABI a flag beside b_tile, which does not hide other values of it."""
    assert open(__file__.replace("tests/test_train_checks_cpu.py", "include/grkan_train.h")).read().count(
        f"#define GRKAN_FP8_SUMS_F32 {train.GRKAN_FP8_SUMS_F32}\n") == 1
    for tile in (18, 19, 15, 32, -1, -16):
        assert matmul(lib, tile=tile) == INVALID
    assert matmul(lib, tile=17, c=None) == INVALID and matmul(lib, tile=16, m=0, a=None, sa=None, c=None, out=F32) == 0
    f8, s = torch.zeros(4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.ones(4, 1)
    with pytest.raises(ValueError, match="sums"):
        train.grkan_fp8_matmul(f8, s, f8, s, sums="fp16")
    from gr_kan_rational_amd.mixer import GRKANStack

    with pytest.raises(ValueError, match="sums"):
        GRKANStack(1, 16, 16, products="fp8", sums="bf16")
