"""Host logic of the block operators' C entry points over fake devices (CPU)."""
import pytest

import fake_device
from expert_routed_ffn_gemm_gb300 import binding

INVALID, UNSUPPORTED, OK = binding.MOE_ERR_INVALID_ARG, binding.MOE_ERR_UNSUPPORTED, binding.MOE_OK


@pytest.fixture(scope="module")
def lib():
    return fake_device.load()


@pytest.mark.parametrize("rows,n,status", [(1 << 27, 1 << 20, UNSUPPORTED), (1 << 30, 1 << 20, UNSUPPORTED),
                                           (120 << 20, 1 << 20, UNSUPPORTED), (119 << 20, 1 << 20, OK),
                                           (1 << 30, 1 << 16, OK)])
@pytest.mark.parametrize("gated", [0, 1])
def test_products_of_more_than_2_31_tiles_are_refused(lib, rows, n, status, gated):
    """Work items are numbered in 32 bits: 240 token rows by 256 weight rows each at these sizes.  One group of 2^27
    rows has 559,241 x 4096 of them."""
    h = fake_device.experts(lib, 1, n, 32, gated)
    p = fake_device.address(0)
    before = fake_device.value(lib, "fake_launches")
    assert lib.moe_mx4_matmul(h, p, p, rows, p, p, None, p, 0, 1, None) == status
    assert fake_device.value(lib, "fake_launches") == before + (status == OK)
    lib.moe_mx4_free(h)
