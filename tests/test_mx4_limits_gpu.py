"""The 4-bit products at the edges of what the header allows, on the GPU."""
import numpy as np
import pytest
import torch

from expert_routed_ffn_gemm_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_more_tiles_than_are_numbered():
    """One group of 2^27 rows, all but one dropped by out_rows, times 2^20 weight rows: refused, not left undone.  Where
    overlapping groups make as many tiles the call's check says so, and the handle works on."""
    rows, n = 1 << 27, 1 << 20
    experts = binding.Mx4Experts(torch.zeros((1, n, 16), dtype=torch.uint8, device=DEV),
                                 torch.zeros((1, n, 4), dtype=torch.uint8, device=DEV), 32)
    codes = torch.zeros((rows, 16), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((rows, 4), dtype=torch.uint8, device=DEV)
    out_rows = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    out_rows[5] = 0
    out = torch.full((1, n), 7.0, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(binding.MoeError) as e:
        experts.matmul(codes, scales, torch.tensor([0, rows], dtype=torch.int32, device=DEV), out_rows=out_rows, n_out=1,
                       out=out)
    assert e.value.status == binding.MOE_ERR_UNSUPPORTED
    experts.close()

    groups, few = 65, 4_000_000  # 33 groups of all rows each: 33 x 16667 x 4096 tiles
    experts = binding.Mx4Experts(torch.zeros((groups, n, 16), dtype=torch.uint8, device=DEV),
                                 torch.zeros((groups, n, 4), dtype=torch.uint8, device=DEV), 32)
    offsets = torch.from_numpy(np.where(np.arange(groups + 1) % 2, few, 0).astype(np.int32)).to(DEV)
    experts.matmul(codes[:few], scales[:few], offsets, out_rows=out_rows[:few], n_out=1, out=out)
    assert experts.check() == binding.MOE_ERR_DEVICE and bool((out == 7).all())
    one = torch.zeros(groups + 1, dtype=torch.int32, device=DEV)
    one[1:] = 6
    experts.matmul(codes[:6], scales[:6], one, out_rows=out_rows[:6], n_out=1, out=out)
    assert experts.check() == binding.MOE_OK and not out.any()
