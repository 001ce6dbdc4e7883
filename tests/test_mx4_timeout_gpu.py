"""Waits of the 4-bit products that run out: the call ends, moe_mx4_check says so, and the handle works on."""
import pytest
import torch

from expert_routed_ffn_gemm_gb300 import binding
from test_mx4_gpu import dev, offsets_of, random_codes

pytestmark = pytest.mark.gpu
TRIES = 40


@pytest.mark.parametrize("counts,N,K,gated", [
    ([90, 64, 20, 96], 4096, 4096, True),   # tiles of 128 rows, whole items
    ([20] * 7, 2048, 4096, False),          # 32 rows, K ranges in parts
    ([1] * 9, 2560, 4096, True),            # 16 rows, K ranges in parts
    ([240, 200, 700], 6400, 1312, False),   # pairs of CTAs
    ([240, 200, 700], 6400, 1312, True),
])
def test_waits_that_run_out(counts, N, K, gated):
    """With a limit of a nanosecond a wait runs out as soon as it is looked at, in whichever role first.  What the call
    leaves behind (part counts, an error word) does not outlast the check."""
    wc, ws = random_codes((len(counts), N), K, 1)
    xc, xs = random_codes((sum(counts),), K, 2)
    experts = binding.Mx4Experts(dev(wc), dev(ws), K, gated=gated)
    x, s, offsets = dev(xc), dev(xs), dev(offsets_of(counts))
    want = experts.matmul(x, s, offsets, dtype=torch.float32)
    assert experts.check() == binding.MOE_OK
    seen = 0
    for _ in range(TRIES):
        experts.set_wait_limit(1)
        got = experts.matmul(x, s, offsets, dtype=torch.float32)
        status = experts.check()
        assert status in (binding.MOE_OK, binding.MOE_ERR_DEVICE)
        # a wait may end in time all the same; then the result is whole
        assert status == binding.MOE_ERR_DEVICE or torch.equal(got, want)
        seen += status == binding.MOE_ERR_DEVICE
        experts.set_wait_limit(0)
        assert torch.equal(experts.matmul(x, s, offsets, dtype=torch.float32), want)
        assert experts.check() == binding.MOE_OK
    assert seen > 0
