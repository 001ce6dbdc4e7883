"""Norm gradients over more rows than the blocks' rings have stages, for every kind of gate, on the GPU."""
import pytest
import torch

from test_norm_residual_gpu import check_backward_against, inputs, run_backward

pytestmark = pytest.mark.gpu


# at least four rows to each of the blocks (152 SMs: 608 blocks of four rows, 1216 of one, 152 of one)
@pytest.mark.parametrize("T,d", [(10001, 40), (5003, 264), (701, 4096), (640, 2056)])
@pytest.mark.parametrize("gate,sigmoid,gate_dtype", [("full", True, None), ("full", True, torch.float32),
                                                     ("full", False, None), ("token", True, None), ("feature", True, None),
                                                     ("none", False, None)])
@pytest.mark.parametrize("stream,block", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16),
                                          (torch.float32, torch.float32)])
def test_many_rows_to_a_block(T, d, gate, sigmoid, gate_dtype, stream, block):
    t = inputs(T, d, 1, gate, stream, block, gate_dtype=gate_dtype, seed=d)
    grads = run_backward(t, 0.7, 1e-6, sigmoid)
    check_backward_against(t, grads, 0.7, 1e-6, sigmoid)
    again = run_backward(t, 0.7, 1e-6, sigmoid)
    assert all(torch.equal(grads[k], again[k]) for k in grads)
