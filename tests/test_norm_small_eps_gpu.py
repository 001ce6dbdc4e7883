"""Gradients of norms of rows of nothing, or almost nothing, where eps is small:
1 / sqrt(eps) is a number, its cube need not be one in fp32."""
import pytest
import torch

from expert_routed_ffn_gemm_gb300 import binding
from test_norm_residual_gpu import check_backward_against, dev, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [2.0 ** -40, 2.0 ** -100, 2.0 ** -140])
@pytest.mark.parametrize("d", [33, 64, 4100, 5120])
@pytest.mark.parametrize("gate", ["none", "token", "full"])
def test_rows_of_almost_nothing(gate, d, eps):
    """A stream of zeros, a small one, terms of zeros, small ones, and a row as others are: each apart."""
    t = inputs(5, d, 1, gate, torch.float32, torch.float32, seed=d)
    t["out"] = t.pop("x")
    t["out"][0], t["y"][2] = 0, 0
    t["out"][1] *= 2.0 ** -50
    t["y"][3] *= 2.0 ** -50
    g = dev(t)
    grads = binding.moe_norm_residual_backward(g["d_out"], g["d_n"], g["out"], g["y"], g["w_post"], g["gate"], g["w_pre"],
                                               0.5, eps, True)
    assert all(bool(torch.isfinite(v).all()) for v in grads.values())
    check_backward_against(t, grads, 0.5, eps, True)


@pytest.mark.parametrize("eps", [2.0 ** -100, 2.0 ** -140])
def test_norm_alone_of_almost_nothing(eps):
    t = inputs(3, 264, 1, "none", torch.float32, torch.float32)
    t["out"] = t.pop("x")
    t["out"][0] = 0
    t["out"][1] *= 2.0 ** -50
    g = dev(t)
    grads = binding.moe_norm_residual_backward(g["d_out"], g["d_n"], g["out"], w_pre=g["w_pre"], eps=eps)
    t["y"] = None
    check_backward_against(t, grads, 1.0, eps, False)
