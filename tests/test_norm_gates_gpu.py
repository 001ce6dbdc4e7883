"""Sigmoid gates far open, far closed and past that, on the GPU: their gradients keep their
digits where g is close to 1 and g (1 - g) is all that is left of it."""
import pytest
import torch

import block_ref as ref
from expert_routed_ffn_gemm_gb300 import binding
from test_norm_residual_gpu import STEPS, check, formula, inputs, made_of, run_backward

pytestmark = pytest.mark.gpu
# open and closed alike, to where the derivative leaves fp32's normal range; exact in bf16 and fp16
GATES = torch.tensor([0.0, 1.0, -1.0, 4.0, -4.0, 8.0, -8.0, 14.0, -14.0, 17.5, -17.5, 30.0, -30.0, 80.0, -80.0, 95.0])


def far_gates(t):
    n = t["gate"].numel()
    t["gate"] = GATES.repeat(-(-n // len(GATES)))[:n].view(t["gate"].shape).to(t["gate"].dtype)
    return t


@pytest.mark.parametrize("T,d", [(17, 72), (40, 33), (3, 4100), (700, 264)])
@pytest.mark.parametrize("stream,block", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16),
                                          (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("gate", ["feature", "token", "full"])
def test_gate_gradients_of_far_gates(gate, stream, block, T, d):
    """g (1 - g) by the approximate exponential: each factor off by 2 + |gate| steps of 2^-22, four half steps of 2^-24
    apiece, beside the half steps of the rest."""
    t = far_gates(inputs(T, d, 1, gate, stream, block, seed=d))
    grads = run_backward(t, 0.5, 1e-6, True)
    # the gradient in g itself, times g (1 - g) from the two sigmoids: autograd's own g (1 - g) loses its digits, in 64
    # bits from a gate of 30 on
    g = t["gate"].double()
    slope = torch.sigmoid(g) * torch.sigmoid(-g)
    plain = {**t, "gate": torch.sigmoid(g)}
    want, mag = formula(plain, 0.5, 1e-6, False)["gate"] * slope, made_of(t, 0.5, 1e-6, True)["gate"]
    steps = STEPS * 2 + 2 * 4 * (2 + g.abs()) + (T if gate == "feature" else 0)
    dtype = t["gate"].dtype if gate == "full" else torch.float32
    check(grads["gate"].view(want.shape), want, slope * mag * steps / STEPS, dtype, gate)


@pytest.mark.parametrize("gate", ["feature", "token", "full"])
def test_gates_past_any_digit_and_no_numbers(gate):
    """Infinite gates: closed, out is x; open, out is x + v; no gradient either way.  A NaN stays in its rows and columns."""
    t = inputs(16, 16, 1, gate, torch.float32, torch.float32, pre=False)
    inf, n = float("inf"), t["gate"].numel()
    t["gate"] = torch.tensor([inf, -inf, 200.0, -200.0]).repeat(-(-n // 4))[:n].view(t["gate"].shape)
    grads = {k: v.cpu() for k, v in run_backward(t, 1.0, 1e-6, True).items()}
    assert not grads["gate"].any() and bool(torch.isfinite(grads["y"]).all())
    t["gate"].view(-1)[2] = float("nan")
    grads = {k: v.cpu() for k, v in run_backward(t, 1.0, 1e-6, True).items()}
    assert bool(torch.isnan(grads["gate"].view(-1)[2]))
    at = {"feature": (slice(None), 2), "token": (2,), "full": (0, 2)}[gate]
    assert bool(torch.isnan(grads["y"][at]).all())
