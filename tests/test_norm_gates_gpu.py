"""Sigmoid gates far open, far closed and past that, on the GPU: their gradients keep their
digits where g is close to 1 and g (1 - g) is all that is left of it."""
import pytest
import torch

import block_ref as ref
from expert_routed_ffn_gemm_gb300 import binding
from test_norm_residual_gpu import STEPS, check, formula, inputs, made_of, run_backward

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
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


@pytest.mark.parametrize("block", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", ["feature", "token", "full", "full32"])
def test_fp32_results_to_the_last_digits(gate, block):
    """One factor each and no norms, so that nothing but the gate is rounded: out = g z, dy = g D, dg = z D g (1 - g).

    The exponential is off by a step (two half steps of 2^-24), 1 + e by a half step, its reciprocal by a step, the
    smaller of g and 1 - g a product more: 6; with two products out and dy by 8; g (1 - g) one rounding more, and two
    products: 9, in half steps."""
    T, d = {"feature": (1, 4096), "token": (4096, 1), "full": (8, 1024), "full32": (8, 1024)}[gate]
    gen = torch.Generator().manual_seed(5)
    z = torch.randn((T, d), generator=gen).to(block)
    D = torch.randn((T, d), generator=gen)
    x = torch.rand({"feature": (d,), "token": (T, 1), "full": (T, d), "full32": (T, d)}[gate],
                   generator=gen) * 160 - 80
    if gate == "full":  # of the block's type, and its gradient too
        x = x.to(block)
    t = {k: v.to(DEV) for k, v in {"z": z, "D": D, "x": x}.items()}
    out, _ = binding.moe_norm_residual(torch.zeros_like(t["D"]), t["z"], gate=t["x"], sigmoid=True)
    grads = binding.moe_norm_residual_backward(t["D"], None, out, t["z"], gate=t["x"], sigmoid=True)
    zd, Dd, xd = z.double(), D.double(), x.double()
    g, slope = torch.sigmoid(xd), torch.sigmoid(xd) * torch.sigmoid(-xd)

    def close(got, want, steps, dtype=torch.float32):
        tol = steps * ref.U * want.abs() * (1 + 2.0 ** -20) + 2.0 ** -149
        if dtype != torch.float32:
            tol = tol + 3 * 4 * (2 + xd.abs()) * ref.U * want.abs() + ref.half_step(dtype) * want.abs() * 1.01
        assert got.dtype == dtype and bool(((got.cpu().double() - want).abs() <= tol).all())

    if gate == "full" and block != torch.float32:
        close(out, g * zd, 8)
        close(grads["gate"], zd * Dd * slope, 9, block)
        return
    close(out, g * zd, 8)
    close(grads["gate"].view(slope.shape), zd * Dd * slope if gate != "feature" else (zd * Dd)[0] * slope, 9)
    close(grads["y"], g * Dd, 8, block)
