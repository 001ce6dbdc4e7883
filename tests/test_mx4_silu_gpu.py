"""The gate of the 4-bit products to the last digits, on the GPU: products of one
column each, so that the gate and up values are exact."""
import numpy as np
import pytest
import torch

import block_ref as ref
from expert_routed_ffn_gemm_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def codes_of(nibbles, exponents):
    """Rows of 32 columns, zero but for column 0: codes and scale bytes."""
    codes = np.zeros((len(nibbles), 16), np.uint8)
    codes[:, 0] = nibbles
    scales = np.zeros((len(nibbles), 4), np.uint8)
    scales[:, 0] = np.asarray(exponents) + 127
    return codes, scales


@pytest.mark.parametrize("rows", [3, 40, 100, 130, 700])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_gates_from_closed_to_open(rows, dtype):
    """Every E2M1 value, either sign, times 2^-9 .. 2^4: gates up to 96, beside up values up to 1.5 x 2^30 (fp16: 2^9).

    fp32: the exponential is off by a step (two half steps of 2^-24), its sum, reciprocal and three products by a half
    step each: 7; where it is subnormal by 2^-149, and its product by half of that.  16 bits: 2 + |gate| steps of 2^-22, three products, the
    result's rounding, and nothing left of a sigmoid under 2^-126."""
    nib = np.tile(np.arange(16), 14)
    exp = np.repeat(np.arange(-9, 5), 16)
    F = len(nib)
    rng = np.random.default_rng(rows)
    up_exp = rng.integers(-6, 9 if dtype == torch.float16 else 31, F)
    gc, gs = codes_of(nib, exp)
    uc, us = codes_of(rng.permutation(np.where(np.arange(F) % 2, 3, 10)), up_exp)  # 1.5 and -1
    w = np.concatenate([gc, uc])[None], np.concatenate([gs, us])[None]
    experts = binding.Mx4Experts(*[torch.from_numpy(a).to(DEV) for a in w], 32, gated=True)
    xc, xs = codes_of(np.where(np.arange(rows) % 3 == 1, 10, 2), np.zeros(rows, int))  # 1 and -1
    got = experts.matmul(torch.from_numpy(xc).to(DEV), torch.from_numpy(xs).to(DEV),
                         torch.tensor([0, rows], dtype=torch.int32, device=DEV), dtype=dtype)
    assert experts.check() == binding.MOE_OK
    x = ref.values_of(xc, xs, 32)[:, :1]
    z = ref.values_of(*w, 32)[0, :, 0]
    gate, up = x * z[:F], x * z[F:]
    want = torch.from_numpy(gate / (1 + np.exp(-gate)) * up)
    g, u = torch.from_numpy(np.abs(gate)), torch.from_numpy(np.abs(up))
    if dtype == torch.float32:
        tol = 7 * ref.U * want.abs() * (1 + 2.0 ** -20) + 2.0 ** -148 * g * u + 2.0 ** -149
    else:
        tol = (4 * (2 + g) + 3) * ref.U * want.abs() + torch.where(torch.from_numpy(gate) < -87, want.abs(), 0.0)
        tol = tol + ref.half_step(dtype) * (want.abs() + tol) + torch.finfo(dtype).tiny
    off = (got.cpu().double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (int(bad.sum()), gate[bad.numpy()][:6], up[bad.numpy()][:6], got.cpu()[bad][:6], want[bad][:6])
