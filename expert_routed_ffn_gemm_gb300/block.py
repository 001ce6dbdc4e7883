"""A decoder block's feed-forward half around 4-bit experts: the operators of
the binding as they are used together.

    n            = norm of the residual stream (from the block before)
    route        the layer's router picks k experts per token (moe_route)
    H            = silu(n Wg) * (n Wu)  by group, rows quantised as gathered
    y[t, j]      = weight(t, j) * (H Wd) of slot j, the shared expert in the last slot
    out, n_next  = x + alpha * gate * norm(sum_j y[t, j]),  norm(out)

``python -m expert_routed_ffn_gemm_gb300.block`` runs a prompt, single tokens
and a few steps that fit the norms and the gate of a block with frozen 4-bit
experts to the same block in bf16, and prints how far the two are apart.
"""
from __future__ import annotations

import torch

from . import binding, synth


class Mx4Block:
    """4-bit experts behind a layer's router, with the norms around them.

    layer: the MoeLayer whose routing is used (it keeps its own expert weights
    beside the 4-bit ones); w_gate_up [G, 2F, d] and w_down
    [G, d, F] in bf16, fp16 or fp32 are quantised here.  w_post, gate and w_pre
    are as in moe_norm_residual, w_pre the norm of the block after this one.
    """

    def __init__(self, layer: binding.MoeLayer, w_gate_up, w_down, w_post=None, gate=None, w_pre=None,
                 alpha: float = 1.0, eps: float = 1e-6, sigmoid: bool = False):
        self.layer = layer
        self.up = binding.Mx4Experts.quantize(w_gate_up, gated=True)
        self.down = binding.Mx4Experts.quantize(w_down)
        self.slots_per_token = layer.k + int(layer.has_shared)
        self.norm = dict(w_post=w_post, gate=gate, w_pre=w_pre)
        self.options = dict(alpha=alpha, eps=eps, sigmoid=sigmoid)

    def slots(self, n: torch.Tensor):
        """(slots [R], offsets [G + 1], weights [R]) of tokens n: slot t * (k + shared) + j of every product row
        in dispatch order, and each slot's gate weight (1 for the shared expert)."""
        T, k, per = n.shape[0], self.layer.k, self.slots_per_token
        _, prob, perm, offsets, _ = self.layer.route(n, with_gap=False)
        if not self.layer.has_shared:
            return perm, offsets[:-1], prob.view(-1)
        last = torch.arange(k, T * per, per, dtype=torch.int32, device=n.device)
        slots = torch.cat([perm + torch.div(perm, k, rounding_mode="floor"), last])
        weights = torch.cat([prob, torch.ones_like(prob[:, :1])], dim=1).view(-1)
        return slots, offsets, weights

    def experts(self, n: torch.Tensor) -> torch.Tensor:
        """The weighted expert outputs of every slot, [T, k + shared, d]."""
        if n.shape[0] == 0:
            return n.new_empty((0, self.slots_per_token, n.shape[1]))
        slots, offsets, weights = self.slots(n)
        rows = binding.moe_mx4_quantize(n, src=slots, src_div=self.slots_per_token)
        hidden = self.up.matmul(*rows, offsets)
        y = self.down.matmul(*binding.moe_mx4_quantize(hidden), offsets, out_rows=slots, row_scale=weights)
        return y.view(n.shape[0], self.slots_per_token, -1)

    def forward(self, x: torch.Tensor, n: torch.Tensor):
        """(out, n_next) of the residual stream x and its norm n, both [T, d]."""
        return binding.moe_norm_residual(x, self.experts(n), **self.norm, **self.options)

    __call__ = forward

    def backward(self, d_out, d_n, out, y) -> dict:
        """Gradients of forward's results with respect to x, the expert outputs y, the norm weights and the gate
        (the 4-bit experts themselves are not trained)."""
        return binding.moe_norm_residual_backward(d_out, d_n, out, y, **self.norm, **self.options)

    def check(self) -> int:
        """MOE_OK, or the first failure a kernel of the block's products reported."""
        return self.up.check() or self.down.check()


def main(tokens: int = 192, steps: int = 40) -> None:
    shape = synth.LayerShape(T=tokens, d=512, E=32, k=4, F=256)
    inp = synth.make_inputs(shape, seed=0, device="cuda")
    layer = binding.MoeLayer(inp.w_router, inp.w_gate_up, inp.w_down, shape.k, max_tokens=tokens)
    d = shape.d
    ones = torch.ones(d, device="cuda")
    block = Mx4Block(layer, inp.w_gate_up, inp.w_down, w_post=ones.clone(), gate=torch.full((d,), -2.0, device="cuda"),
                     w_pre=ones.clone(), sigmoid=True)
    x = inp.x
    _, n = binding.moe_norm_residual(x, w_pre=ones)

    # the same block in bf16: the layer's own output in the place of the slots'
    y16 = layer.forward(n)
    out16, n16 = binding.moe_norm_residual(x, y16, **block.norm, **block.options)
    out, n_next = block(x, n)
    err = (out.float() - out16.float()).norm() / (out16.float() - x.float()).norm()
    print(f"prompt of {tokens} tokens: branch of the 4-bit block off by {err:.3f} of the bf16 block's")

    alone = [block(x[t : t + 1], n[t : t + 1])[0] for t in range(4)]
    same = all(torch.equal(a[0], out[t]) for t, a in enumerate(alone))
    print(f"tokens one at a time: {'the same bits' if same else 'within rounding'} as in the prompt")

    # norms and gate, which starts nearly closed, fitted to the bf16 block with an open gate
    target = binding.moe_norm_residual(x, y16, w_post=ones, gate=ones, w_pre=ones, sigmoid=True)[1].float()
    y = block.experts(n)
    for step in range(steps):
        out, n_next = binding.moe_norm_residual(x, y, **block.norm, **block.options)
        diff = n_next.float() - target
        if step % 10 == 0 or step == steps - 1:
            print(f"step {step:3d}: mean square distance {diff.square().mean():.6f}")
        grads = block.backward(None, (diff * (2.0 / diff.numel())).to(n_next.dtype), out, y)
        for name, rate in (("w_post", 0.02), ("gate", 0.3), ("w_pre", 0.02)):  # steps of one length, shrinking
            g = grads[name]
            block.norm[name] -= rate * (1 - step / steps) * g / g.square().mean().sqrt()
    status = block.check()
    if status != binding.MOE_OK:
        raise RuntimeError(binding.moe_status_string(status))


if __name__ == "__main__":
    main()
