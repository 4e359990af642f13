"""The operators around the sparse layer, put together as a decoder uses them.

``SparseBlock`` is the FFN half of a decoder block: residual add + RMSNorm
(which also gives the hidden state in e4m3), the sparse layer, and an optional
biased projection MLP (linear, SiLU, linear) read from the e4m3 copy.
``router_step`` is the training signal of its router: logits in fp32, the load
balance and log-sum-exp losses over the tokens that a mask leaves in, and the
gradient of the router's weights.

``python -m sparse_moe_ffn_gb300.block`` runs a block and then balances a
skewed router by gradient steps, printing the load before and after.
"""
from __future__ import annotations

import torch

from . import binding


class ProjectionMLP:
    """y = silu(x W1^T + b1) W2^T + b2 [+ residual]: W1 [I, H] is kept in e4m3
    with a scale per output (converted once, here), W2 [O, I] in bf16; b1 [I]
    and b2 [O] in bf16."""

    def __init__(self, w1, b1, w2, b2):
        self.w1, self.s1 = binding.moe_quantize_fp8(w1)
        self.b1, self.w2, self.b2 = b1, w2, b2

    def __call__(self, q, scale, residual=None, out=None):
        h = binding.moe_linear(q, self.w1, bias=self.b1, activation="silu", x_scale=scale,
                               w_scale=self.s1)
        return binding.moe_linear(h, self.w2, bias=self.b2, residual=residual, out=out)


class SparseBlock:
    """norm_weight [H] bf16; weights: the sparse layer's tensors, as
    moe_forward takes them (with or without the shared expert); projection: a
    ProjectionMLP or None."""

    def __init__(self, norm_weight, weights: dict, k: int, norm_topk_prob: bool = True,
                 projection: ProjectionMLP | None = None, eps: float = 1e-6):
        self.norm_weight, self.weights, self.k = norm_weight, weights, k
        self.norm_topk_prob, self.projection, self.eps = norm_topk_prob, projection, eps
        self.shared = ({n: weights[n] for n in binding.SHARED_KEYS}
                       if "shared_gate" in weights else None)

    def __call__(self, x, residual):
        """residual <- bf16(x + residual) in place; returns (the sparse layer's
        output [N, H], the projection of the normed hidden state or None, the
        normed hidden state [N, H])."""
        q, scale, normed = binding.moe_add_rmsnorm_fp8(x, residual, self.norm_weight,
                                                       eps=self.eps, want_normed=True)
        w = self.weights
        out = binding.moe_forward(normed, w["router"], w["w_gate"], w["w_up"], w["w_down"],
                                  self.k, self.norm_topk_prob, self.shared)
        projected = None if self.projection is None else self.projection(q, scale)
        return out, projected, normed


def router_step(normed, router, k: int, balance_weight: float = 0.01, z_weight: float = 0.001,
                mask=None):
    """(losses fp32 [2], counts int32 [E], gradient fp32 [E, H]) of
    balance_weight * load balance + z_weight * mean squared log-sum-exp with
    respect to the router's weights."""
    logits = binding.moe_linear(normed, router, out_dtype=torch.float32)
    ids = binding.moe_route_raw(normed, router, k, True)[1]
    losses, counts, tokens = binding.moe_balance_loss(logits, ids, mask)
    grad = torch.tensor([balance_weight, z_weight], dtype=torch.float32, device=normed.device)
    dlogits = binding.moe_balance_loss_backward(logits, counts, tokens, k, grad, mask)
    hidden = normed.float()
    if mask is not None:  # whatever a token left out holds: 0 * NaN is NaN
        hidden = hidden.masked_fill(mask.logical_not()[:, None], 0)
    return losses, counts, dlogits.t() @ hidden


def main(N: int = 2048, H: int = 512, E: int = 32, k: int = 4, I: int = 256, steps: int = 60):
    from .inputs import MoEShape, make_inputs, to_device
    shape = MoEShape("block", N=N, H=H, E=E, k=k, I=I, skew=True)
    w = to_device(make_inputs(shape, seed=0))
    x = w.pop("x")
    g = torch.Generator(device="cuda")
    g.manual_seed(0)

    def normal(*s, std):
        return (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)

    mlp = ProjectionMLP(normal(2 * H, H, std=0.02), normal(2 * H, std=0.1),
                        normal(H, 2 * H, std=0.02), normal(H, std=0.1))
    block = SparseBlock(torch.ones(H, dtype=torch.bfloat16, device="cuda"), w, k, projection=mlp)
    residual = torch.zeros_like(x)
    out, projected, normed = block(x, residual)
    print(f"block: out {tuple(out.shape)} rms {float(out.float().square().mean().sqrt()):.4f}, "
          f"projection rms {float(projected.float().square().mean().sqrt()):.4f}")
    master = w["router"].float()
    for step in range(steps):
        losses, counts, grad = router_step(normed, master.to(torch.bfloat16), k, 1.0, 1e-4)
        if step in (0, steps - 1):
            print(f"step {step}: balance {float(losses[0]):.4f}, largest load "
                  f"{int(counts.max())} of {N * k} slots, experts without one "
                  f"{int((counts == 0).sum())}")
        master -= 2.0 * grad
    return losses


if __name__ == "__main__":
    main()
