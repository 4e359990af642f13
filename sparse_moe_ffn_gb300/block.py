"""The operators around the sparse layer, put together as a decoder uses them.

``SparseBlock`` is the FFN half of a decoder block: residual add + RMSNorm
(which also gives the hidden state in e4m3), the sparse layer, and an optional
biased projection MLP (linear, SiLU, linear) read from the e4m3 copy.
``router_step`` is the training signal of its router: logits in fp32, the load
balance and log-sum-exp losses over the tokens that a mask leaves in, and the
gradient of the router's weights.
``DenseBlock`` is the FFN half of a decoder block without experts: residual add +
layer norm and the gated feed-forward block onto the residual stream, for
serving and, with what ``forward(..., keep=True)`` keeps, for training.
``clip_step`` scales a set of gradients to a largest norm.

``python -m sparse_moe_ffn_gb300.block`` runs a block, balances a skewed router
by gradient steps, printing the load before and after, and takes steps of a
dense block.
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


class DenseBlock:
    """r = x + residual, out = FFN(layernorm(r)) + r: norm_weight [H], norm_bias
    [H] or None, w_gate and w_up [I, H], w_down [H, I], all bf16; activation as
    moe_gated_ffn takes it."""

    def __init__(self, norm_weight, norm_bias, w_gate, w_up, w_down, activation: str = "silu",
                 eps: float = 1e-5):
        self.norm_weight, self.norm_bias = norm_weight, norm_bias
        self.w_gate, self.w_up, self.w_down = w_gate, w_up, w_down
        self.activation, self.eps = activation, eps

    def __call__(self, x, residual, keep: bool = False, workspace=None):
        """out [N, H], the residual stream behind the block; with ``keep`` also
        what ``backward`` needs.  residual becomes r."""
        normed, mean, rstd = binding.moe_layernorm(x, self.norm_weight, self.norm_bias, residual,
                                                   self.eps)
        out, gate, up = binding.moe_gated_ffn(normed, self.w_gate, self.w_up, self.w_down,
                                              self.activation, residual=residual, keep=keep,
                                              workspace=workspace)
        return (out, (residual, normed, mean, rstd, gate, up)) if keep else out

    def backward(self, dout, kept, workspace=None):
        """(the gradient of r, which is x's and the residual's, {name: gradient}
        of the weights) for the gradient dout of out: bf16 for the projections,
        fp32 for the norm."""
        r, normed, mean, rstd, gate, up = kept
        dnormed, dw_gate, dw_up, dw_down = binding.moe_gated_ffn_backward(
            dout, normed, self.w_gate, self.w_up, self.w_down, gate, up, self.activation,
            workspace=workspace)
        dr, dweight, dbias = binding.moe_layernorm_backward(
            dnormed, r, self.norm_weight, mean, rstd, dresidual=dout,
            want_dbias=self.norm_bias is not None)
        grads = {"w_gate": dw_gate, "w_up": dw_up, "w_down": dw_down, "norm_weight": dweight}
        if dbias is not None:
            grads["norm_bias"] = dbias
        return dr, grads


def clip_step(grads: dict, max_norm: float):
    """Scales the gradients in place so that the norm of all of them together is
    max_norm at most; returns the norm before (fp32 [1], on the device)."""
    kept = binding.GradSet(grads.values())
    norm = binding.moe_grad_norm(kept)
    binding.moe_clip_grads(kept, norm, max_norm)
    return norm


def dense_steps(N: int = 1000, H: int = 256, I: int = 512, steps: int = 20, max_norm: float = 1.0):
    """Gradient steps of a DenseBlock towards a random target, the gradients
    clipped; returns the norms before clipping."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def normal(*s, std):
        return torch.randn(s, generator=g, device="cuda") * std

    master = {"norm_weight": torch.ones(H, device="cuda"),
              "norm_bias": torch.zeros(H, device="cuda"), "w_gate": normal(I, H, std=H ** -0.5),
              "w_up": normal(I, H, std=H ** -0.5), "w_down": normal(H, I, std=I ** -0.5)}
    x, residual = (normal(N, H, std=1.0).to(torch.bfloat16) for _ in range(2))
    target = normal(N, H, std=1.0)
    norms = []
    for step in range(steps):
        block = DenseBlock(**{n: t.to(torch.bfloat16) for n, t in master.items()})
        out, kept = block(x, residual.clone(), keep=True)
        diff = out.float() - target
        _, grads = block.backward((2.0 / N * diff).to(torch.bfloat16), kept)
        norms.append(float(clip_step(grads, max_norm)))
        for name, t in master.items():
            t -= 0.1 * grads[name].float()
        if step in (0, steps - 1):
            print(f"dense step {step}: loss {float(diff.square().sum() / N):.4f}, gradient norm "
                  f"{norms[-1]:.4f}")
    return norms


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
    dense_steps()
    return losses


if __name__ == "__main__":
    main()
