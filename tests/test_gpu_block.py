"""The operators put together (block.py): the block's pieces against plain
forms, and the router's balance under gradient steps."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding
from sparse_moe_ffn_gb300.block import ProjectionMLP, SparseBlock, router_step
from sparse_moe_ffn_gb300.inputs import MoEShape, make_inputs, to_device

pytestmark = pytest.mark.gpu


def _setup(N, skew=False, H=256, E=32, I=128, k=4):
    w = to_device(make_inputs(MoEShape("block", N=N, H=H, E=E, k=k, I=I, skew=skew), seed=3))
    x = w.pop("x")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def normal(*s, std):
        return (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)

    raw = (normal(512, H, std=0.05), normal(512, std=0.1), normal(H, 512, std=0.05),
           normal(H, std=0.1))
    return x, w, normal(N, H, std=2.0), raw, k


@pytest.mark.parametrize("N", [1, 77, 700])
def test_block_pieces(N):
    x, w, residual, raw, k = _setup(N)
    mlp = ProjectionMLP(*raw)
    norm = torch.ones(x.shape[1], dtype=torch.bfloat16, device="cuda")
    before = residual.clone()
    out, projected, normed = SparseBlock(norm, w, k, projection=mlp)(x, residual)
    assert torch.equal(residual, (x.float() + before.float()).to(torch.bfloat16))
    # the sparse layer reads the same bf16 hidden state as moe_add_rmsnorm gives,
    # up to the last bit of the row's fp32 norm
    r2 = before.clone()
    plain = binding.moe_add_rmsnorm(x, r2, norm)
    assert float((plain.float() - normed.float()).abs().max()) <= 2.0 ** -7 * float(
        normed.float().abs().max())
    assert torch.equal(out, binding.moe_forward(normed, w["router"], w["w_gate"], w["w_up"],
                                                w["w_down"], k))
    # the projection from its e4m3 operands, in 64 bits: the hidden values are
    # rounded to bf16 (2^-8 of each), the rest are fp32 sums of at most 512 terms
    # (2^-16 of their magnitudes) and the output's rounding
    q, s, _ = binding.moe_add_rmsnorm_fp8(x, before.clone(), norm)
    v = (q.double() * s.double()[:, None]) @ (mlp.w1.double() * mlp.s1.double()[:, None]).T
    v = v + raw[1].double()
    mag = (q.double().abs() * s.double()[:, None]) @ (mlp.w1.double().abs() *
                                                      mlp.s1.double()[:, None]).T
    h = v * torch.sigmoid(v)
    dh = 2.0 ** -8 * h.abs() + 2.0 ** -15 * (mag + raw[1].double().abs())
    y = h @ raw[2].double().T + raw[3].double()
    tol = dh @ raw[2].double().abs().T + 2.0 ** -15 * (h.abs() @ raw[2].double().abs().T)
    tol = tol + 2.0 ** -8 * (y.abs() + tol)
    assert bool(((projected.double() - y).abs() <= tol).all())


def test_router_step_gradient_and_balance():
    x, w, residual, _, k = _setup(1024, skew=True)
    router, mask = w["router"], torch.arange(1024, device="cuda") % 5 != 0
    losses, counts, grad = router_step(x, router, k, 0.3, 0.01, mask)
    # the same losses by autograd in 64 bits, the counts held fixed
    r = router.double().requires_grad_()
    lg = (x.double() @ r.T)[mask]
    f = counts.double() / (k * int(mask.sum()))
    bal = 32 * (f * torch.softmax(lg, 1).mean(0)).sum()
    z = torch.logsumexp(lg, 1).square().mean()
    (0.3 * bal + 0.01 * z).backward()
    # fp32 logits and gradient sums over 820 tokens: 2^-12 of the largest one
    assert float((grad.double() - r.grad).abs().max()) <= 2.0 ** -12 * float(r.grad.abs().max())
    assert abs(float(losses[0]) - float(bal.detach())) <= 2.0 ** -14 * float(bal.detach())
    assert abs(float(losses[1]) - float(z.detach())) <= 2.0 ** -14 * float(z.detach())
    assert int(counts.sum()) == k * int(mask.sum())
    master = router.float()
    for _ in range(40):
        last, _, g = router_step(x, master.to(torch.bfloat16), k, 1.0, 1e-4, mask)
        master -= 2.0 * g
    assert float(last[0]) < 1.0 + 0.5 * (float(losses[0]) - 1.0)
