"""The router's training step over tokens that the mask leaves out."""
import pytest
import torch

from sparse_moe_ffn_gb300.block import router_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [torch.bool, torch.uint8])
def test_tokens_left_out_may_hold_anything(bad, dtype):
    """Their hidden states reach neither the losses nor the gradient: the same
    bits as with zeros in their place."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(300, 256, generator=g, device="cuda").to(torch.bfloat16)
    router = (torch.randn(32, 256, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    keep = torch.arange(300, device="cuda") % 7 != 3
    x[~keep] = 0
    mask = keep.to(dtype)
    clean = router_step(x, router, 4, 0.3, 0.01, mask)
    x[~keep] = bad
    got = router_step(x, router, 4, 0.3, 0.01, mask)
    assert bool(got[2].isfinite().all())
    for a, b in zip(clean, got):
        assert torch.equal(a, b)
