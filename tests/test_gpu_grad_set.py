"""A GradSet whose tensors got other storage is refused; one that holds what it had
goes on."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("change", ["data", "resize", "set"])
def test_tensors_with_other_storage(change):
    grads = [torch.full((n,), 2.0, device="cuda") for n in (100, 5000)]
    out = [torch.zeros_like(t) for t in grads]
    kept = binding.GradSet(grads, out)
    norm = binding.moe_grad_norm(kept)
    assert float(norm) == pytest.approx(2 * 5100 ** 0.5, rel=2.0 ** -20)
    for tensors, name in ((grads, "grads"), (out, "out")):
        t = tensors[1]
        old = t.untyped_storage(), t.storage_offset(), t.shape, t.stride()
        if change == "data":
            keep = t.data
            t.data = torch.ones_like(t)
        elif change == "resize":
            old = None
            t.resize_(1 << 22)
        else:
            t.set_(torch.ones_like(t))
        with pytest.raises(ValueError, match=rf"{name}\[1\] has another storage"):
            binding.moe_clip_grads(kept, norm, 1.0)
        if name == "grads":
            with pytest.raises(ValueError, match="another storage"):
                binding.moe_grad_norm(kept)
        if old is None:
            return
        if change == "data":
            t.data = keep
        else:
            t.set_(*old)
    got = binding.moe_clip_grads(kept, binding.moe_grad_norm(kept), 1.0)
    assert float(torch.cat([t.reshape(-1) for t in got]).norm()) == pytest.approx(1.0, rel=1e-5)
