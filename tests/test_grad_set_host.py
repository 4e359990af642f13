"""A GradSet whose tensors have moved since it was made is refused before the library
sees their old addresses; on the host, with stand-ins for the tensors."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding
from test_block_ops_devices_host import Stand

BF16, F32 = torch.bfloat16, torch.float32
P = 1 << 20


class At(Stand):
    def __init__(self, dtype, n, place):
        super().__init__(dtype, n)
        self.place = place

    def data_ptr(self):
        return self.place


@pytest.fixture
def calls(monkeypatch):
    seen = []

    class Fake:
        def __getattr__(self, name):
            return lambda *args: seen.append(name) or 0

    monkeypatch.setattr(binding, "lib", lambda: Fake())
    monkeypatch.setattr(binding, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_data_ptr", lambda t: t.data_ptr())
    return seen


def both(kept):
    norm, ws = At(F32, 1, 64 * P), At(torch.uint8, 4096, 65 * P)
    binding.moe_grad_norm(kept, norm=norm, workspace=ws)
    binding.moe_clip_grads(kept, norm, 1.0)


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("which", range(3))
def test_a_gradient_that_moved(calls, which, apart):
    grads = [At(t, 100, (i + 1) * P) for i, t in enumerate((BF16, F32, BF16))]
    out = [At(F32, 100, (i + 10) * P) for i in range(3)] if apart else None
    kept = binding.GradSet(grads, out)
    both(kept)
    assert calls == ["moe_grad_norm", "moe_clip_grads"]
    grads[which].place += 16 * P
    with pytest.raises(ValueError, match=rf"grads\[{which}\] has another storage"):
        binding.moe_grad_norm(kept)
    with pytest.raises(ValueError, match=rf"grads\[{which}\] has another storage"):
        binding.moe_clip_grads(kept, At(F32, 1, 64 * P), 1.0)
    assert len(calls) == 2
    grads[which].place -= 16 * P
    both(kept)


def test_an_output_that_moved(calls):
    grads, out = [At(F32, 8, P), At(F32, 8, 2 * P)], [At(F32, 8, 3 * P), At(BF16, 8, 4 * P)]
    kept = binding.GradSet(grads, out)
    out[1].place = 5 * P
    binding.moe_grad_norm(kept, norm=At(F32, 1, 64 * P), workspace=At(torch.uint8, 4096, 65 * P))
    with pytest.raises(ValueError, match=r"out\[1\] has another storage"):
        binding.moe_clip_grads(kept, At(F32, 1, 64 * P), 1.0)
    assert calls == ["moe_grad_norm"]


def test_a_list_that_changed(calls):
    kept = binding.GradSet([At(F32, 8, P), At(F32, 8, 2 * P)])
    kept.grads.append(At(F32, 8, 3 * P))
    with pytest.raises(ValueError, match="3 tensors instead of 2"):
        binding.moe_grad_norm(kept)
    kept.grads.pop()
    both(kept)
