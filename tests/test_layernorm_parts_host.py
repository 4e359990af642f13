"""What the layer norm's backward wrapper hands to the library for each part of the
gradients, with stand-ins for the tensors."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding
from test_block_ops_devices_host import Stand

BF16, F32 = torch.bfloat16, torch.float32
N, H = 4, 64


@pytest.fixture
def calls(monkeypatch):
    seen = []

    class Fake:
        def moe_layernorm_backward_workspace_bytes(self, N, H):
            return 512

        def moe_layernorm_backward(self, *args):
            seen.append(args)
            return 0

    monkeypatch.setattr(binding, "lib", lambda: Fake())
    monkeypatch.setattr(binding, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty",
                        lambda shape, dtype, device: Stand(dtype, *([shape] if isinstance(shape, int)
                                                                    else shape)))
    binding._layernorm_backward_workspace_bytes.cache_clear()
    yield seen
    binding._layernorm_backward_workspace_bytes.cache_clear()


@pytest.mark.parametrize("want", range(8))
def test_only_what_is_wanted_is_asked_for(calls, want):
    ins = [Stand(BF16, N, H), Stand(BF16, N, H), Stand(BF16, H), Stand(F32, N), Stand(F32, N)]
    which = [bool(want & 1), bool(want & 2), bool(want & 4)]
    got = binding.moe_layernorm_backward(*ins, want_dx=which[0], want_dweight=which[1],
                                         want_dbias=which[2])
    assert [t is not None for t in got] == which
    (args,) = calls
    dx, dweight, dbias, workspace, bytes_ = args[9:14]
    assert [p is not None for p in (dx, dweight, dbias)] == which
    sums = which[1] or which[2]
    assert (workspace is not None) == sums and (bytes_ >= 512 if sums else bytes_ == 0)


def test_a_workspace_that_is_given_is_handed_on(calls):
    ins = [Stand(BF16, N, H), Stand(BF16, N, H), Stand(BF16, H), Stand(F32, N), Stand(F32, N)]
    binding.moe_layernorm_backward(*ins, want_dweight=False, want_dbias=False,
                                   workspace=Stand(torch.uint8, 256))
    assert calls[0][12] is not None and calls[0][13] == 256
