"""Tensors on different devices, or on another than the current one, are
refused before the library is called: the operators launch on the current
device, whose stream and memory another device's are not.  On the host, with
stand-ins that report a device."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding

BF16, F32, F8, I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


class Stand:
    """What the wrappers ask of a tensor, on a device that this machine lacks."""

    def __init__(self, dtype, *shape, index=0):
        self.dtype, self.shape, self.index = dtype, torch.Size(shape), index
        self.device = torch.device("cuda", index)
        self.is_cuda = True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


class Library:
    """Counts the calls instead of making them."""

    def __init__(self):
        self.calls = 0

    def moe_balance_loss_workspace_bytes(self, N, E):
        return 256

    def __getattr__(self, name):
        def entry(*args):
            self.calls += 1
            return 0
        return entry


N, H, O, E, k = 4, 64, 48, 8, 2


def rms(**t):
    return binding.moe_add_rmsnorm_fp8(t["x"], t["residual"], t["weight"], q=t["q"],
                                       scale=t["scale"], normed=t["normed"],
                                       residual_out=t["residual_out"])


def quantize(**t):
    return binding.moe_quantize_fp8(t["x"], t["q"], t["scale"])


def linear(**t):
    return binding.moe_linear(t["x"], t["weight"], bias=t["bias"], residual=t["residual"],
                              x_scale=t.get("x_scale"), w_scale=t.get("w_scale"), out=t["out"],
                              workspace=t["workspace"])


def balance(**t):
    return binding.moe_balance_loss(t["logits"], t["topk_ids"], t["mask"], t["losses"],
                                    t["counts"], t["tokens"], t["workspace"])


def balance_backward(**t):
    return binding.moe_balance_loss_backward(t["logits"], t["counts"], t["tokens"], k, t["grad"],
                                             t["mask"], t["dlogits"])


LINEAR = dict(bias=(BF16, O), residual=(BF16, N, O), out=(BF16, N, O),
              workspace=(torch.uint8, 256))
CASES = {
    "rms": (rms, dict(x=(BF16, N, H), residual=(BF16, N, H), weight=(BF16, H), q=(F8, N, H),
                      scale=(F32, N), normed=(BF16, N, H), residual_out=(BF16, N, H))),
    "quantize": (quantize, dict(x=(BF16, N, H), q=(F8, N, H), scale=(F32, N))),
    "linear": (linear, dict(x=(BF16, N, H), weight=(BF16, O, H), **LINEAR)),
    "linear e4m3": (linear, dict(x=(F8, N, H), weight=(F8, O, H), x_scale=(F32, N),
                                 w_scale=(F32, O), **LINEAR)),
    "balance": (balance, dict(logits=(F32, N, E), topk_ids=(I32, N, k), mask=(torch.bool, N),
                              losses=(F32, 2), counts=(I32, E), tokens=(I32, 1),
                              workspace=(torch.uint8, 256))),
    "balance backward": (balance_backward, dict(logits=(BF16, N, E), counts=(I32, E),
                                                tokens=(I32, 1), grad=(F32, 2),
                                                mask=(torch.uint8, N), dlogits=(BF16, N, E))),
}


@pytest.fixture
def library(monkeypatch):
    fake = Library()
    monkeypatch.setattr(binding, "lib", lambda: fake)
    monkeypatch.setattr(binding, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    binding._balance_workspace_bytes.cache_clear()
    yield fake
    binding._balance_workspace_bytes.cache_clear()


@pytest.mark.parametrize("name", CASES)
def test_operands_on_one_device(library, name, monkeypatch):
    call, specs = CASES[name]
    call(**{n: Stand(*s) for n, s in specs.items()})
    assert library.calls == 1
    for other in specs:  # each of them in turn elsewhere
        with pytest.raises(ValueError, match="cuda:"):
            call(**{n: Stand(*s, index=int(n == other)) for n, s in specs.items()})
    # all together elsewhere, with the current device unchanged
    with pytest.raises(ValueError, match="current device"):
        call(**{n: Stand(*s, index=1) for n, s in specs.items()})
    assert library.calls == 1
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    call(**{n: Stand(*s, index=1) for n, s in specs.items()})
    assert library.calls == 2
