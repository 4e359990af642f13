"""Refusals of the e4m3, linear and balance entry points, on the host: every
bad argument is rejected before anything is enqueued."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding
from sparse_moe_ffn_gb300 import build as lib_build

OK, INVALID, SMALL, UNSUPPORTED = 0, 1, 2, 3
P = 0x10000  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def L():
    lib_build.build()
    return binding.lib()


def test_add_rmsnorm_fp8_argument_errors(L):
    def call(x=P, r=P, w=P, N=4, H=64, eps=1e-6, ro=P, q=P, s=P, n=P):
        return L.moe_add_rmsnorm_fp8(x, r, w, N, H, eps, 0, ro, q, s, n, None)

    assert call(N=-1) == INVALID
    assert call(H=0) == INVALID
    assert call(H=60) == INVALID
    assert call(H=65536 + 8) == UNSUPPORTED
    assert call(eps=-1.0) == INVALID
    assert call(eps=float("nan")) == INVALID
    for name in ("x", "w", "q", "s"):
        assert call(**{name: None}) == INVALID, name
    for name in ("x", "r", "w", "ro", "q", "n"):
        assert call(**{name: P + 8}) == INVALID, name
    assert call(s=P + 2) == INVALID
    assert b"aligned" in L.moe_last_error()
    assert call(N=0, x=None) == OK


def test_quantize_fp8_argument_errors(L):
    def call(x=P, N=4, H=64, q=P, s=P):
        return L.moe_quantize_fp8(x, N, H, q, s, None)

    assert call(N=-1) == INVALID
    assert call(H=12) == INVALID
    assert call(H=65536 + 8) == UNSUPPORTED
    assert call(x=None) == INVALID
    assert call(q=None) == INVALID
    assert call(s=None) == INVALID
    assert call(x=P + 2) == INVALID
    assert call(q=P + 8) == INVALID
    assert call(s=P + 1) == INVALID
    assert call(N=0, x=None) == OK


@pytest.mark.parametrize("fp8", [False, True])
def test_linear_argument_errors(L, fp8):
    def call(x=P, w=P, sx=P, sw=P, b=P, r=P, N=4, K=64, O=48, act=0, out=P * 2, fp32=0, ws=P,
             wsb=256):
        if fp8:
            return L.moe_linear_fp8(x, sx, w, sw, b, r, N, K, O, act, out, fp32, ws, wsb, None)
        return L.moe_linear(x, w, b, r, N, K, O, act, out, fp32, ws, wsb, None)

    assert call(N=-1) == INVALID
    assert call(K=0) == INVALID
    assert call(K=8 if fp8 else 4) == INVALID
    assert call(K=72 if fp8 else 68) == INVALID
    assert call(O=0) == INVALID
    assert call(act=5) == INVALID
    assert call(act=-1) == INVALID
    assert call(N=1 << 31) == UNSUPPORTED
    assert call(O=(1 << 31) - 16) == UNSUPPORTED
    assert call(K=(1 << 31) - 16) == UNSUPPORTED
    assert call(wsb=0) == SMALL
    assert call(ws=P + 2) == INVALID
    for name in ("x", "w", "out") + (("sx", "sw") if fp8 else ()):
        assert call(**{name: None}) == INVALID, name
    for name in ("x", "w"):
        assert call(**{name: P + 8}) == INVALID, name
    for name in ("b", "r", "out"):
        assert call(**{name: P + 1}) == INVALID, name
    assert call(fp32=1, out=P * 2 + 2) == INVALID
    assert call(fp32=1, out=P, r=P) == INVALID
    assert call(N=0, x=None, out=None) == OK
    assert L.moe_linear_workspace_bytes() <= 256


def test_balance_argument_errors(L):
    need = L.moe_balance_loss_workspace_bytes(100000, 64)
    assert need > 256
    assert L.moe_balance_loss_workspace_bytes(100, 64) == 256  # the status word alone
    assert L.moe_balance_loss_workspace_bytes(-1, 64) == 0
    assert L.moe_balance_loss_workspace_bytes(100, 257) == 0

    def fwd(lg=P, bf16=0, ids=P, m=None, N=100000, E=64, k=8, lo=P, c=P, t=P, ws=P, wsb=need):
        return L.moe_balance_loss(lg, bf16, ids, m, N, E, k, lo, c, t, ws, wsb, None)

    assert fwd(N=-1) == INVALID
    assert fwd(E=0) == INVALID
    assert fwd(k=0) == INVALID
    assert fwd(k=65) == INVALID
    assert fwd(E=257) == UNSUPPORTED
    assert fwd(N=1 << 28, k=8) == UNSUPPORTED
    for name in ("lg", "ids", "lo", "c", "t", "ws"):
        assert fwd(**{name: None}) == INVALID, name
    for name in ("lg", "ids", "lo", "c", "t"):
        assert fwd(**{name: P + 2}) == INVALID, name
    assert fwd(bf16=1, lg=P + 1) == INVALID
    assert fwd(ws=P + 64) == INVALID
    assert fwd(wsb=need - 1) == SMALL

    def bwd(lg=P, bf16=0, c=P, t=P, m=None, g=P, N=100, E=64, k=8, d=P):
        return L.moe_balance_loss_backward(lg, bf16, c, t, m, g, N, E, k, d, None)

    assert bwd(N=-1) == INVALID
    assert bwd(E=300) == UNSUPPORTED
    assert bwd(k=0) == INVALID
    for name in ("lg", "c", "t", "g", "d"):
        assert bwd(**{name: None}) == INVALID, name
        assert bwd(**{name: P + 2}) == INVALID, name
    assert bwd(N=0, lg=None) == OK


def test_binding_refuses_wrong_tensors():
    """The binding's own checks: type, place, shape, contiguity."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_add_rmsnorm_fp8(x, x, w)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_quantize_fp8(x)
    with pytest.raises(ValueError, match="two dimensions"):
        binding.moe_quantize_fp8(w)
    with pytest.raises(ValueError, match="two dimensions"):
        binding.moe_linear(x, w)
    with pytest.raises(ValueError, match="two dimensions"):
        binding.moe_balance_loss(w, torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="workspace"):
        binding.moe_linear(x, x, out=x, workspace=torch.zeros(64))
    with pytest.raises(ValueError, match="activation"):
        binding.moe_linear(x, x, activation="swish")
    with pytest.raises(ValueError, match="x_scale"):
        binding.moe_linear(x.to(torch.float8_e4m3fn), x.to(torch.float8_e4m3fn), out=x)
    with pytest.raises(ValueError, match="e4m3"):
        binding.moe_linear(x, x, x_scale=torch.ones(4), out=x)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_linear(x, x)
    with pytest.raises(ValueError, match="fp32 or bf16"):
        binding.moe_balance_loss(x.half(), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="mask"):
        binding._mask(torch.ones(4), 4)
