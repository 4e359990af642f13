"""ctypes binding of libsparse_moe_ffn.so, with the same entry-point names as
include/moe.h.  Argument marshalling only: torch tensors supply device
pointers and the current stream; every step of the layer runs in the
library's CUDA kernels.  There is no fallback: a missing library raises.

Down-projection weights may be the model's bf16 tensors or the fp16 copies
``prepare_weights`` makes once at load; the wrappers pick the library entry
point that takes that form (``moe_forward`` or ``moe_forward_prepared``, and
likewise for the host, experts and dense-MLP calls).
"""
from __future__ import annotations

import array
import ctypes
import functools
import os

import torch

from .build import LIB

MOE_OK = 0
MOE_BLOCK_M = 128
MOE_NUM_STAGES = 7
STAGE_NAMES = ("route", "align", "gather", "gate_up", "down", "shared", "combine")
SHARED_KEYS = ("shared_gate_proj", "shared_up_proj", "shared_down_proj", "shared_gate")


class MoEError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


class _Layout(ctypes.Structure):
    _fields_ = [(name, ctypes.c_size_t) for name in (
        "status", "topk_w", "topk_ids", "gamma", "counts", "offsets", "pad_offsets",
        "num_padded", "align_scratch", "sorted_pair", "block_expert", "ready", "x_sorted", "act",
        "ypair", "ypair_res", "total")] + [
        ("capacity", ctypes.c_int64), ("slots", ctypes.c_int), ("groups", ctypes.c_int)]


_lib = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB):
        raise RuntimeError(f"{LIB} is missing: build it first (python -m sparse_moe_ffn_gb300.build)")
    L = ctypes.CDLL(LIB)
    P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sig = {
        "moe_status_string": ([i32], ctypes.c_char_p),
        "moe_last_error": ([], ctypes.c_char_p),
        "moe_route_workspace_bytes": ([], sz),
        "moe_route": ([P, P, P, i64, i32, i32, i32, i32, P, P, P, P, P, sz, P], i32),
        "moe_align_capacity": ([i64, i32, i32, i32], i64),
        "moe_align_workspace_bytes": ([i64, i32, i32, i32], sz),
        "moe_align": ([P, i64, i32, i32, i32, P, P, P, P, P, P, sz, P], i32),
        "moe_forward_workspace_bytes": ([i64, i32, i32, i32, i32, i32], sz),
        "moe_forward": ([P] * 9 + [i64, i32, i32, i32, i32, i32, i32, P, P, sz, P], i32),
        "moe_forward_prepared": ([P] * 9 + [i64, i32, i32, i32, i32, i32, i32, P, P, sz, P], i32),
        "moe_forward_host": ([P] * 12 + [i64, i32, i32, i32, i32, i32, i32, P, sz, P], i32),
        "moe_forward_host_prepared": ([P] * 12 + [i64, i32, i32, i32, i32, i32, i32, P, sz, P],
                                      i32),
        "moe_experts_workspace_bytes": ([i64, i32, i32, i32], sz),
        "moe_experts": ([P, P, P, i64, i32, i32, i32, P, P, P, P, P, P, sz, P], i32),
        "moe_experts_prepared": ([P, P, P, i64, i32, i32, i32, P, P, P, P, P, P, sz, P], i32),
        "moe_combine": ([P, P, P, P, i32, i64, i32, i32, P, P], i32),
        "moe_combine_indexed": ([P, P, i64, P, P, P, i32, i64, i32, i32, P, P], i32),
        "moe_shared_chunks": ([i32, i32], i32),
        "moe_shared_expert_workspace_bytes": ([i64, i32, i32, i32], sz),
        "moe_shared_expert": ([P, P, i64, i32, i32, i32, P, P, P, P, P, P, sz, P], i32),
        "moe_shared_expert_prepared": ([P, P, i64, i32, i32, i32, P, P, P, P, P, P, sz, P],
                                       i32),
        "moe_ep_dispatch_workspace_bytes": ([i64, i32, i32], sz),
        "moe_ep_dispatch": ([P, P, P, i64, i32, i32, i32, i32, P, P, P, P, P, P, sz, P], i32),
        "moe_convert_bf16_to_f16": ([P, P, i64, P, P], i32),
        "moe_forward_layout": ([i64, i32, i32, i32, i32, i32, ctypes.POINTER(_Layout)], i32),
        "moe_read_device_status": ([P, P], i32),
        "moe_kernel_launch_count": ([], ctypes.c_uint64),
        "moe_set_stage_events": ([P, i32], i32),
        "moe_selftest_wait_timeout": ([P, sz, ctypes.c_uint64, P], i32),
        "moe_selftest_portable_clusters": ([i32], None),
        "moe_align_noalloc": ([P, i64, i32, i32, i32, P, P, P, P, P, P, P], i32),
        "moe_dense_mlp_workspace_bytes": ([i64, i32, i32], sz),
        "moe_add_rmsnorm": ([P, P, P, i64, i32, ctypes.c_float, i32, P, P], i32),
        "moe_add_rmsnorm_fp8": ([P, P, P, i64, i32, ctypes.c_float, i32, P, P, P, P, P], i32),
        "moe_quantize_fp8": ([P, i64, i32, P, P, P], i32),
        "moe_linear_workspace_bytes": ([], sz),
        "moe_linear": ([P, P, P, P, i64, i32, i32, i32, P, i32, P, sz, P], i32),
        "moe_linear_fp8": ([P, P, P, P, P, P, i64, i32, i32, i32, P, i32, P, sz, P], i32),
        "moe_balance_loss_workspace_bytes": ([i64, i32], sz),
        "moe_balance_loss": ([P, i32, P, P, i64, i32, i32, P, P, P, P, sz, P], i32),
        "moe_balance_loss_backward": ([P, i32, P, P, P, P, i64, i32, i32, P, P], i32),
        "moe_gated_ffn_workspace_bytes": ([i64, i32, i32], sz),
        "moe_gated_ffn": ([P] * 5 + [i64, i32, i32, i32, P, P, P, P, sz, P], i32),
        "moe_gated_ffn_backward_workspace_bytes": ([i64, i32, i32], sz),
        "moe_gated_ffn_backward": ([P] * 7 + [i64, i32, i32, i32] + [P] * 5 + [sz, P], i32),
        "moe_layernorm": ([P, P, P, P, i32, i64, i32, ctypes.c_float, P, P, P, P, P], i32),
        "moe_layernorm_backward_workspace_bytes": ([i64, i32], sz),
        "moe_layernorm_backward": ([P] * 6 + [i32, i64, i32] + [P] * 4 + [sz, P], i32),
        "moe_grad_norm_workspace_bytes": ([i64], sz),
        "moe_grad_norm": ([P, P, P, i64, P, P, sz, P], i32),
        "moe_clip_grads": ([P, P, P, i64, P, ctypes.c_float, P, P, P], i32),
        "moe_dense_mlp": ([P, P, P, P, i64, i32, i32, P, P, sz, P], i32),
        "moe_dense_mlp_prepared": ([P, P, P, P, i64, i32, i32, P, P, sz, P], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def _check(status: int, what: str) -> None:
    if status != MOE_OK:
        L = lib()
        detail = L.moe_last_error().decode()
        raise MoEError(status, f"{what}: {L.moe_status_string(status).decode()}"
                               + (f" -- {detail}" if detail else ""))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _bf16(t, name, shape=None):
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _f16(t, name, shape=None):
    if t.dtype != torch.float16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp16 CUDA tensor "
                         "(convert the bf16 weights once with prepare_weights)")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _down(t, name, shape=None) -> bool:
    """Checks a down-projection weight; True if it is the prepared fp16 copy."""
    if t.dtype == torch.float16:
        _f16(t, name, shape)
        return True
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bf16 (or its fp16 copy from prepare_weights)")
    _bf16(t, name, shape)
    return False


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def moe_kernel_launch_count() -> int:
    return int(lib().moe_kernel_launch_count())


def moe_route_raw(x, router, k: int, norm_topk_prob: bool, shared_gate=None,
                  want_bf16: bool = False):
    """Routing in the library's own types: (topk_w fp32 [N,k], topk_ids int32
    [N,k], gamma fp32 [N] or None, topk_w_bf16 or None)."""
    N, H = x.shape
    E = router.shape[0]
    _bf16(x, "x")
    _bf16(router, "router", (E, H))
    if shared_gate is not None:
        _bf16(shared_gate, "shared_gate", (1, H))
    dev = x.device
    w = torch.empty((N, k), dtype=torch.float32, device=dev)
    ids = torch.empty((N, k), dtype=torch.int32, device=dev)
    wb = torch.empty((N, k), dtype=torch.bfloat16, device=dev) if want_bf16 else None
    gamma = torch.empty(N, dtype=torch.float32, device=dev) if shared_gate is not None else None
    ws = torch.empty(lib().moe_route_workspace_bytes(), dtype=torch.uint8, device=dev)
    _check(lib().moe_route(_ptr(x), _ptr(router), _ptr(shared_gate), N, H, E, k,
                           int(bool(norm_topk_prob)), _ptr(w), _ptr(ids), _ptr(wb), _ptr(gamma),
                           _ptr(ws), ws.numel(), _stream()), "moe_route")
    return w, ids, gamma, wb


def moe_route(x, router, k: int, norm_topk_prob: bool = True):
    """The pages' route(): (weights in x.dtype, ids int64), each [N, k]."""
    _, ids, _, wb = moe_route_raw(x, router, k, norm_topk_prob, want_bf16=True)
    return wb, ids.long()


def moe_align(topk_ids, E: int, block_m: int = MOE_BLOCK_M):
    """Grouping of the pairs by expert; returns a dict of CUDA tensors."""
    if topk_ids.dtype != torch.int32 or not topk_ids.is_cuda or not topk_ids.is_contiguous():
        raise ValueError("topk_ids must be a contiguous int32 CUDA tensor")
    N, k = topk_ids.shape
    L = lib()
    cap = int(L.moe_align_capacity(N, k, E, block_m))
    dev = topk_ids.device
    sp = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    be = torch.empty(max(cap // block_m, 1), dtype=torch.int32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    npad = torch.empty(1, dtype=torch.int32, device=dev)
    wsb = int(L.moe_align_workspace_bytes(N, k, E, block_m))
    ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    _check(L.moe_align(_ptr(topk_ids), N, k, E, block_m, _ptr(sp), _ptr(be), _ptr(counts),
                       _ptr(offsets), _ptr(npad), _ptr(ws), wsb, _stream()), "moe_align")
    return {"sorted_pair": sp, "block_expert": be, "counts": counts, "offsets": offsets,
            "num_padded": npad, "capacity": cap, "workspace": ws}


def moe_align_noalloc(topk_ids, E: int, block_m: int = MOE_BLOCK_M):
    """moe_align for callers that cannot allocate scratch (see moe.h): the
    library's static device array serves as the workspace.  Returns the same
    dict as moe_align, with "status" (int32 [1]) in place of "workspace"."""
    if topk_ids.dtype != torch.int32 or not topk_ids.is_cuda or not topk_ids.is_contiguous():
        raise ValueError("topk_ids must be a contiguous int32 CUDA tensor")
    N, k = topk_ids.shape
    L = lib()
    cap = int(L.moe_align_capacity(N, k, E, block_m))
    dev = topk_ids.device
    sp = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    be = torch.empty(max(cap // block_m, 1), dtype=torch.int32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    npad = torch.empty(1, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    _check(L.moe_align_noalloc(_ptr(topk_ids), N, k, E, block_m, _ptr(sp), _ptr(be),
                               _ptr(counts), _ptr(offsets), _ptr(npad), _ptr(status), _stream()),
           "moe_align_noalloc")
    return {"sorted_pair": sp, "block_expert": be, "counts": counts, "offsets": offsets,
            "num_padded": npad, "capacity": cap, "status": status}


def moe_forward_layout(N, H, E, I, k, I_s=0) -> dict:
    lay = _Layout()
    _check(lib().moe_forward_layout(N, H, E, I, k, I_s, ctypes.byref(lay)), "moe_forward_layout")
    return {name: getattr(lay, name) for name, _ in _Layout._fields_}


def moe_forward_workspace_bytes(N, H, E, I, k, I_s=0) -> int:
    return int(lib().moe_forward_workspace_bytes(N, H, E, I, k, I_s))


def alloc_workspace(N, H, E, I, k, I_s=0, device="cuda"):
    """A workspace tensor for moe_forward (the caller owns it and may reuse it)."""
    return torch.empty(max(moe_forward_workspace_bytes(N, H, E, I, k, I_s), 256),
                       dtype=torch.uint8, device=device)


def moe_forward(x, router, w_gate, w_up, w_down, k: int, norm_topk_prob: bool = True,
                shared=None, out=None, workspace=None):
    """The whole layer.  ``shared`` is None or a dict with shared_gate_proj,
    shared_up_proj, shared_down_proj and shared_gate.  Every tensor is bf16,
    except that w_down and shared_down_proj may instead be the fp16 copies
    from ``prepare_weights`` (then moe_forward_prepared runs).  Returns out
    [N, H] bf16."""
    N, H = x.shape
    E, I, _ = w_gate.shape
    _bf16(x, "x")
    _bf16(router, "router", (E, H))
    _bf16(w_gate, "w_gate", (E, I, H))
    _bf16(w_up, "w_up", (E, I, H))
    prepared = _down(w_down, "w_down", (E, H, I))
    sp = [None] * 4
    I_s = 0
    if shared is not None:
        sp = [shared[n] for n in SHARED_KEYS]
        I_s = sp[0].shape[0]
        _bf16(sp[0], "shared_gate_proj", (I_s, H))
        _bf16(sp[1], "shared_up_proj", (I_s, H))
        if _down(sp[2], "shared_down_proj", (H, I_s)) != prepared:
            raise ValueError("w_down and shared_down_proj must both be bf16 or both fp16")
        _bf16(sp[3], "shared_gate", (1, H))
    if out is None:
        out = torch.empty((N, H), dtype=torch.bfloat16, device=x.device)
    _bf16(out, "out", (N, H))
    if workspace is None:
        workspace = alloc_workspace(N, H, E, I, k, I_s, x.device)
    fn = lib().moe_forward_prepared if prepared else lib().moe_forward
    _check(fn(_ptr(x), _ptr(router), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
              *[_ptr(t) for t in sp], N, H, E, I, I_s, k, int(bool(norm_topk_prob)), _ptr(out),
              _ptr(workspace), workspace.numel(), _stream()),
           "moe_forward_prepared" if prepared else "moe_forward")
    return out


def moe_add_rmsnorm(x, residual, weight, eps: float = 1e-6, gemma: bool = False, normed=None):
    """residual <- bf16(x + residual) in place; returns RMSNorm(residual) (bf16)."""
    N, H = x.shape
    _bf16(x, "x")
    _bf16(residual, "residual", (N, H))
    _bf16(weight, "weight", (H,))
    if normed is None:
        normed = torch.empty((N, H), dtype=torch.bfloat16, device=x.device)
    _bf16(normed, "normed", (N, H))
    _check(lib().moe_add_rmsnorm(_ptr(x), _ptr(residual), _ptr(weight), N, H, float(eps),
                                 int(bool(gemma)), _ptr(normed), _stream()), "moe_add_rmsnorm")
    return normed


# The operators below take a few microseconds each, so their wrappers keep to
# what the checks need: plain integers for pointers, and the current stream of
# the tensors' device without a Stream object (2.9 us of a 12 us call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # none without CUDA
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream_of(device):
    """The current stream of a device, which has to be the current one: the
    library launches there, and takes its number of SMs from there."""
    if device != _current_device():
        raise ValueError(f"the tensors are on cuda:{device}, which is not the current device "
                         f"(cuda:{_current_device()}): call within torch.cuda.device({device})")
    return _raw_stream(device)


def _typed(t, name, dtype, shape, device=-1):
    """The data pointer of a contiguous tensor of this type and shape on the
    CUDA device of this index (negative: the first operand is on none)."""
    if (t.dtype is dtype and t.get_device() == device >= 0 and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)}"
                     f"{f' on cuda:{device} like the first operand' if device >= 0 else ''}, got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}"
                     f"{'' if t.is_contiguous() else ', not contiguous'}")


def _matrix(t, name):
    raise ValueError(f"{name} must have two dimensions, got shape {tuple(t.shape)}")


_BF16, _F32, _I32, _E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def moe_add_rmsnorm_fp8(x, residual, weight, eps: float = 1e-6, gemma: bool = False, q=None,
                        scale=None, normed=None, residual_out=None, want_normed: bool = False):
    """r = bf16(x + residual) (x without a residual), y = RMSNorm(r): returns
    (q e4m3 [N, H], scale fp32 [N], normed bf16 [N, H] or None) with q * scale
    = y.  r goes to ``residual_out``, or without one back to ``residual``."""
    if x.dim() != 2:
        _matrix(x, "x")
    shape = N, H = x.shape
    dev = x.get_device()
    if residual_out is None:
        residual_out = residual
    if q is None:
        q = torch.empty(shape, dtype=_E4M3, device=x.device)
    if scale is None:
        scale = torch.empty(N, dtype=_F32, device=x.device)
    if normed is None and want_normed:
        normed = torch.empty(shape, dtype=_BF16, device=x.device)
    status = lib().moe_add_rmsnorm_fp8(
        _typed(x, "x", _BF16, shape, dev),
        None if residual is None else _typed(residual, "residual", _BF16, shape, dev),
        _typed(weight, "weight", _BF16, (H,), dev), N, H, eps, bool(gemma),
        None if residual_out is None else _typed(residual_out, "residual_out", _BF16, shape, dev),
        _typed(q, "q", _E4M3, shape, dev), _typed(scale, "scale", _F32, (N,), dev),
        None if normed is None else _typed(normed, "normed", _BF16, shape, dev),
        _stream_of(dev))
    if status:
        _check(status, "moe_add_rmsnorm_fp8")
    return q, scale, normed


def moe_quantize_fp8(x, q=None, scale=None):
    """Rows of a bf16 matrix to e4m3: (q [N, H], scale fp32 [N]), q * scale = x.
    Used for weights (once, at load) and for activations."""
    if x.dim() != 2:
        _matrix(x, "x")
    shape = N, H = x.shape
    dev = x.get_device()
    if q is None:
        q = torch.empty(shape, dtype=_E4M3, device=x.device)
    if scale is None:
        scale = torch.empty(N, dtype=_F32, device=x.device)
    status = lib().moe_quantize_fp8(_typed(x, "x", _BF16, shape, dev), N, H,
                                    _typed(q, "q", _E4M3, shape, dev),
                                    _typed(scale, "scale", _F32, (N,), dev), _stream_of(dev))
    if status:
        _check(status, "moe_quantize_fp8")
    return q, scale


ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4}


def moe_linear(x, weight, bias=None, residual=None, activation: str = "none", x_scale=None,
               w_scale=None, out=None, out_dtype=torch.bfloat16, workspace=None):
    """act(x weight^T [* x_scale * w_scale] + bias) + residual, [N, O] in bf16
    or fp32 (``out_dtype``, or ``out``'s type).  x [N, K] and weight [O, K] are
    both bf16 (moe_linear) or both e4m3 with their scales (moe_linear_fp8).
    ``workspace`` (uint8 CUDA tensor, optional) receives the status word of
    moe_read_device_status."""
    if x.dim() != 2:
        _matrix(x, "x")
    if weight.dim() != 2:
        _matrix(weight, "weight")
    N, K = x.shape
    O = weight.shape[0]
    dev = x.get_device()
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    if out is None:
        out = torch.empty((N, O), dtype=out_dtype, device=x.device)
    fp32 = out.dtype is _F32
    b = None if bias is None else _typed(bias, "bias", _BF16, (O,), dev)
    r = None if residual is None else _typed(residual, "residual", _BF16, (N, O), dev)
    ws, bytes_ = None, 0
    if workspace is not None:
        bytes_ = workspace.numel()
        ws = _typed(workspace, "workspace", torch.uint8, (bytes_,), dev)
    if x.dtype is _E4M3:
        if x_scale is None or w_scale is None:
            raise ValueError("e4m3 operands need x_scale and w_scale")
        status = lib().moe_linear_fp8(
            _typed(x, "x", _E4M3, (N, K), dev), _typed(x_scale, "x_scale", _F32, (N,), dev),
            _typed(weight, "weight", _E4M3, (O, K), dev),
            _typed(w_scale, "w_scale", _F32, (O,), dev), b, r, N, K, O, act,
            _typed(out, "out", _F32 if fp32 else _BF16, (N, O), dev), fp32, ws, bytes_,
            _stream_of(dev))
    else:
        if x_scale is not None or w_scale is not None:
            raise ValueError("x_scale and w_scale belong to e4m3 operands")
        status = lib().moe_linear(
            _typed(x, "x", _BF16, (N, K), dev), _typed(weight, "weight", _BF16, (O, K), dev), b, r,
            N, K, O, act, _typed(out, "out", _F32 if fp32 else _BF16, (N, O), dev), fp32, ws,
            bytes_, _stream_of(dev))
    if status:
        _check(status, "moe_linear_fp8" if x.dtype is _E4M3 else "moe_linear")
    return out


@functools.lru_cache(maxsize=256)
def _balance_workspace_bytes(N, E):
    return max(lib().moe_balance_loss_workspace_bytes(N, E), 256)


def _logits(logits, dev):
    dtype = logits.dtype
    if dtype is not _F32 and dtype is not _BF16:
        raise ValueError(f"logits must be fp32 or bf16, got {dtype}")
    if logits.dim() != 2:
        _matrix(logits, "logits")
    return dtype is _BF16, _typed(logits, "logits", dtype, logits.shape, dev)


def _mask(mask, N, dev=-1):
    if mask.dtype is not torch.bool and mask.dtype is not torch.uint8:
        raise ValueError(f"mask must be bool or uint8, got {mask.dtype}")
    return _typed(mask, "mask", mask.dtype, (N,), dev)


def moe_balance_loss(logits, topk_ids, mask=None, losses=None, counts=None, tokens=None,
                     workspace=None):
    """The router's losses and load: (losses fp32 [2] = load balance and mean
    squared log-sum-exp, counts int32 [E], tokens int32 [1]) of the logits
    [N, E] (fp32 or bf16) and the ids [N, k] that moe_route chose; ``mask``
    (bool [N], optional) leaves tokens out, a negative id is a dropped slot.
    ``workspace`` (uint8 CUDA tensor, optional) receives the status word of
    moe_read_device_status."""
    dev = logits.get_device()
    bf16, lp = _logits(logits, dev)
    N, E = logits.shape
    if topk_ids.dim() != 2:
        _matrix(topk_ids, "topk_ids")
    k = topk_ids.shape[1]
    if losses is None:
        losses = torch.empty(2, dtype=_F32, device=logits.device)
    if counts is None:
        counts = torch.empty(E, dtype=_I32, device=logits.device)
    if tokens is None:
        tokens = torch.empty(1, dtype=_I32, device=logits.device)
    need = _balance_workspace_bytes(N, E)
    if workspace is None and need > 256:  # else the status word alone
        workspace = torch.empty(need, dtype=torch.uint8, device=logits.device)
    ws, bytes_ = None, 0
    if workspace is not None:
        bytes_ = workspace.numel()
        ws = _typed(workspace, "workspace", torch.uint8, (bytes_,), dev)
    status = lib().moe_balance_loss(
        lp, bf16, _typed(topk_ids, "topk_ids", _I32, (N, k), dev),
        None if mask is None else _mask(mask, N, dev), N, E, k,
        _typed(losses, "losses", _F32, (2,), dev), _typed(counts, "counts", _I32, (E,), dev),
        _typed(tokens, "tokens", _I32, (1,), dev), ws, bytes_, _stream_of(dev))
    if status:
        _check(status, "moe_balance_loss")
    return losses, counts, tokens


def moe_balance_loss_backward(logits, counts, tokens, k: int, grad, mask=None, dlogits=None):
    """Gradient of grad[0] * losses[0] + grad[1] * losses[1] (grad fp32 [2] on
    the device) with respect to the logits, in their type; counts, tokens, k
    and mask as in the forward call."""
    dev = logits.get_device()
    bf16, lp = _logits(logits, dev)
    N, E = logits.shape
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    status = lib().moe_balance_loss_backward(
        lp, bf16, _typed(counts, "counts", _I32, (E,), dev),
        _typed(tokens, "tokens", _I32, (1,), dev), None if mask is None else _mask(mask, N, dev),
        _typed(grad, "grad", _F32, (2,), dev), N, E, k,
        _typed(dlogits, "dlogits", logits.dtype, (N, E), dev), _stream_of(dev))
    if status:
        _check(status, "moe_balance_loss_backward")
    return dlogits


def _activation(name):
    act = ACTIVATIONS.get(name)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}")
    return act


def moe_gated_ffn_workspace_bytes(N, H, I) -> int:
    return int(lib().moe_gated_ffn_workspace_bytes(N, H, I))


def moe_gated_ffn_backward_workspace_bytes(N, H, I) -> int:
    return int(lib().moe_gated_ffn_backward_workspace_bytes(N, H, I))


def _scratch(workspace, need, device, dev):
    """(pointer, bytes) of the workspace, one of `need` bytes if there is none."""
    if workspace is None:
        workspace = torch.empty(max(need(), 256), dtype=torch.uint8, device=device)
    bytes_ = workspace.numel()
    return workspace, _typed(workspace, "workspace", torch.uint8, (bytes_,), dev), bytes_


def moe_gated_ffn(x, w_gate, w_up, w_down, activation: str = "silu", residual=None, gate=None,
                  up=None, out=None, keep: bool = False, workspace=None):
    """(act(x Wg^T) * (x Wu^T)) Wd^T + residual: returns (out [N, H], gate, up).
    gate and up [N, I] are what moe_gated_ffn_backward needs; they are stored
    with ``keep`` or where tensors for them are given, else None.  x [N, H],
    w_gate and w_up [I, H], w_down [H, I], all bf16."""
    if x.dim() != 2:
        _matrix(x, "x")
    if w_gate.dim() != 2:
        _matrix(w_gate, "w_gate")
    shape = N, H = x.shape
    I = w_gate.shape[0]
    dev = x.get_device()
    act = _activation(activation)
    if keep or gate is not None or up is not None:
        if gate is None:
            gate = torch.empty((N, I), dtype=_BF16, device=x.device)
        if up is None:
            up = torch.empty((N, I), dtype=_BF16, device=x.device)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=x.device)
    xp = _typed(x, "x", _BF16, shape, dev)
    weights = (_typed(w_gate, "w_gate", _BF16, (I, H), dev),
               _typed(w_up, "w_up", _BF16, (I, H), dev),
               _typed(w_down, "w_down", _BF16, (H, I), dev))
    rp = None if residual is None else _typed(residual, "residual", _BF16, shape, dev)
    gp = None if gate is None else _typed(gate, "gate", _BF16, (N, I), dev)
    upp = None if up is None else _typed(up, "up", _BF16, (N, I), dev)
    op = _typed(out, "out", _BF16, shape, dev)
    stream = _stream_of(dev)
    workspace, ws, bytes_ = _scratch(
        workspace, lambda: lib().moe_gated_ffn_workspace_bytes(N, H, I), x.device, dev)
    status = lib().moe_gated_ffn(xp, *weights, rp, N, H, I, act, gp, upp, op, ws, bytes_, stream)
    if status:
        _check(status, "moe_gated_ffn")
    return out, gate, up


def moe_gated_ffn_backward(dout, x, w_gate, w_up, w_down, gate, up, activation: str = "silu",
                           dx=None, dw_gate=None, dw_up=None, dw_down=None,
                           want_dx: bool = True, want_dw: bool = True, workspace=None):
    """The gradients (dx, dw_gate, dw_up, dw_down) for the gradient dout of
    moe_gated_ffn's out, with the gate and up that it kept; those not wanted are
    None (the residual's gradient is dout itself)."""
    if x.dim() != 2:
        _matrix(x, "x")
    if w_gate.dim() != 2:
        _matrix(w_gate, "w_gate")
    shape = N, H = x.shape
    I = w_gate.shape[0]
    dev = x.get_device()
    act = _activation(activation)
    if dx is None and want_dx:
        dx = torch.empty(shape, dtype=_BF16, device=x.device)
    if want_dw:
        if dw_gate is None:
            dw_gate = torch.empty((I, H), dtype=_BF16, device=x.device)
        if dw_up is None:
            dw_up = torch.empty((I, H), dtype=_BF16, device=x.device)
        if dw_down is None:
            dw_down = torch.empty((H, I), dtype=_BF16, device=x.device)
    inputs = (_typed(dout, "dout", _BF16, shape, dev), _typed(x, "x", _BF16, shape, dev),
              _typed(w_gate, "w_gate", _BF16, (I, H), dev),
              _typed(w_up, "w_up", _BF16, (I, H), dev),
              _typed(w_down, "w_down", _BF16, (H, I), dev),
              _typed(gate, "gate", _BF16, (N, I), dev), _typed(up, "up", _BF16, (N, I), dev))
    outputs = (None if dx is None else _typed(dx, "dx", _BF16, shape, dev),
               None if dw_gate is None else _typed(dw_gate, "dw_gate", _BF16, (I, H), dev),
               None if dw_up is None else _typed(dw_up, "dw_up", _BF16, (I, H), dev),
               None if dw_down is None else _typed(dw_down, "dw_down", _BF16, (H, I), dev))
    stream = _stream_of(dev)
    workspace, ws, bytes_ = _scratch(
        workspace, lambda: lib().moe_gated_ffn_backward_workspace_bytes(N, H, I), x.device, dev)
    status = lib().moe_gated_ffn_backward(*inputs, N, H, I, act, *outputs, ws, bytes_, stream)
    if status:
        _check(status, "moe_gated_ffn_backward")
    return dx, dw_gate, dw_up, dw_down


def _bf16_or_fp32(t, name):
    if t.dtype is not _BF16 and t.dtype is not _F32:
        raise ValueError(f"{name} must be bf16 or fp32, got {t.dtype}")
    if t.dim() != 2:
        _matrix(t, name)
    return t.dtype


def moe_layernorm(x, weight, bias=None, residual=None, eps: float = 1e-5, out=None,
                  residual_out=None, mean=None, rstd=None):
    """r = x + residual in their type (x without a residual), out = (r - mean(r))
    / std(r) * weight + bias: returns (out [N, H], mean fp32 [N], rstd fp32 [N]).
    r goes to ``residual_out``, or without one back to ``residual``.  bf16 or
    fp32, the same for every array but the statistics."""
    dtype = _bf16_or_fp32(x, "x")
    shape = N, H = x.shape
    dev = x.get_device()
    if residual_out is None:
        residual_out = residual
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
    if mean is None:
        mean = torch.empty(N, dtype=_F32, device=x.device)
    if rstd is None:
        rstd = torch.empty(N, dtype=_F32, device=x.device)
    status = lib().moe_layernorm(
        _typed(x, "x", dtype, shape, dev),
        None if residual is None else _typed(residual, "residual", dtype, shape, dev),
        _typed(weight, "weight", dtype, (H,), dev),
        None if bias is None else _typed(bias, "bias", dtype, (H,), dev), dtype is _BF16, N, H,
        eps,
        None if residual_out is None else _typed(residual_out, "residual_out", dtype, shape, dev),
        _typed(out, "out", dtype, shape, dev), _typed(mean, "mean", _F32, (N,), dev),
        _typed(rstd, "rstd", _F32, (N,), dev), _stream_of(dev))
    if status:
        _check(status, "moe_layernorm")
    return out, mean, rstd


@functools.lru_cache(maxsize=256)
def _layernorm_backward_workspace_bytes(N, H, device):
    return int(lib().moe_layernorm_backward_workspace_bytes(N, H))


def moe_layernorm_backward_workspace_bytes(N, H) -> int:
    return int(lib().moe_layernorm_backward_workspace_bytes(N, H))


def moe_layernorm_backward(dout, x, weight, mean, rstd, dresidual=None, dx=None, dweight=None,
                           dbias=None, want_dbias: bool = True, workspace=None,
                           want_dx: bool = True, want_dweight: bool = True):
    """(dx [N, H], dweight fp32 [H], dbias fp32 [H]) for the gradient dout of
    moe_layernorm's out; those not wanted are None (without dweight and dbias no
    workspace is needed and none made).  x is what was normalised (the
    residual_out where there was a residual), dresidual the gradient that
    reaches it by the residual stream and is added to dx."""
    dtype = _bf16_or_fp32(x, "x")
    shape = N, H = x.shape
    dev = x.get_device()
    if dx is None and want_dx:
        dx = torch.empty(shape, dtype=dtype, device=x.device)
    if dweight is None and want_dweight:
        dweight = torch.empty(H, dtype=_F32, device=x.device)
    if dbias is None and want_dbias:
        dbias = torch.empty(H, dtype=_F32, device=x.device)
    inputs = (_typed(dout, "dout", dtype, shape, dev), _typed(x, "x", dtype, shape, dev),
              _typed(weight, "weight", dtype, (H,), dev), _typed(mean, "mean", _F32, (N,), dev),
              _typed(rstd, "rstd", _F32, (N,), dev),
              None if dresidual is None else _typed(dresidual, "dresidual", dtype, shape, dev))
    outputs = (None if dx is None else _typed(dx, "dx", dtype, shape, dev),
               None if dweight is None else _typed(dweight, "dweight", _F32, (H,), dev),
               None if dbias is None else _typed(dbias, "dbias", _F32, (H,), dev))
    stream = _stream_of(dev)
    ws, bytes_ = None, 0
    if workspace is not None or dweight is not None or dbias is not None:
        workspace, ws, bytes_ = _scratch(
            workspace, lambda: _layernorm_backward_workspace_bytes(N, H, dev), x.device, dev)
    status = lib().moe_layernorm_backward(*inputs, dtype is _BF16, N, H, *outputs, ws, bytes_,
                                          stream)
    if status:
        _check(status, "moe_layernorm_backward")
    return dx, dweight, dbias


_data_ptr = torch.Tensor.data_ptr


class GradSet:
    """Gradient tensors as moe_grad_norm and moe_clip_grads take them, for a
    program that keeps its gradients where they are: checked once, here, instead
    of on every call.  ``grads``: contiguous bf16 and fp32 CUDA tensors of one
    device; ``out``: where the clipped ones go, as many tensors of the same
    numbers of values (either type), or None: in place.  The set keeps the
    tensors; they keep their storage, size and type as long as it is used.  Every
    call looks where they are (4 us for 60 tensors) and refuses a set of which
    one has moved."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        if len(self.out) != len(self.grads):
            raise ValueError(f"out must have as many tensors as grads ({len(self.grads)}), got "
                             f"{len(self.out)}")
        self.device = self.grads[0].device if self.grads else None
        self.index = self.grads[0].get_device() if self.grads else -1
        self._sizes = array.array("q", [t.numel() for t in self.grads])
        self._src, self._src_bf16 = self._pointers(self.grads, "grads")
        self._dst, self._dst_bf16 = self._src, self._src_bf16
        if self.out is not self.grads:
            for i, (g, o) in enumerate(zip(self.grads, self.out)):
                if g.numel() != o.numel():
                    raise ValueError(f"out[{i}] must have {g.numel()} values like grads[{i}], "
                                     f"got {o.numel()}")
            self._dst, self._dst_bf16 = self._pointers(self.out, "out")
        self._check_overlaps()
        self._places = self._src.tolist()
        self._out_places = self._dst.tolist()
        n = len(self.grads)
        self._norm_args = (self._src.buffer_info()[0], self._sizes.buffer_info()[0],
                           self._src_bf16, n)
        self._out_args = (self._dst.buffer_info()[0], self._dst_bf16)

    def _pointers(self, tensors, name):
        for i, t in enumerate(tensors):
            if ((t.dtype is not _BF16 and t.dtype is not _F32) or not t.is_contiguous()
                    or not t.get_device() == self.index >= 0):
                raise ValueError(
                    f"{name}[{i}] must be a contiguous bf16 or fp32 CUDA tensor"
                    f"{f' on cuda:{self.index} like the first' if self.index >= 0 else ''}, got "
                    f"{t.dtype} on {t.device}{'' if t.is_contiguous() else ', not contiguous'}")
        return (array.array("Q", [t.data_ptr() for t in tensors]),
                bytes([t.dtype is _BF16 for t in tensors]))

    def _check_places(self, out):
        """The gradients, and with `out` the clipped ones, are where they were."""
        if list(map(_data_ptr, self.grads)) != self._places:
            self._moved(self.grads, self._places, "grads")
        if (out and self.out is not self.grads
                and list(map(_data_ptr, self.out)) != self._out_places):
            self._moved(self.out, self._out_places, "out")

    def _moved(self, tensors, places, name):
        if len(tensors) != len(places):
            raise ValueError(f"{name} has {len(tensors)} tensors instead of {len(places)}: make a "
                             "new GradSet")
        i = next(i for i, (t, p) in enumerate(zip(tensors, places)) if _data_ptr(t) != p)
        raise ValueError(f"{name}[{i}] has another storage than when the GradSet was made: make a "
                         "new one")

    def _check_overlaps(self):
        """No output may lie in another tensor (its own gradient apart)."""
        spans = []
        for i, n in enumerate(self._sizes):
            if n == 0:
                continue
            dst, src = self._dst[i], self._src[i]
            spans.append((dst, dst + n * (2 if self._dst_bf16[i] else 4), True, i))
            if src != dst or self._src_bf16[i] != self._dst_bf16[i]:
                spans.append((src, src + n * (2 if self._src_bf16[i] else 4), False, i))
        spans.sort()
        far_out = far = (0, 0, False, -1)  # the spans that reach farthest so far
        for s in spans:
            if s[0] < far_out[1] or (s[2] and s[0] < far[1]):
                other = far_out if s[0] < far_out[1] else far
                raise ValueError(f"tensors {other[3]} and {s[3]} overlap: a clipped gradient may "
                                 "lie in its own gradient only")
            if s[1] > far[1]:
                far = s
            if s[2] and s[1] > far_out[1]:
                far_out = s


def _grad_set(grads, clips, out=None):
    if isinstance(grads, GradSet):
        if out is not None:
            raise ValueError("a GradSet has its out tensors already")
        grads._check_places(clips)
        return grads
    return GradSet(grads, out)


def moe_grad_norm_workspace_bytes(n) -> int:
    return int(lib().moe_grad_norm_workspace_bytes(n))


@functools.lru_cache(maxsize=256)
def _grad_norm_workspace_bytes(n, device):
    return int(lib().moe_grad_norm_workspace_bytes(n))


def moe_grad_norm(grads, norm=None, workspace=None):
    """sqrt of the sum of squares of all values of the tensors (a GradSet, or a
    sequence of bf16 and fp32 CUDA tensors): norm fp32 [1], on the device."""
    g = _grad_set(grads, False)
    if not g.grads:
        raise ValueError("grads must have at least one tensor")
    if norm is None:
        norm = torch.empty(1, dtype=_F32, device=g.device)
    n = len(g.grads)
    np_ = _typed(norm, "norm", _F32, (1,), g.index)
    stream = _stream_of(g.index)
    workspace, ws, bytes_ = _scratch(
        workspace, lambda: _grad_norm_workspace_bytes(n, g.index), g.device, g.index)
    status = lib().moe_grad_norm(*g._norm_args, np_, ws, bytes_, stream)
    if status:
        _check(status, "moe_grad_norm")
    return norm


def moe_clip_grads(grads, norm, max_norm: float, out=None):
    """The tensors scaled by max_norm / norm where norm (moe_grad_norm's, on the
    device) is above max_norm, in place or to ``out`` (bf16 or fp32, whatever the
    gradients are); returns the list of scaled tensors."""
    g = _grad_set(grads, True, out)
    if not g.grads:
        return []
    status = lib().moe_clip_grads(*g._norm_args, _typed(norm, "norm", _F32, (1,), g.index),
                                  max_norm, *g._out_args, _stream_of(g.index))
    if status:
        _check(status, "moe_clip_grads")
    return g.out


def moe_dense_mlp(x, w_gate, w_up, w_down, out=None, workspace=None):
    """Dense SwiGLU MLP (silu(x Wg^T) * (x Wu^T)) Wd^T on the grouped GEMM
    kernels; w_down bf16 (moe_dense_mlp) or its fp16 copy (_prepared)."""
    N, H = x.shape
    I = w_gate.shape[0]
    _bf16(x, "x")
    _bf16(w_gate, "w_gate", (I, H))
    _bf16(w_up, "w_up", (I, H))
    prepared = _down(w_down, "w_down", (H, I))
    if out is None:
        out = torch.empty((N, H), dtype=torch.bfloat16, device=x.device)
    _bf16(out, "out", (N, H))
    L = lib()
    if workspace is None:
        workspace = torch.empty(max(int(L.moe_dense_mlp_workspace_bytes(N, H, I)), 256),
                                dtype=torch.uint8, device=x.device)
    fn = L.moe_dense_mlp_prepared if prepared else L.moe_dense_mlp
    _check(fn(_ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), N, H, I, _ptr(out),
              _ptr(workspace), workspace.numel(), _stream()), "moe_dense_mlp")
    return out


def moe_experts(x_rows, ids, weights, w_gate, w_up, w_down, y=None, workspace=None):
    """Per-row expert outputs y[r] = weights[r] * Expert_{ids[r]}(x_rows[r]) as
    pair rows (``(hi bf16 [R, H], res int8 [R, H])``, the format moe.h
    describes): the receiving side of expert-parallel dispatch.  w_down bf16
    (moe_experts) or its fp16 copy (moe_experts_prepared).  Returns (y,
    workspace)."""
    R, H = x_rows.shape
    E, I, _ = w_gate.shape
    _bf16(x_rows, "x_rows")
    _bf16(w_gate, "w_gate", (E, I, H))
    _bf16(w_up, "w_up", (E, I, H))
    prepared = _down(w_down, "w_down", (E, H, I))
    if ids.dtype != torch.int32 or not ids.is_cuda or tuple(ids.shape) != (R,):
        raise ValueError("ids must be a CUDA int32 tensor of shape [R]")
    if weights.dtype != torch.float32 or not weights.is_cuda or tuple(weights.shape) != (R,):
        raise ValueError("weights must be a CUDA float32 tensor of shape [R]")
    ids, weights = ids.contiguous(), weights.contiguous()
    if y is None:
        y = alloc_pair_rows(R, H, x_rows.device)
    _check_pair_rows(y, R, H, "y")
    if workspace is None:
        workspace = torch.empty(max(lib().moe_experts_workspace_bytes(R, H, E, I), 256),
                                dtype=torch.uint8, device=x_rows.device)
    fn = lib().moe_experts_prepared if prepared else lib().moe_experts
    _check(fn(_ptr(x_rows), _ptr(ids), _ptr(weights), R, H, E, I, _ptr(w_gate), _ptr(w_up),
              _ptr(w_down), _ptr(y[0]), _ptr(y[1]), _ptr(workspace), workspace.numel(),
              _stream()), "moe_experts")
    return y, workspace


def alloc_pair_rows(R: int, H: int, device="cuda"):
    """Empty pair rows of [R, H] values: (hi bf16 [R, H], res int8 [R, H])."""
    return (torch.empty((R, H), dtype=torch.bfloat16, device=device),
            torch.empty((R, H), dtype=torch.int8, device=device))


def _check_pair_rows(y, R, H, name):
    hi, res = y
    if (hi.dtype != torch.bfloat16 or res.dtype != torch.int8 or tuple(hi.shape) != (R, H)
            or tuple(res.shape) != (R, H) or not hi.is_contiguous() or not res.is_contiguous()
            or not hi.is_cuda or not res.is_cuda):
        raise ValueError(f"{name} must be pair rows: (bf16 [{R}, {H}], int8 [{R}, {H}]) "
                         "contiguous CUDA tensors")


def _shared_rows(yshared, N, H):
    """(planes, S) of the shared expert's pair rows [N*S, H] (S rows per
    token, moe_shared_expert's output), or ((None, None), 0)."""
    if yshared is None:
        return (None, None), 0
    rows = yshared[0].shape[0]
    if N == 0 or rows % N or rows == 0:
        raise ValueError("yshared must hold S >= 1 rows per token ([N*S, H])")
    _check_pair_rows(yshared, rows, H, "yshared")
    return yshared, rows // N


def moe_combine(ypair, N: int, k: int, yshared=None, out=None):
    """out[n] = bf16(sum_j ypair[n*k + j] + sum_c yshared[n*S + c]) in fp32,
    slot order; ypair and yshared are pair rows (hi, res), yshared (optional)
    with S rows per token (moe_shared_expert's chunks)."""
    H = ypair[0].shape[1]
    _check_pair_rows(ypair, N * k, H, "ypair")
    sh, S = _shared_rows(yshared, N, H)
    if out is None:
        out = torch.empty((N, H), dtype=torch.bfloat16, device=ypair[0].device)
    _bf16(out, "out", (N, H))
    _check(lib().moe_combine(_ptr(ypair[0]), _ptr(ypair[1]), _ptr(sh[0]), _ptr(sh[1]), S, N, H,
                             k, _ptr(out), _stream()), "moe_combine")
    return out


def moe_combine_indexed(yrows, row_index, N: int, k: int, yshared=None, out=None):
    """moe_combine over pair rows in another order: pair p reads row
    row_index[p] of yrows (pair rows (hi, res), [R, H]); an index outside
    [0, R) contributes nothing."""
    R, H = yrows[0].shape
    _check_pair_rows(yrows, R, H, "yrows")
    if (row_index.dtype != torch.int32 or tuple(row_index.shape) != (N * k,) or
            not row_index.is_cuda or not row_index.is_contiguous()):
        raise ValueError("row_index must be a contiguous int32 CUDA tensor of shape [N*k]")
    sh, S = _shared_rows(yshared, N, H)
    if out is None:
        out = torch.empty((N, H), dtype=torch.bfloat16, device=row_index.device)
    _bf16(out, "out", (N, H))
    _check(lib().moe_combine_indexed(_ptr(yrows[0]), _ptr(yrows[1]), R, _ptr(row_index),
                                     _ptr(sh[0]), _ptr(sh[1]), S, N, H, k, _ptr(out),
                                     _stream()),
           "moe_combine_indexed")
    return out


def moe_shared_chunks(I: int, I_s: int) -> int:
    """C = ceil(I_s / I): the chunks (virtual experts) of the shared expert."""
    return int(lib().moe_shared_chunks(I, I_s))


def moe_shared_expert(x, gamma, I: int, shared_gate_proj, shared_up_proj, shared_down_proj,
                      y=None, workspace=None):
    """The gated shared expert on its own, as moe_forward computes it: pair
    rows [N*C, H], row n*C + c = gamma[n] * (chunk c of SharedMLP)(x[n]), C =
    ceil(I_s / I) with I the routed experts' intermediate size (moe.h).
    shared_down_proj bf16 or its fp16 copy.  Returns (y, workspace)."""
    N, H = x.shape
    I_s = shared_gate_proj.shape[0]
    _bf16(x, "x")
    _bf16(shared_gate_proj, "shared_gate_proj", (I_s, H))
    _bf16(shared_up_proj, "shared_up_proj", (I_s, H))
    prepared = _down(shared_down_proj, "shared_down_proj", (H, I_s))
    if gamma.dtype != torch.float32 or not gamma.is_cuda or tuple(gamma.shape) != (N,):
        raise ValueError("gamma must be a CUDA float32 tensor of shape [N]")
    gamma = gamma.contiguous()
    C = moe_shared_chunks(I, I_s)
    if y is None:
        y = alloc_pair_rows(N * C, H, x.device)
    _check_pair_rows(y, N * C, H, "y")
    if workspace is None:
        workspace = torch.empty(max(lib().moe_shared_expert_workspace_bytes(N, H, I, I_s), 256),
                                dtype=torch.uint8, device=x.device)
    fn = lib().moe_shared_expert_prepared if prepared else lib().moe_shared_expert
    _check(fn(_ptr(x), _ptr(gamma), N, H, I, I_s, _ptr(shared_gate_proj), _ptr(shared_up_proj),
              _ptr(shared_down_proj), _ptr(y[0]), _ptr(y[1]), _ptr(workspace), workspace.numel(),
              _stream()), "moe_shared_expert")
    return y, workspace


def moe_ep_dispatch(x, topk_ids, topk_w, E: int, world: int):
    """The sending side of expert-parallel dispatch on the device (moe.h):
    returns a dict with send_x [N*k, H] bf16, send_ids [N*k] int32 (local
    expert ids), send_w [N*k] fp32, send_counts [world] int32 (device),
    inv_order [N*k] int32 and the workspace (status word first)."""
    N, H = x.shape
    _bf16(x, "x")
    k = topk_ids.shape[1]
    if topk_ids.dtype != torch.int32 or tuple(topk_ids.shape) != (N, k) or not topk_ids.is_cuda:
        raise ValueError("topk_ids must be an int32 CUDA tensor of shape [N, k]")
    if topk_w.dtype != torch.float32 or tuple(topk_w.shape) != (N, k) or not topk_w.is_cuda:
        raise ValueError("topk_w must be a float32 CUDA tensor of shape [N, k]")
    topk_ids, topk_w = topk_ids.contiguous(), topk_w.contiguous()
    dev = x.device
    P = N * k
    r = {"send_x": torch.empty((P, H), dtype=torch.bfloat16, device=dev),
         "send_ids": torch.empty(P, dtype=torch.int32, device=dev),
         "send_w": torch.empty(P, dtype=torch.float32, device=dev),
         "send_counts": torch.zeros(world, dtype=torch.int32, device=dev),
         "inv_order": torch.empty(P, dtype=torch.int32, device=dev)}
    L = lib()
    wsb = int(L.moe_ep_dispatch_workspace_bytes(N, k, world))
    r["workspace"] = torch.empty(max(wsb, 256), dtype=torch.uint8, device=dev)
    _check(L.moe_ep_dispatch(_ptr(x), _ptr(topk_ids), _ptr(topk_w), N, H, k, E, world,
                             _ptr(r["send_x"]), _ptr(r["send_ids"]), _ptr(r["send_w"]),
                             _ptr(r["send_counts"]), _ptr(r["inv_order"]), _ptr(r["workspace"]),
                             r["workspace"].numel(), _stream()), "moe_ep_dispatch")
    return r


def convert_bf16_to_f16(src, out=None, status=None):
    """fp16 copy of a bf16 CUDA tensor (round to nearest even; exact for
    |v| >= 2^-14).  ``status`` (int32 CUDA tensor, optional) receives
    MOE_ERR_DEVICE_CHECK when a value exceeds fp16's range or is NaN."""
    if src.dtype != torch.bfloat16 or not src.is_cuda or not src.is_contiguous():
        raise ValueError("src must be a contiguous bf16 CUDA tensor")
    if out is None:
        out = torch.empty(src.shape, dtype=torch.float16, device=src.device)
    _f16(out, "out", src.shape)
    _check(lib().moe_convert_bf16_to_f16(_ptr(src), _ptr(out), src.numel(), _ptr(status),
                                         _stream()), "moe_convert_bf16_to_f16")
    return out


DOWN_KEYS = ("w_down", "shared_down_proj")


def prepare_weights(weights: dict) -> dict:
    """The layer's weights in the form the *_prepared entry points take: the
    same dict with the down projections (w_down, shared_down_proj) converted
    to fp16 once; bf16 entries pass through.  Raises if a down weight is
    outside fp16's range."""
    out = dict(weights)
    dev = next(t.device for t in weights.values() if torch.is_tensor(t))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    for name in DOWN_KEYS:
        if name in weights and weights[name].dtype == torch.bfloat16:
            out[name] = convert_bf16_to_f16(weights[name], status=status)
    code = int(status.item())
    if code != MOE_OK:
        raise MoEError(code, "prepare_weights: a down-projection weight exceeds fp16's range")
    return out


def moe_forward_from_host(x_host, out_host, x_dev, out_dev, weights: dict, k: int,
                          norm_topk_prob: bool, workspace):
    """End-to-end call with host buffers through moe_forward_host: x (pinned
    host) is copied to the device staging buffer x_dev, the layer runs, and
    the result is copied from out_dev back to pinned host memory, all on the
    current stream.  Weights stay resident on the device."""
    N, H = x_host.shape
    E, I, _ = weights["w_gate"].shape
    if x_host.is_cuda or out_host.is_cuda:
        raise ValueError("x_host and out_host must be host tensors")
    if x_host.dtype != torch.bfloat16 or out_host.dtype != torch.bfloat16:
        raise ValueError("x_host and out_host must be bf16")
    if not (x_host.is_contiguous() and out_host.is_contiguous()) or out_host.shape != (N, H):
        raise ValueError("x_host and out_host must be contiguous [N, H]")
    _bf16(x_dev, "x_dev", (N, H))
    _bf16(out_dev, "out_dev", (N, H))
    prepared = _down(weights["w_down"], "w_down", (E, H, I))
    shared = "shared_gate" in weights
    if shared and _down(weights["shared_down_proj"], "shared_down_proj") != prepared:
        raise ValueError("w_down and shared_down_proj must both be bf16 or both fp16")
    sp = [weights[n] if shared else None for n in SHARED_KEYS]
    I_s = weights["shared_gate_proj"].shape[0] if shared else 0
    fn = lib().moe_forward_host_prepared if prepared else lib().moe_forward_host
    _check(fn(x_host.data_ptr(), out_host.data_ptr(), _ptr(x_dev), _ptr(out_dev),
              _ptr(weights["router"]), _ptr(weights["w_gate"]), _ptr(weights["w_up"]),
              _ptr(weights["w_down"]), *[_ptr(t) for t in sp], N, H, E, I, I_s, k,
              int(bool(norm_topk_prob)), _ptr(workspace), workspace.numel(), _stream()),
           "moe_forward_host")
    return out_host


class ForwardGraph:
    """moe_forward captured once in a CUDA graph for a token bucket of
    `bucket` rows, then replayed: the serving decode loop's way of removing
    per-step launch cost.  A batch of n <= bucket tokens is copied into the
    first n rows of the static input (the rest zero); since every token's
    result is independent of the others, out[:n] equals an eager call on the
    n tokens bit for bit."""

    def __init__(self, weights: dict, k: int, norm_topk_prob: bool, bucket: int):
        dev = weights["router"].device
        H = weights["router"].shape[1]
        E, I, _ = weights["w_gate"].shape
        self.shared = ({n: weights[n] for n in SHARED_KEYS} if "shared_gate" in weights
                       else None)
        I_s = self.shared["shared_gate_proj"].shape[0] if self.shared else 0
        self.w, self.k, self.norm, self.bucket = weights, k, norm_topk_prob, bucket
        self.x = torch.zeros((bucket, H), dtype=torch.bfloat16, device=dev)
        self.out = torch.empty((bucket, H), dtype=torch.bfloat16, device=dev)
        self.ws = alloc_workspace(bucket, H, E, I, k, I_s, dev)
        side = torch.cuda.Stream(device=dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            for _ in range(2):
                self._call()
        torch.cuda.current_stream(dev).wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self._call()

    def _call(self):
        w = self.w
        moe_forward(self.x, w["router"], w["w_gate"], w["w_up"], w["w_down"], self.k, self.norm,
                    self.shared, out=self.out, workspace=self.ws)

    def __call__(self, x):
        n = x.shape[0]
        if n > self.bucket:
            raise ValueError(f"{n} tokens exceed the graph's bucket of {self.bucket}")
        self.x[:n].copy_(x)
        if n < self.bucket:
            self.x[n:].zero_()
        self.graph.replay()
        return self.out[:n]


DECODE_BUCKETS = (1, 2, 4, 8, 16, 32, 64, 128)


class ForwardGraphSet:
    """The layer captured once per token bucket (1, 2, 4, ... 128 by default)
    and replayed for the smallest bucket that holds each step's batch: the
    decode loop of a serving engine, whose batch size changes from step to
    step, without per-step launch cost (the Nano-vLLM notes' model runner
    captures its decode step for a ladder of batch sizes the same way).

    Every bucket's graph reads the first b rows of one static input and
    writes the first b rows of one static output, and all of them use one
    workspace sized for the largest bucket: replays on one stream never
    overlap, and each graph carries its own workspace layout.  A batch of
    n tokens is copied into the input's first n rows (rows n..b-1 zeroed);
    since every token's result is independent of the others, the first n
    output rows equal an eager call on the n tokens bit for bit."""

    def __init__(self, weights: dict, k: int, norm_topk_prob: bool,
                 buckets=DECODE_BUCKETS):
        self.buckets = tuple(sorted(set(int(b) for b in buckets)))
        if not self.buckets or self.buckets[0] < 1:
            raise ValueError("buckets must be positive token counts")
        dev = weights["router"].device
        H = weights["router"].shape[1]
        E, I, _ = weights["w_gate"].shape
        self.shared = ({n: weights[n] for n in SHARED_KEYS} if "shared_gate" in weights
                       else None)
        I_s = self.shared["shared_gate_proj"].shape[0] if self.shared else 0
        self.w, self.k, self.norm = weights, k, norm_topk_prob
        top = self.buckets[-1]
        self.x = torch.zeros((top, H), dtype=torch.bfloat16, device=dev)
        self.out = torch.empty((top, H), dtype=torch.bfloat16, device=dev)
        self.ws = torch.empty(max(max(moe_forward_workspace_bytes(b, H, E, I, k, I_s)
                                      for b in self.buckets), 256),
                              dtype=torch.uint8, device=dev)
        self.graphs = {}
        side = torch.cuda.Stream(device=dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            for b in self.buckets:  # warm every shape once before capture
                self._call(b)
        torch.cuda.current_stream(dev).wait_stream(side)
        for b in self.buckets:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self._call(b)
            self.graphs[b] = g

    def _call(self, b):
        w = self.w
        moe_forward(self.x[:b], w["router"], w["w_gate"], w["w_up"], w["w_down"], self.k,
                    self.norm, self.shared, out=self.out[:b], workspace=self.ws)

    def bucket_of(self, n: int) -> int:
        for b in self.buckets:
            if b >= n:
                return b
        raise ValueError(f"{n} tokens exceed the largest bucket ({self.buckets[-1]})")

    def __call__(self, x):
        """out[:n] for this step's x [n, H] (a view of the static output,
        valid until the next call)."""
        n = x.shape[0]
        if n == 0:
            return self.out[:0]
        b = self.bucket_of(n)
        self.x[:n].copy_(x)
        if n < b:
            self.x[n:b].zero_()
        self.graphs[b].replay()
        return self.out[:n]

    def read_device_status(self) -> int:
        """Status word of the last replay (synchronises the stream)."""
        return moe_read_device_status(self.ws)


def decode_loop(graphs: ForwardGraphSet, steps):
    """Runs a multi-step decode: for each step's activations x_t [n_t, H]
    (n_t may change from step to step), the MoE layer by graph replay.
    Returns the per-step outputs (copies) and raises if a kernel recorded a
    device-side failure."""
    outs = [graphs(x).clone() for x in steps]
    status = graphs.read_device_status()
    if status != MOE_OK:
        raise MoEError(status, f"decode loop: {moe_status_string(status)}")
    return outs


def workspace_views(workspace, N, H, E, I, k, I_s=0) -> dict:
    """Typed views of moe_forward's intermediate buffers inside ``workspace``.

    With the shared expert every token has ``slots`` = k + C slots (the
    routed ones, then the shared expert's C chunks as virtual experts E + c)
    grouped over ``groups`` = E + C experts; topk_w / topk_ids / ypair hold
    all slots, ``routed_w`` / ``routed_ids`` only the first k."""
    lay = moe_forward_layout(N, H, E, I, k, I_s)
    cap = lay["capacity"]
    slots, groups = lay["slots"], lay["groups"]
    P = N * slots
    base = workspace

    def view(off, dtype, shape):
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return base[off:off + nbytes].view(dtype).view(shape)

    v = {
        "slots": slots,
        "groups": groups,
        "status": view(lay["status"], torch.int32, (1,)),
        "topk_w": view(lay["topk_w"], torch.float32, (N, slots)),
        "topk_ids": view(lay["topk_ids"], torch.int32, (N, slots)),
        "counts": view(lay["counts"], torch.int32, (groups,)),
        "offsets": view(lay["offsets"], torch.int32, (groups + 1,)),
        "pad_offsets": view(lay["pad_offsets"], torch.int32, (groups + 1,)),
        "num_padded": view(lay["num_padded"], torch.int32, (1,)),
        "sorted_pair": view(lay["sorted_pair"], torch.int32, (cap,)),
        "block_expert": view(lay["block_expert"], torch.int32, (cap // MOE_BLOCK_M,)),
        "x_sorted": view(lay["x_sorted"], torch.bfloat16, (cap, H)),
        # the activation: a bf16 hi/lo pair (bf16 down weights) or fp16
        # (prepared fp16 down weights), in the same bytes
        "act_hi": view(lay["act"], torch.bfloat16, (cap, I)),
        "act_lo": view(lay["act"] + 2 * cap * I, torch.bfloat16, (cap, I)),
        "act_f16": view(lay["act"], torch.float16, (cap, I)),
        # pair rows (hi, res) of w * Expert(x), one row per slot
        "ypair": (view(lay["ypair"], torch.bfloat16, (P, H)),
                  view(lay["ypair_res"], torch.int8, (P, H))),
    }
    v["routed_w"] = v["topk_w"][:, :k]
    v["routed_ids"] = v["topk_ids"][:, :k]
    if I_s:
        v["gamma"] = view(lay["gamma"], torch.float32, (N,))
    return v


def moe_selftest_wait_timeout(workspace, limit_ns: int) -> None:
    """Enqueue the device wait-timeout self-check (see moe.h)."""
    _check(lib().moe_selftest_wait_timeout(_ptr(workspace), workspace.numel(), int(limit_ns),
                                           _stream()), "moe_selftest_wait_timeout")


def moe_read_device_status(workspace) -> int:
    """Synchronise the current stream and return the workspace's status word."""
    return int(lib().moe_read_device_status(_ptr(workspace), _stream()))


def set_stage_events(events) -> None:
    """Record the given torch.cuda.Event objects (None entries skipped) around
    the stages of the next moe_forward calls on this thread (None to stop)."""
    L = lib()
    if events is None:
        _check(L.moe_set_stage_events(None, 0), "moe_set_stage_events")
        return
    if len(events) != MOE_NUM_STAGES + 1:
        raise ValueError(f"need {MOE_NUM_STAGES + 1} events")
    for e in events:
        if e is not None and not e.cuda_event:  # torch creates it on first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(
        *[ctypes.c_void_p(e.cuda_event if e is not None else None) for e in events])
    _check(L.moe_set_stage_events(arr, len(events)), "moe_set_stage_events")
