"""Parts of the layer norm's gradients through the library's own entry point, where
any of the three outputs may be NULL.  What is wanted has the bits of the call
that asks for all of it (which test_gpu_layernorm.py holds to the formulas), and
what is not wanted is not touched: neither a workspace that the call may not use
nor its surroundings."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding
from test_gpu_layernorm import BF16, F32, check, gen, normal

pytestmark = pytest.mark.gpu


def inputs(N, H, dtype):
    g = gen(N + H)
    x, dy, dr = (normal(g, N, H, dtype=dtype) for _ in range(3))
    w = normal(g, H, dtype=dtype) + 1
    _, mean, rstd = binding.moe_layernorm(x, w)
    return dy, x, w, mean, rstd, dr


def call(ins, dx, dw, db, ws, ws_bytes):
    """The C entry point; returns its launches."""
    dy, x, w, mean, rstd, dr = ins
    N, H = x.shape
    p = [None if t is None else t.data_ptr() for t in (*ins[:5], dr, dx, dw, db, ws)]
    before = binding.moe_kernel_launch_count()
    status = binding.lib().moe_layernorm_backward(
        *p[:6], int(x.dtype is BF16), N, H, *p[6:], ws_bytes,
        torch.cuda.current_stream().cuda_stream)
    assert status == 0
    return binding.moe_kernel_launch_count() - before


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("H", [1, 64, 100, 1111, 2048, 4096, 4099, 8192])
@pytest.mark.parametrize("N", [1, 701])
def test_parts_of_the_gradients(N, H, dtype):
    check(N, H, dtype)
    ins = inputs(N, H, dtype)
    dx, dw, db = binding.moe_layernorm_backward(*ins)
    need = binding.moe_layernorm_backward_workspace_bytes(N, H)

    # dx alone: no workspace, or the start of one that is too small for sums
    got = torch.full_like(dx, 7.0)
    assert call(ins, got, None, None, None, 0) == 1
    assert torch.equal(got, dx)
    room = torch.full((2 * need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    got = torch.full_like(dx, 7.0)
    assert call(ins, got, None, None, room[1024:], 256) == 1
    assert torch.equal(got, dx) and bool((room == 0x5A).all())

    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for want_dx in (False, True):
        for want in ("w", "b", "wb"):
            gx = torch.full_like(dx, 7.0) if want_dx else None
            gw = torch.full_like(dw, 7.0) if "w" in want else None
            gb = torch.full_like(db, 7.0) if "b" in want else None
            call(ins, gx, gw, gb, ws, need)
            for a, b in ((gx, dx), (gw, dw), (gb, db)):
                assert a is None or torch.equal(a, b)


def test_dx_alone_in_place_and_captured():
    for H in (1000, 9000):
        ins = inputs(333, H, BF16)
        dx, _, _ = binding.moe_layernorm_backward(*ins)
        for which in (0, 1, 5):
            again = [t.clone() for t in ins]
            call(again, again[which], None, None, None, 0)
            assert torch.equal(again[which], dx)
        got = torch.zeros_like(dx)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call(ins, got, None, None, None, 0)
        torch.cuda.current_stream().wait_stream(s)
        got.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(ins, got, None, None, None, 0)
        graph.replay()
        assert torch.equal(got, dx)


@pytest.mark.parametrize("H", [100, 2048, 8192])
def test_parts_by_the_wrapper(H):
    ins = inputs(77, H, BF16)
    both = binding.moe_layernorm_backward(*ins)
    for want in range(8):
        which = [bool(want & 1), bool(want & 2), bool(want & 4)]
        before = torch.cuda.memory_stats()["allocation.all.allocated"]
        got = binding.moe_layernorm_backward(*ins, want_dx=which[0], want_dweight=which[1],
                                             want_dbias=which[2])
        made = torch.cuda.memory_stats()["allocation.all.allocated"] - before
        for g, b, w in zip(got, both, which):
            assert torch.equal(g, b) if w else g is None
        # the outputs, and a workspace where sums are wanted
        assert made == sum(which) + (which[1] or which[2])
    dw = torch.zeros_like(both[1])
    got = binding.moe_layernorm_backward(*ins, dweight=dw, want_dx=False, want_dweight=False,
                                         want_dbias=False)
    assert got[0] is None and got[1] is dw and got[2] is None and torch.equal(dw, both[1])
