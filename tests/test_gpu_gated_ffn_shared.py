"""The gated feed-forward block's products whose last wave of tiles is shared: pairs
take equal runs of the tiles' K slices, and a second kernel joins the partial sums.
That it is shared here, on a device of 148 or 152 SMs, shows in the launches: one
more per shared product."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding
from test_gpu_gated_ffn import (BF16, act64, assert_close, check_forward, gen, inputs, normal,
                                product, rounded)

pytestmark = pytest.mark.gpu


def launches(call):
    before = binding.moe_kernel_launch_count()
    out = call()
    return binding.moe_kernel_launch_count() - before, out


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("N,H,I", [(600, 72, 16384),      # all tiles shared, 128 columns
                                   (600, 520, 12288),     # the same, several tiles a run
                                   (5000, 1032, 4096),    # whole tiles first, 256 columns
                                   (5003, 1000, 4104)])   # the same, odd sizes
def test_down_step_joined(N, H, I, residual):
    count, _ = launches(lambda: check_forward(N, H, I, "silu", residual=residual, keep=False))
    assert count == 3  # gate/up, down, its join


def test_down_step_joined_in_place():
    N, H, I = 5000, 1032, 4096
    x, wg, wu, wd, res = inputs(N, H, I, 3)
    want, _, _ = binding.moe_gated_ffn(x, wg, wu, wd, residual=res)
    count, _ = launches(lambda: binding.moe_gated_ffn(x, wg, wu, wd, residual=res, out=res))
    assert count == 3 and torch.equal(res, want)
    want, _, _ = binding.moe_gated_ffn(x, wg, wu, wd, residual=x)
    binding.moe_gated_ffn(x, wg, wu, wd, residual=x, out=x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("N,H,I,dx_joined,dw_joined",
                         [(5000, 1032, 4096, True, True),   # whole tiles first, 256 columns
                          (600, 72, 16384, True, False),    # dx: all tiles shared
                          (20011, 72, 520, False, True)])   # dW: all tiles shared
def test_gradients_joined(N, H, I, dx_joined, dw_joined):
    """dx alone and the weights alone, so that each has a launch of its own."""
    x, wg, wu, wd, _ = inputs(N, H, I, 1)
    g = gen(N)
    dout, gate, up = normal(g, N, H, std=0.1), normal(g, N, I), normal(g, N, I)
    ins = (dout, x, wg, wu, wd, gate, up, "gelu")
    count, got = launches(lambda: binding.moe_gated_ffn_backward(*ins, want_dw=False))
    assert count == 2 + dx_joined  # dh, dx
    dx = got[0]
    count, got = launches(lambda: binding.moe_gated_ffn_backward(*ins, want_dx=False))
    assert count == 2 + dw_joined  # dh, the weights' gradients
    _, dwg, dwu, dwd = got

    gd, ud = gate.double(), up.double()
    a, slope = act64(gd, "gelu")
    ea, es = 2.0 ** -20 * gd.abs(), 2.0 ** -20 * torch.ones_like(gd)
    h = a * ud
    eh = rounded(h, ud.abs() * ea + 2.0 ** -24 * h.abs())
    dh, edh = product(dout.double(), wd.double().T)
    dg = dh * ud * slope
    edg = ud.abs() * (slope.abs() * edh + (dh.abs() + edh) * es) + 3 * 2.0 ** -24 * dg.abs()
    edg = rounded(dg, edg)
    du = dh * a
    edu = rounded(du, (a.abs() + ea) * edh + dh.abs() * ea + 2.0 ** -24 * du.abs())
    r, e = product(torch.cat([dg, du], 1), torch.cat([wg.double().T, wu.double().T], 1),
                   torch.cat([edg, edu], 1))
    assert_close(dx, r, rounded(r, e), "dx", 2)
    xt = x.double().T
    for got, d, ed, what in ((dwg, dg, edg, "dw_gate"), (dwu, du, edu, "dw_up")):
        r, e = product(d.T, xt, ed.T)
        assert_close(got, r, rounded(r, e), what, 2)
    r, e = product(dout.double().T, h.T, None, eh.T)
    assert_close(dwd, r, rounded(r, e), "dw_down", 2)


def test_joined_sums_have_the_same_bits_and_one_workspace():
    """Call after call in one workspace, and in a replayed graph."""
    N, H, I = 5000, 1032, 4096
    x, wg, wu, wd, res = inputs(N, H, I, 5)
    dout = normal(gen(6), N, H, std=0.1)
    ws = torch.empty(max(binding.moe_gated_ffn_workspace_bytes(N, H, I),
                         binding.moe_gated_ffn_backward_workspace_bytes(N, H, I)),
                     dtype=torch.uint8, device="cuda")
    bufs = [torch.empty(s, dtype=BF16, device="cuda") for s in ((N, H), (N, I), (N, I), (N, H),
                                                                (I, H), (I, H), (H, I))]
    out, gate, up, dx, dwg, dwu, dwd = bufs

    def step():
        binding.moe_gated_ffn(x, wg, wu, wd, residual=res, gate=gate, up=up, out=out, workspace=ws)
        binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate, up, dx=dx, want_dw=False,
                                       workspace=ws)
        binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate, up, dw_gate=dwg, dw_up=dwu,
                                       dw_down=dwd, want_dx=False, workspace=ws)

    step()
    want = [t.clone() for t in bufs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for run in (step, graph.replay):
        for t in bufs:
            t.zero_()
        run()
        assert all(torch.equal(a, b) for a, b in zip(bufs, want))
