"""The gated feed-forward block and its backward pass on the GPU against the
formulas in 64 bits.

Tolerances count roundings.  A rounding to bf16 is off by at most 2^-8 of the
value, one to fp32 by 2^-24.  Products of two bf16 values are exact in fp32; the
tensor cores add at least 16 of them at a time to the fp32 accumulator, each
time off by at most a whole fp32 step of the sum of the magnitudes, and parts of
a sum are joined by at most 80 additions.  The activations and their slopes are
within 2^-20 of |v| and of 1 by their description, the slopes at most 1.13 and
their own slopes at most 0.8 in magnitude.
"""
import math

import pytest
import torch

from sparse_moe_ffn_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = 2.0 ** -8
GUARD = 512
ACTS = ["silu", "gelu", "gelu_tanh", "relu", "none"]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


class Guarded:
    """A bf16 output between two guard areas that no kernel may touch."""

    def __init__(self, *shape):
        n = math.prod(shape)
        self.flat = torch.empty(n + 2 * GUARD, dtype=BF16, device="cuda")
        self.bits = self.flat.view(torch.int16)
        self.bits.fill_(0x7FC1)  # a NaN: what is left out shows
        self.t = self.flat[GUARD:GUARD + n].view(shape)
        self.n = n

    def check(self):
        assert bool((self.bits[:GUARD] == 0x7FC1).all())
        assert bool((self.bits[GUARD + self.n:] == 0x7FC1).all())


def act64(v, act):
    """(act(v), act'(v)) in 64 bits."""
    if act == "silu":
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.erfc(-v / math.sqrt(2))
        return v * c, c + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(k * (v + 0.044715 * v ** 3))
        return v * s, s + v * s * (1 - s) * k * (1 + 0.134145 * v * v)
    if act == "relu":
        return v.clamp(min=0), (v > 0).double()
    return v, torch.ones_like(v)


def product(a, b, ea=None, eb=None):
    """(a b^T, its error) in 64 bits, for operands off by ea and eb."""
    K = a.shape[1]
    v, mag = a @ b.T, a.abs() @ b.abs().T
    err = (K / 16 + 88) * 2.0 ** -23 * mag
    if ea is not None:
        err = err + ea @ (b.abs() + (0 if eb is None else eb)).T
    if eb is not None:
        err = err + a.abs() @ eb.T
    return v, err


def rounded(v, err):
    return err + HALF * (v.abs() + err) + 1e-38


def assert_close(got, ref, tol, what, roundings):
    """Within the bound of every element; and, as the roundings of independent
    values go either way, within `roundings` times half a step of the whole's
    root mean square (for sums long enough to say so)."""
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst by "
        f"{float((err / tol).nan_to_num(nan=math.inf).max())} of its bound")
    rms = float(ref.square().mean().sqrt())
    if ref.numel() >= 4096:
        got_rms = float(err.square().mean().sqrt())
        assert got_rms <= roundings * HALF * rms + 1e-38, f"{what}: rms {got_rms / rms}"


def inputs(N, H, I, seed):
    g = gen(seed)
    return (normal(g, N, H), normal(g, I, H, std=H ** -0.5), normal(g, I, H, std=H ** -0.5),
            normal(g, H, I, std=I ** -0.5), normal(g, N, H, std=2.0))


def check_forward(N, H, I, act, residual, keep, seed=0):
    x, wg, wu, wd, res = inputs(N, H, I, seed + N * 7 + H * 3 + I)
    res = res if residual else None
    out = Guarded(N, H)
    gate, up = (Guarded(N, I), Guarded(N, I)) if keep else (None, None)
    ws = torch.full((binding.moe_gated_ffn_workspace_bytes(N, H, I),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    got = binding.moe_gated_ffn(x, wg, wu, wd, act, residual=res, gate=gate and gate.t,
                                up=up and up.t, out=out.t, workspace=ws)
    assert binding.moe_read_device_status(ws) == 0
    assert got[0] is out.t and (got[1] is not None) == keep
    out.check()
    xd = x.double()
    g, eg = product(xd, wg.double())
    u, eu = product(xd, wu.double())
    if keep:
        gate.check()
        up.check()
        assert_close(gate.t, g, rounded(g, eg), "gate", 1)
        assert_close(up.t, u, rounded(u, eu), "up", 1)
    a, _ = act64(g, act)
    h = a * u
    ea = 1.13 * eg + 2.0 ** -20 * (g.abs() + eg)
    eh = rounded(h, (u.abs() + eu) * ea + a.abs() * eu + 2.0 ** -24 * h.abs())
    y, ey = product(h, wd.double(), eh)
    if residual:
        y = y + res.double()
        ey = ey + 2.0 ** -24 * y.abs()
    assert_close(out.t, y, rounded(y, ey), "out", 2)


SIZES = [(1, 8, 8), (3, 8, 8), (20, 8, 72), (300, 8, 8), (1, 64, 64), (2, 72, 200), (7, 1000, 136), (16, 512, 1024), (33, 264, 520),
         (64, 2048, 768), (100, 128, 2056), (129, 640, 640), (256, 256, 256), (257, 1000, 1400),
         (500, 64, 4096), (1021, 1000, 1400), (1300, 2056, 72), (4099, 136, 264)]


@pytest.mark.parametrize("N,H,I", SIZES)
@pytest.mark.parametrize("keep", [False, True])
def test_forward(N, H, I, keep):
    check_forward(N, H, I, "silu", residual=not keep, keep=keep)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N", [3, 70, 300])
def test_forward_activations(N, act):
    check_forward(N, 328, 456, act, residual=True, keep=N == 300)


@pytest.mark.parametrize("N,H,I", [(1, 512, 5000), (2, 5000, 512), (1, 20000, 64), (2, 264, 16384),
                                   (1, 40000, 72), (3, 72, 40000), (128, 1000, 5000)])
def test_forward_rows_shared_by_warps_or_clusters(N, H, I):
    """Few long rows: steps of K that do not divide evenly among warps or CTAs."""
    check_forward(N, H, I, "gelu", residual=True, keep=N != 2)


@pytest.mark.parametrize("N,H,I", [(1, 2048, 8192), (300, 256, 8192), (2048, 512, 4096)])
def test_forward_long_sums(N, H, I):
    """Long K: the slices of the last wave are shared."""
    check_forward(N, H, I, "silu", residual=True, keep=False)


def check_backward(N, H, I, act, seed=0):
    g = gen(seed + N * 5 + H + I * 11)
    x, wg, wu, wd, _ = inputs(N, H, I, seed + 1)
    dout = normal(g, N, H, std=0.1)
    gate, up = normal(g, N, I), normal(g, N, I)
    if act == "relu":
        gate[0, 0] = 0.0
    dx, dwg, dwu, dwd = (Guarded(N, H), Guarded(I, H), Guarded(I, H), Guarded(H, I))
    ws = torch.full((binding.moe_gated_ffn_backward_workspace_bytes(N, H, I),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate, up, act, dx=dx.t, dw_gate=dwg.t,
                                   dw_up=dwu.t, dw_down=dwd.t, workspace=ws)
    assert binding.moe_read_device_status(ws) == 0
    for o in (dx, dwg, dwu, dwd):
        o.check()
    gd, ud = gate.double(), up.double()
    a, slope = act64(gd, act)
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
    assert_close(dx.t, r, rounded(r, e), "dx", 2)
    xt = x.double().T
    for got, d, ed, what in ((dwg, dg, edg, "dw_gate"), (dwu, du, edu, "dw_up")):
        r, e = product(d.T, xt, ed.T)
        assert_close(got.t, r, rounded(r, e), what, 2)
    r, e = product(dout.double().T, h.T, None, eh.T)
    assert_close(dwd.t, r, rounded(r, e), "dw_down", 2)


@pytest.mark.parametrize("N,H,I", SIZES)
def test_backward(N, H, I):
    check_backward(N, H, I, "silu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("N", [5, 300])
def test_backward_activations(N, act):
    check_backward(N, 328, 456, act)


BETWEEN = [(130, 768, 2048), (160, 2048, 768), (200, 264, 2056), (256, 512, 4096), (257, 520, 2816),
           (400, 1024, 2816), (512, 72, 2056), (513, 256, 2048)]


@pytest.mark.parametrize("N,H,I", BETWEEN)
def test_sizes_between_the_kernels_both_ways(N, H, I):
    """Batches that take one kernel for some products and another for the rest."""
    check_forward(N, H, I, "silu", residual=True, keep=True)
    check_backward(N, H, I, "silu")


@pytest.mark.parametrize("N,H,I", [(600, 1024, 1400), (1500, 2048, 768), (2500, 520, 264), (3000, 72, 72),
                                   (1030, 776, 3000)])
def test_gradients_in_one_launch(N, H, I):
    """Batches whose dx and weights' gradients share a launch."""
    check_backward(N, H, I, "gelu")


@pytest.mark.parametrize("N,H,I", [(5000, 256, 256), (300, 256, 8192), (9001, 72, 520)])
def test_backward_long_sums(N, H, I):
    """Long K: the slices of the last wave are shared."""
    check_backward(N, H, I, "gelu_tanh")
