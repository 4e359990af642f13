"""More than 2^31 values in an array: rows and tensors at either side of that border and
at the end come out as they do on their own."""
import math

import pytest
import torch

from sparse_moe_ffn_gb300 import binding
from test_gpu_gated_ffn import act64, assert_close, product, rounded

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
FAR = 1 << 31


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0):
    """In pieces: no fp32 copy of the whole."""
    out = torch.empty(shape, dtype=BF16, device="cuda")
    flat = out.view(-1)
    for piece in flat.split(1 << 27):
        piece.copy_(torch.randn(piece.numel(), generator=g, device="cuda") * std)
    return out


def pieces(N, H):
    """The first rows, those around value 2^31, and the last."""
    at = FAR // H
    assert at + 4 < N
    return [slice(0, 5), slice(at - 3, at + 4), slice(N - 5, N)]


@pytest.mark.parametrize("N,H", [(1048700, 2056), (524400, 4100), (430000, 5000), (32800, 65535)])
def test_layernorm(N, H):
    g = gen(H)
    x, dy = normal(g, N, H), normal(g, N, H)
    w, b = normal(g, H), normal(g, H)
    out, mean, rstd = binding.moe_layernorm(x, w, b)
    dx, dw, db = binding.moe_layernorm_backward(dy, x, w, mean, rstd)
    for s in pieces(N, H):
        part = binding.moe_layernorm(x[s].clone(), w, b)
        assert torch.equal(out[s], part[0])
        assert torch.equal(mean[s], part[1]) and torch.equal(rstd[s], part[2])
        grad = binding.moe_layernorm_backward(dy[s].clone(), x[s].clone(), w, mean[s].clone(),
                                              rstd[s].clone())
        assert torch.equal(dx[s], grad[0])
    # fp32 sums of 128 rows, of those in a part (64 and more), of eight parts
    ref_w, ref_b, mag_w, mag_b = (torch.zeros(H, dtype=torch.float64, device="cuda")
                                  for _ in range(4))
    step = (1 << 27) // H
    for n in range(0, N, step):
        y = dy[n:n + step].double()
        m = (x[n:n + step].double() - mean[n:n + step, None].double()) * rstd[n:n + step, None].double()
        ref_b += y.sum(0)
        mag_b += y.abs().sum(0)
        ref_w += (y * m).sum(0)
        mag_w += (y * m).abs().sum(0)
    runs = 128 + math.ceil(N / 128 / 2) + 20
    assert bool(((dw.double() - ref_w).abs() <= runs * 2.0 ** -24 * mag_w).all())
    assert bool(((db.double() - ref_b).abs() <= runs * 2.0 ** -24 * mag_b).all())


@pytest.mark.parametrize("place", ["in place", "fp32"])
def test_clipping(place):
    g = gen(1)
    n = FAR + 8191 * 3
    grads = [normal(g, n), normal(g, 77).float()]
    out = None if place == "in place" else [torch.empty(n, device="cuda"),
                                            torch.empty(77, device="cuda")]
    total = math.fsum(float(p.double().square().sum())
                      for t in grads for p in t.view(-1).split(1 << 27))
    norm = binding.moe_grad_norm(grads)
    assert abs(float(norm) - math.sqrt(total)) <= (33 / 2 + 2) * 2.0 ** -24 * math.sqrt(total)
    before = [t.clone() for t in grads]
    got = binding.moe_clip_grads(grads, norm, 100.0, out=out)
    factor = 100.0 / float(norm)
    for k, o in zip(before, got):
        half = 2.0 ** -8 if o.dtype is BF16 else 2.0 ** -24
        for a, b in zip(k.split(1 << 27), o.split(1 << 27)):
            v = a.double() * factor
            assert bool(((b.double() - v).abs() <= (half + 3 * 2.0 ** -24) * v.abs() + 1e-40).all())


@pytest.mark.parametrize("N,H,I", [(1048700, 8, 2056), (1048700, 2056, 8)])
def test_gated_ffn(N, H, I):
    g = gen(I)
    x, res, dout = normal(g, N, H), normal(g, N, H), normal(g, N, H, std=0.1)
    wg, wu, wd = (normal(g, I, H, std=H ** -0.5), normal(g, I, H, std=H ** -0.5),
                  normal(g, H, I, std=I ** -0.5))
    out, gate, up = binding.moe_gated_ffn(x, wg, wu, wd, residual=res, keep=True)
    dx, dwg, dwu, dwd = binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate, up)
    for s in pieces(N, max(H, I)):
        xd, yd = x[s].double(), dout[s].double()
        gd, eg = product(xd, wg.double())
        ud, eu = product(xd, wu.double())
        assert_close(gate[s], gd, rounded(gd, eg), "gate", 1)
        assert_close(up[s], ud, rounded(ud, eu), "up", 1)
        a, _ = act64(gd, "silu")
        h = a * ud
        ea = 1.13 * eg + 2.0 ** -20 * (gd.abs() + eg)
        eh = rounded(h, (ud.abs() + eu) * ea + a.abs() * eu + 2.0 ** -24 * h.abs())
        y, ey = product(h, wd.double(), eh)
        y = y + res[s].double()
        assert_close(out[s], y, rounded(y, ey + 2.0 ** -24 * y.abs()), "out", 2)
        # the backward pass starts from the kept gate and up
        gd, ud = gate[s].double(), up[s].double()
        a, slope = act64(gd, "silu")
        ea, es = 2.0 ** -20 * gd.abs(), 2.0 ** -20 * torch.ones_like(gd)
        dh, edh = product(yd, wd.double().T)
        dg = dh * ud * slope
        edg = ud.abs() * (slope.abs() * edh + (dh.abs() + edh) * es) + 3 * 2.0 ** -24 * dg.abs()
        du = dh * a
        edu = (a.abs() + ea) * edh + dh.abs() * ea + 2.0 ** -24 * du.abs()
        r, e = product(torch.cat([dg, du], 1), torch.cat([wg.double().T, wu.double().T], 1),
                       torch.cat([rounded(dg, edg), rounded(du, edu)], 1))
        assert_close(dx[s], r, rounded(r, e), "dx", 2)
    # the weights' gradients are sums over all tokens: each rounding to bf16 on the
    # way (of dgate, dup or h, and of the result) is off by at most 2^-8 of its value
    ref = [torch.zeros(s, dtype=torch.float64, device="cuda") for s in ((I, H), (I, H), (H, I))]
    mag = [torch.zeros_like(t) for t in ref]
    step = (1 << 27) // max(H, I)
    for n in range(0, N, step):
        xd, yd = x[n:n + step].double(), dout[n:n + step].double()
        gd, ud = gate[n:n + step].double(), up[n:n + step].double()
        a, slope = act64(gd, "silu")
        dh = yd @ wd.double()
        mags = yd.abs() @ wd.double().abs()
        terms = ((dh * ud * slope, mags * ud.abs() * (slope.abs() + 2.0 ** -11), xd),
                 (dh * a, mags * (a.abs() + 2.0 ** -11 * gd.abs()), xd), (yd, yd.abs(), a * ud))
        for i, (left, big, right) in enumerate(terms):
            ref[i] += left.T @ right
            mag[i] += big.T @ right.abs()
    # the sum over N values in fp32: 16 at a time, each time a step of the magnitudes
    rel = 1.02 * 2.0 ** -8 + (N / 16 + 88) * 2.0 ** -23
    for got, r, m in zip((dwg, dwu, dwd), ref, mag):
        assert bool(((got.double() - r).abs() <= rel * m + 2.0 ** -8 * r.abs() + 1e-38).all())
