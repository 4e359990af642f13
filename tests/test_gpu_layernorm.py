"""Layer norm and its backward pass on the GPU against the formulas in 64 bits.

Tolerances count roundings: 2^-8 of a value for bf16, 2^-24 for fp32.  A thread
adds at most 64 values, a tree over at most 1024 threads 32 more (ten levels
within and across warps, or 32 warps one by one): 128 roundings of the sum of the
magnitudes bound a row's sums.
"""
import math

import pytest
import torch

from sparse_moe_ffn_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
ROW = 128 * 2.0 ** -24
GUARD = 256
EPS = 1e-5


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


class Guarded:
    def __init__(self, shape, dtype, offset=0):
        n = math.prod(shape)
        self.flat = torch.full((n + 2 * GUARD + offset,), float("nan"), dtype=dtype, device="cuda")
        self.lo, self.n = GUARD + offset, n
        self.t = self.flat[self.lo:self.lo + n].view(shape)

    def check(self):
        assert bool(self.flat[:self.lo].isnan().all())
        assert bool(self.flat[self.lo + self.n:].isnan().all())
        assert not bool(self.t.isnan().any())


def assert_within(got, ref, tol, what):
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off"


def offset_by(t, k):
    """The same values in storage that starts k values later."""
    flat = torch.empty(t.numel() + k, dtype=t.dtype, device="cuda")
    flat[k:].copy_(t.reshape(-1))
    return flat[k:].view(t.shape)


def forward64(r, w, b):
    """(out, its error; mean, its error; rstd, its error) of the rows r."""
    H = r.shape[1]
    mean = r.mean(1)
    emean = ROW * r.abs().mean(1)
    d = r - mean[:, None]
    ed = emean[:, None] + 2.0 ** -24 * (d.abs() + emean[:, None])
    var = (d * d).mean(1)
    # the deviations are taken from a mean that is off by emean: second order
    # in the sum, plus the roundings
    evar = emean ** 2 + (2 * 2.0 ** -24 + ROW) * var + 2 * (d.abs() * 2.0 ** -24 * d.abs()).mean(1)
    rstd = 1 / torch.sqrt(var + EPS)
    erstd = rstd * (0.5 * evar / (var + EPS) * 1.01 + 8 * 2.0 ** -24)
    n = d * rstd[:, None]
    en = ed * rstd[:, None] + d.abs() * erstd[:, None] + 2.0 ** -24 * n.abs()
    y = n * w
    ey = en * w.abs() + 2.0 ** -24 * y.abs()
    if b is not None:
        y = y + b
        ey = ey + 2.0 ** -24 * y.abs()
    return y, ey, mean, emean, rstd, erstd, n, en


def check(N, H, dtype, residual=True, bias=True, offset=0, seed=0, mean=0.5):
    g = gen(seed + N * 31 + H)
    x = offset_by(normal(g, N, H, dtype=dtype) + torch.tensor(mean, dtype=dtype), offset)
    res = offset_by(normal(g, N, H, std=3.0, dtype=dtype), offset) if residual else None
    w = normal(g, H, std=0.2, dtype=dtype) + 1
    b = normal(g, H, dtype=dtype) if bias else None
    r = x if res is None else (x.float() + res.float()).to(dtype)
    out, mu, rs = Guarded((N, H), dtype, offset), Guarded((N,), F32), Guarded((N,), F32)
    ro = Guarded((N, H), dtype, offset) if residual else None
    got = binding.moe_layernorm(x, w, b, res, EPS, out=out.t, residual_out=ro and ro.t, mean=mu.t,
                                rstd=rs.t)
    assert got[0] is out.t and got[1] is mu.t and got[2] is rs.t
    for t in (out, mu, rs):
        t.check()
    if residual:
        ro.check()
        assert torch.equal(ro.t, r)
    y, ey, mean64, emean, rstd, erstd, n, en = forward64(
        r.double(), w.double(), None if b is None else b.double())
    assert_within(mu.t, mean64, emean + 1e-38, "mean")
    assert_within(rs.t, rstd, erstd, "rstd")
    assert_within(out.t, y, ey + HALF[dtype] * (y.abs() + ey) + 1e-38, "out")

    # backward, from the statistics that the forward call gave
    dy = offset_by(normal(g, N, H, std=0.1, dtype=dtype), offset)
    dr = offset_by(normal(g, N, H, std=0.1, dtype=dtype), offset) if residual else None
    dx, dw = Guarded((N, H), dtype, offset), Guarded((H,), F32)
    db = Guarded((H,), F32) if bias else None
    ws = torch.full((binding.moe_layernorm_backward_workspace_bytes(N, H),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    binding.moe_layernorm_backward(dy, r, w, mu.t, rs.t, dr, dx=dx.t, dweight=dw.t,
                                   dbias=db and db.t, want_dbias=bias, workspace=ws)
    dx.check()
    dw.check()
    yd = dy.double()
    t = yd * w.double()
    et = 2.0 ** -24 * t.abs()
    m1, m2 = t.mean(1, keepdim=True), (t * n).mean(1, keepdim=True)
    e1 = ROW * t.abs().mean(1, keepdim=True)
    e2 = ((ROW + 2.0 ** -23) * (t * n).abs() + t.abs() * en).mean(1, keepdim=True)
    v = t - m1 - n * m2
    ev = et + e1 + en * m2.abs() + (n.abs() + en) * e2 + 3 * 2.0 ** -24 * (
        t.abs() + m1.abs() + (n * m2).abs())
    d = v * rstd[:, None]
    ed = ev * rstd[:, None] + v.abs() * erstd[:, None] + 2.0 ** -24 * d.abs()
    if residual:
        d = d + dr.double()
        ed = ed + 2.0 ** -24 * d.abs()
    assert_within(dx.t, d, ed + HALF[dtype] * (d.abs() + ed) + 1e-38, "dx")
    # sums over rows: at most N roundings in fp32 (fewer: a block's rows), one at
    # the end
    rows = min(N, 512)
    mag = (yd * n).abs().sum(0)
    ref = (yd * n).sum(0)
    assert_within(dw.t, ref, (yd.abs() * en).sum(0) + (rows + 4) * 2.0 ** -24 * mag, "dweight")
    if bias:
        db.check()
        assert_within(db.t, yd.sum(0), (rows + 4) * 2.0 ** -24 * yd.abs().sum(0), "dbias")


HS = [1, 2, 7, 8, 31, 64, 100, 256, 264, 511, 512, 520, 1000, 1024, 1111, 2048, 2056, 4096, 4100,
      8192, 8200, 10001, 16384, 16400, 20000, 40000, 65535, 65536]


@pytest.mark.parametrize("H", HS)
@pytest.mark.parametrize("N", [1, 5, 77])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_rows(N, H, dtype):
    check(N, H, dtype)


@pytest.mark.parametrize("N,H", [(4001, 64), (3000, 256), (2501, 512), (1301, 1000), (999, 2048),
                                 (701, 4096), (401, 8192), (333, 1111), (257, 16384)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_batches(N, H, dtype):
    check(N, H, dtype, residual=N % 2 == 0, bias=N % 3 != 0)


@pytest.mark.parametrize("offset", [1, 3, 8])
@pytest.mark.parametrize("H", [256, 2048, 10000])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_arrays_that_start_anywhere(H, offset, dtype):
    check(19, H, dtype, offset=offset)


def test_large_mean():
    """The variance is that of the deviations, not a difference of large sums."""
    check(9, 2048, F32, residual=False, mean=4096.0)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_constant_rows_nan_and_infinities(dtype):
    x = normal(gen(0), 5, 256, dtype=dtype)
    x[1] = 3.0
    x[2, 7] = float("nan")
    x[3, 255] = float("inf")
    w = torch.full((256,), 2.0, dtype=dtype, device="cuda")
    b = torch.full((256,), 0.5, dtype=dtype, device="cuda")
    out, mean, rstd = binding.moe_layernorm(x, w, b)
    assert bool((out[1] == 0.5).all()) and float(mean[1]) == 3.0
    assert abs(float(rstd[1]) - EPS ** -0.5) <= 2.0 ** -21 * EPS ** -0.5
    assert bool(out[2].isnan().all()) and bool(out[3].isnan().all())
    assert bool(out[[0, 1, 4]].isfinite().all())


@pytest.mark.parametrize("H", [48, 2048, 9000])
def test_outputs_in_place_of_inputs(H):
    g = gen(H)
    N = 37
    x, res = normal(g, N, H), normal(g, N, H)
    w, b = normal(g, H), normal(g, H)
    ro = torch.empty_like(x)
    out, mean, rstd = binding.moe_layernorm(x, w, b, res, residual_out=ro)
    x2, res2 = x.clone(), res.clone()
    out2, _, _ = binding.moe_layernorm(x2, w, b, res2, out=x2)  # the sum goes to res2
    assert out2 is x2 and torch.equal(x2, out) and torch.equal(res2, ro)
    dy, dr = normal(g, N, H), normal(g, N, H)
    dx, dw, db = binding.moe_layernorm_backward(dy, ro, w, mean, rstd, dr)
    for which in range(3):
        ins = [dy.clone(), ro.clone(), dr.clone()]
        got = binding.moe_layernorm_backward(ins[0], ins[1], w, mean, rstd, ins[2], dx=ins[which])
        assert torch.equal(ins[which], dx) and torch.equal(got[1], dw) and torch.equal(got[2], db)


@pytest.mark.parametrize("H", [10001, 20000, 40001, 65536])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_long_rows(H, dtype):
    """More rows than blocks, and the outputs in place of the inputs: rows that
    are read again find what they had."""
    N = 701
    check(N, H, dtype, residual=H % 2 == 0)
    g = gen(H)
    x, res, w, b = (normal(g, *s, dtype=dtype) for s in ((N, H), (N, H), (H,), (H,)))
    ro = torch.empty_like(x)
    out, mean, rstd = binding.moe_layernorm(x, w, b, res, residual_out=ro)
    for sum_in in (0, 1):  # r over x, out over the residual, and the other way round
        ins = [x.clone(), res.clone()]
        got = binding.moe_layernorm(ins[0], w, b, ins[1], out=ins[1 - sum_in],
                                    residual_out=ins[sum_in])
        assert torch.equal(ins[sum_in], ro) and torch.equal(ins[1 - sum_in], out)
        assert torch.equal(got[1], mean) and torch.equal(got[2], rstd)
    dy, dr = normal(g, N, H, dtype=dtype), normal(g, N, H, dtype=dtype)
    want = binding.moe_layernorm_backward(dy, ro, w, mean, rstd, dr)
    for which in range(3):
        ins = [dy.clone(), ro.clone(), dr.clone()]
        got = binding.moe_layernorm_backward(ins[0], ins[1], w, mean, rstd, ins[2], dx=ins[which])
        for a, e in zip(got, want):
            assert torch.equal(a, e)


@pytest.mark.parametrize("H", [64, 100])
def test_sum_stored_without_a_residual(H):
    x, w = normal(gen(H), 7, H), normal(gen(1), H)
    copy = torch.empty_like(x)
    out, _, _ = binding.moe_layernorm(x, w, residual_out=copy)
    assert torch.equal(copy, x) and torch.equal(out, binding.moe_layernorm(x, w)[0])


def test_no_rows():
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    out, mean, rstd = binding.moe_layernorm(x, w)
    assert out.shape == (0, 64) and mean.shape == (0,)
    dw = torch.full((64,), 7.0, device="cuda")
    dx, dw, db = binding.moe_layernorm_backward(x, x, w, mean, rstd, dweight=dw)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


def test_gradients_against_differences():
    """The directional difference of sum(c * layernorm(r)) in 64 bits against the
    gradients: fp32 sums of 64 rows of 136 values, 2^-14 of the magnitudes; the
    central difference with step 1e-4 is off by its third derivative, about
    1e-8 of them."""
    g = gen(5)
    N, H = 64, 136
    r, w, b, c = (normal(g, *s, dtype=F32) for s in ((N, H), (H,), (H,), (N, H)))
    out, mean, rstd = binding.moe_layernorm(r, w, b)
    dx, dw, db = binding.moe_layernorm_backward(c, r, w, mean, rstd)
    vr, vw, vb = (normal(g, *s, dtype=F32).double() for s in ((N, H), (H,), (H,)))

    def loss(e):
        x = r.double() + e * vr
        d = x - x.mean(1, keepdim=True)
        n = d / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
        return float((c.double() * (n * (w.double() + e * vw) + b.double() + e * vb)).sum())

    slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
    parts = [dx.double() * vr, dw.double() * vw, db.double() * vb]
    mag = sum(float(p.abs().sum()) for p in parts)
    assert abs(slope - sum(float(p.sum()) for p in parts)) <= 2.0 ** -14 * mag


@pytest.mark.parametrize("H", [512, 9000])
def test_same_bits_and_other_streams(H):
    g = gen(2)
    r, dy, w = normal(g, 3001, H), normal(g, 3001, H), normal(g, H)
    out, mean, rstd = binding.moe_layernorm(r, w)
    first = binding.moe_layernorm_backward(dy, r, w, mean, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(3):
            out2, _, _ = binding.moe_layernorm(r, w)
            again = binding.moe_layernorm_backward(dy, r, w, mean, rstd)
    s.synchronize()
    assert torch.equal(out, out2)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
