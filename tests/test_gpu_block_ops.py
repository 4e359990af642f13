"""The e4m3, linear and balance operators on the GPU against plain forms in 64
bits.

Tolerances count roundings.  A rounding to a type is off by at most half a
step: 2^-8 of the value for bf16, 2^-24 for fp32, 2^-4 for e4m3 (2^-10 below
its smallest normal value).
"""
import math

import pytest
import torch

from sparse_moe_ffn_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
GUARD = 512


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


class Guarded:
    """An output between two guard areas that no kernel may touch."""

    def __init__(self, shape, dtype, offset=0):
        n = math.prod(shape)
        self.lo = GUARD + offset
        self.flat = torch.empty(n + self.lo + GUARD, dtype=F32 if dtype == F32 else dtype,
                                device="cuda")
        self.bytes = self.flat.view(torch.uint8)
        self.bytes.fill_(0x5A)
        self.size = self.flat.element_size()
        self.t = self.flat[self.lo:self.lo + n].view(shape)
        self.n = n

    def check(self):
        b = self.bytes
        assert bool((b[:self.lo * self.size] == 0x5A).all())
        assert bool((b[(self.lo + self.n) * self.size:] == 0x5A).all())


def assert_within(got, ref, tol, what=""):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        i = int(torch.argmax(torch.where(bad, err / tol, torch.zeros_like(err))))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: got "
                             f"{float(got.double().reshape(-1)[i])}, want "
                             f"{float(ref.reshape(-1)[i])}, off {float(err.reshape(-1)[i])} > "
                             f"{float(tol.reshape(-1)[i])}")


# ----------------------------------------------------------- rows to e4m3

# a thread sums at most 64 squares, then a tree over at most 1024 threads: 80
# roundings, halved by the root; division, root, products: 8 more
ROW_REL = (80 / 2 + 8) * 2.0 ** -24


def check_e4m3(q, scale, y, scale_ref):
    assert_within(scale, scale_ref, scale_ref * ROW_REL, "scale")
    v = y / scale_ref[:, None]
    half = torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10))
    assert_within(q.float(), v, half + 2 * ROW_REL * v.abs() + 1e-30, "q")


def scale_of(y):
    return (y.abs().amax(1) / 448).clamp(min=2.0 ** -100)


@pytest.mark.parametrize("H", [8, 64, 256, 264, 520, 1000, 2048, 2056, 4104, 8192, 8200, 65536])
@pytest.mark.parametrize("N", [1, 3, 129])
@pytest.mark.parametrize("form", ["full", "gemma", "plain", "inplace"])
def test_add_rmsnorm_fp8(N, H, form):
    g = gen(N * 100003 + H)
    x = normal(g, N, H).to(BF16)
    res = None if form == "plain" else normal(g, N, H, std=3.0).to(BF16)
    w = (normal(g, H, std=0.2) + (0 if form == "gemma" else 1)).to(BF16)
    r = x if res is None else (x.float() + res.float()).to(BF16)
    q, s = Guarded((N, H), F8), Guarded((N,), F32)
    nm = Guarded((N, H), BF16) if form != "plain" else None
    ro = Guarded((N, H), BF16) if form in ("full", "gemma") else None
    keep = None if res is None else res.clone()
    out = binding.moe_add_rmsnorm_fp8(x, res, w, eps=1e-5, gemma=form == "gemma", q=q.t,
                                      scale=s.t, normed=nm and nm.t, residual_out=ro and ro.t)
    assert out[0] is q.t and out[1] is s.t
    for t in (q, s, nm, ro):
        if t is not None:
            t.check()
    if ro is not None:
        assert torch.equal(ro.t, r) and torch.equal(res, keep)
    elif res is not None:
        assert torch.equal(res, r)
    rd = r.double()
    y = rd / torch.sqrt((rd * rd).mean(1, keepdim=True) + 1e-5)
    y = y * (w.double() + (1 if form == "gemma" else 0))
    check_e4m3(q.t, s.t, y, scale_of(y))
    if nm is not None:
        assert_within(nm.t, y, (2.0 ** -8 + 2 * ROW_REL) * y.abs() + 1e-38, "normed")


@pytest.mark.parametrize("N,H", [(7001, 256), (4001, 512), (3001, 1000), (1501, 2040), (33, 16384),
                                 (17, 20000), (9, 40000)])
def test_add_rmsnorm_fp8_larger(N, H):
    """Batches and rows that take the other threads-per-row variants."""
    test_add_rmsnorm_fp8(N, H, "full")


@pytest.mark.parametrize("N,H", [(1, 8), (1, 2048), (5, 72), (1000, 264), (333, 4104),
                                 (2, 65536), (40000, 64), (7001, 512), (2001, 1000),
                                 (1501, 2040), (33, 16384), (17, 20000), (9, 40000)])
def test_quantize_fp8(N, H):
    g = gen(H + N)
    x = (normal(g, N, H) * torch.exp(normal(g, N, 1, std=4.0))).to(BF16)
    q, s = Guarded((N, H), F8), Guarded((N,), F32)
    binding.moe_quantize_fp8(x, q=q.t, scale=s.t)
    q.check()
    s.check()
    check_e4m3(q.t, s.t, x.double(), scale_of(x.double()))


def test_rows_with_zeros_nan_and_infinities():
    x = normal(gen(1), 6, 256).to(BF16)
    x[1] = 0
    x[2, 7] = float("nan")
    x[3, 255] = float("inf")
    x[4] = 1e-38
    q, s = binding.moe_quantize_fp8(x)
    assert float(s[1]) == 2.0 ** -100 and bool((q[1].float() == 0).all())
    assert math.isnan(float(s[2])) and bool(q[2].float().isnan().all())
    assert math.isinf(float(s[3])) and bool(q[3, 255].float().isnan())
    assert bool((q[3, :255].float() == 0).all())
    check_e4m3(q[[0, 5]], s[[0, 5]], x[[0, 5]].double(), scale_of(x[[0, 5]].double()))
    # 1e-38 / 448 is below the smallest scale: 1e-38 / 2^-100 rounds to 0
    assert float(s[4]) == 2.0 ** -100 and bool((q[4].float() == 0).all())
    w = torch.ones(256, dtype=BF16, device="cuda")
    q, s, n = binding.moe_add_rmsnorm_fp8(x, None, w, want_normed=True)
    assert bool((q[1].float() == 0).all()) and bool((n[1] == 0).all())
    for i in (2, 3):
        assert math.isnan(float(s[i])) and bool(q[i].float().isnan().all())
    assert bool(n[[0, 1, 4, 5]].isfinite().all())


def test_empty_rows():
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    q, s = binding.moe_quantize_fp8(x)
    assert q.shape == (0, 64) and s.shape == (0,)
    out = binding.moe_linear(x, torch.zeros(8, 64, dtype=BF16, device="cuda"))
    assert out.shape == (0, 8)


# ------------------------------------------------------------------ linear

def act64(v, act):
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return torch.clamp(v, min=0) if act == "relu" else v


def linear_case(N, K, O, kind, seed):
    g = gen(seed)
    x, w = normal(g, N, K).to(BF16), normal(g, O, K, std=0.05).to(BF16)
    if kind == "e4m3":
        x, sx = binding.moe_quantize_fp8(x)
        w, sw = binding.moe_quantize_fp8(w)
        return x, w, dict(x_scale=sx, w_scale=sw)
    return x, w, {}


def linear_ref(x, w, scales, bias, residual, act, out_dtype):
    """(the value in 64 bits, the tolerance).  The products of two bf16 or two
    e4m3 values are exact in fp32.  The tensor cores add at least 16 of them at
    a time to the fp32 accumulator: K / 16 additions and a handful to join,
    each off by at most a whole fp32 step of the sum of the magnitudes.  An
    activation's slope is at most 1.13; the fast exponential and division, and
    erf, are off by less than 2^-20 |v|."""
    K = x.shape[1]
    xd, wd = x.double(), w.double()
    v, mag = xd @ wd.T, xd.abs() @ wd.abs().T
    if scales:
        f = scales["x_scale"].double()[:, None] * scales["w_scale"].double()[None, :]
        v, mag = v * f, mag * f
    err = (K / 16 + 8) * 2.0 ** -23 * mag + 2 * 2.0 ** -24 * v.abs()
    if bias is not None:
        v = v + bias.double()
        err = err + 2.0 ** -24 * v.abs()
    out = act64(v, act)
    err = 1.13 * err + (2.0 ** -20 * v.abs() if act != "none" else 0)
    if residual is not None:
        out = out + residual.double()
        err = err + 2.0 ** -24 * out.abs()
    return out, err + HALF[out_dtype] * (out.abs() + err) + 1e-37


def run_linear(N, K, O, kind, act="none", bias=False, residual=False, out=BF16, seed=None,
               offset=0):
    seed = seed if seed is not None else N * 7919 + K * 31 + O
    x, w, scales = linear_case(N, K, O, kind, seed)
    g = gen(seed + 1)
    b = normal(g, O, std=0.3).to(BF16) if bias else None
    r = normal(g, N, O).to(BF16) if residual else None
    o = Guarded((N, O), out, offset)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    binding.moe_linear(x, w, bias=b, residual=r, activation=act, out=o.t, workspace=ws, **scales)
    ref, tol = linear_ref(x, w, scales, b, r, act, out)
    assert binding.moe_read_device_status(ws) == 0
    o.check()
    assert_within(o.t, ref, tol, f"linear {kind} N={N} K={K} O={O}")


KINDS = ["bf16", "e4m3"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 33, 64, 65, 127, 128, 129, 200, 256, 257, 511])
@pytest.mark.parametrize("K,O", [(16, 8), (64, 128), (144, 1), (528, 130), (2048, 128),
                                 (2064, 264)])
def test_linear_sizes(N, K, O, kind):
    run_linear(N, K, O, kind, bias=True, act="silu")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N,K,O", [(1, 8192, 2048), (3, 2048, 8192), (96, 4096, 4096),
                                   (700, 2048, 2048), (1500, 1040, 1000), (2500, 512, 777),
                                   (4096, 256, 1024), (1030, 4096, 4104), (20000, 64, 72),
                                   (5, 64, 40000), (300, 16, 6), (5000, 2048, 16)])
def test_linear_larger(N, K, O, kind):
    run_linear(N, K, O, kind, residual=True)


def test_linear_bf16_smallest_k():
    run_linear(40, 8, 24, "bf16", bias=True)
    run_linear(700, 8, 300, "bf16", bias=True)
    run_linear(300, 1000, 1111, "bf16", act="gelu", bias=True, residual=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("act", sorted(binding.ACTIVATIONS))
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("N,O", [(7, 96), (150, 200), (1100, 520)])
def test_linear_epilogues(N, O, kind, act, out):
    for bias in (False, True):
        for residual in (False, True):
            run_linear(N, 320, O, kind, act, bias, residual, out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N", [3, 150, 1100])
@pytest.mark.parametrize("out,offset", [(BF16, 1), (BF16, 4), (F32, 1)])
def test_linear_output_at_any_element(N, kind, out, offset):
    """An output that starts on no 16-byte boundary (a slice of a larger one)."""
    run_linear(N, 128, 264, kind, "relu", True, False, out, offset=offset)


@pytest.mark.parametrize("N", [5, 140, 1300])
def test_linear_residual_at_any_element_and_in_place(N):
    x, w, _ = linear_case(N, 256, 200, "bf16", 5)
    r = Guarded((N, 200), BF16, 1)
    r.t.copy_(normal(gen(6), N, 200).to(BF16))
    ref, tol = linear_ref(x, w, {}, None, r.t.clone(), "none", BF16)
    binding.moe_linear(x, w, residual=r.t, out=r.t)
    r.check()
    assert_within(r.t, ref, tol, "in place")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N", [4, 130, 1200])
def test_linear_nonfinite_rows_stay_in_their_rows(N, kind):
    x, w, scales = linear_case(N, 272, 136, kind, 9)
    clean = binding.moe_linear(x, w, **scales)
    bad = x.clone()
    bad[1, 3] = float("nan")
    w2 = w.clone()
    w2[7, 5] = float("nan")
    got = binding.moe_linear(bad, w2, **scales)
    assert bool(got[1].isnan().all()) and bool(got[:, 7].isnan().all())
    rows = [n for n in range(N) if n != 1]
    cols = [o for o in range(136) if o != 7]
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])


@pytest.mark.parametrize("N", [2, 300, 1500])
def test_linear_same_bits_every_time_and_in_a_graph(N):
    x, w, _ = linear_case(N, 2048, 520, "bf16", 3)
    first = binding.moe_linear(x, w)
    out = torch.empty_like(first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # another stream than the tensors' own
        other = binding.moe_linear(x, w)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.moe_linear(x, w, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(first, out)


# ----------------------------------------------------------------- balance

def balance64(logits, ids, mask, k):
    """(p, lse, f, T, counts) in 64 bits, loops over nothing but tokens kept."""
    N, E = logits.shape
    keep = torch.ones(N, dtype=torch.bool, device="cuda") if mask is None else mask
    lg = logits.double()
    lse = torch.logsumexp(lg, 1)
    empty = torch.isneginf(lg).all(1)
    lse = torch.where(empty, torch.zeros_like(lse), lse)
    p = torch.where(empty[:, None], torch.zeros_like(lg), torch.exp(lg - lse[:, None]))
    p, lse = p * keep[:, None], lse * keep
    T = int(keep.sum())
    kept = ids[keep].reshape(-1).long()
    counts = torch.bincount(kept[(kept >= 0) & (kept < E)], minlength=E)
    f = counts.double() / max(k * T, 1)
    return p, lse, f, T, counts


def losses64(p, lse, f, T):
    E = p.shape[1]
    return torch.stack([E * (f * p.sum(0)).sum(), (lse * lse).sum()]) / max(T, 1)


# e^(x - top): the fast exponential is off by (2 + 1.16 |x - top|) steps, and
# what is further down than e^-20 adds nothing; the sum, the quotient and the
# division: 14 more half steps
P_REL = (2 * 26 + 14) * 2.0 ** -24


def grad64(p, lse, f, T, grad):
    """(dlogits, their tolerance before the rounding to the output's type)."""
    E = p.shape[1]
    d = f - 1.0 / E
    g0, g1 = float(grad[0]) * E / max(T, 1), 2 * float(grad[1]) / max(T, 1)
    u = d - (p * d).sum(1, keepdim=True)
    got = p * (g0 * u + g1 * lse[:, None])
    around = (p * d.abs()).sum(1, keepdim=True)
    du = (P_REL + 16 * 2.0 ** -24) * around + 4 * 2.0 ** -24 * (d.abs() + around)
    dl = P_REL + 2.0 ** -22 * lse.abs()[:, None]
    tol = (P_REL + 8 * 2.0 ** -24) * got.abs() + p * (abs(g0) * du + abs(g1) * dl)
    tol = tol + 4 * 2.0 ** -24 * p * (abs(g0) * u.abs() + abs(g1) * lse.abs()[:, None])
    return got, tol + 1e-9 * 2.0 ** -10 * (abs(g0) + abs(g1)) / 1.0


def balance_case(N, E, k, dtype, seed, masked):
    g = gen(seed)
    logits = normal(g, N, E, std=1.5) + normal(g, E, std=0.5)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    mask = None
    if masked:
        mask = torch.rand(N, generator=g, device="cuda") > 0.25
        ids = ids.masked_fill(torch.rand(N, k, generator=g, device="cuda") < 0.1, -1)
        if E > 2:
            logits[:, 1] = float("-inf")
        logits[torch.rand(N, generator=g, device="cuda") < 0.05] = float("-inf")
        logits[~mask] = float("nan")  # a masked token is not read
        ids[~mask] = 1 << 30
    return logits.to(dtype), ids.contiguous(), mask


def check_balance(logits, ids, mask, k):
    N, E = logits.shape
    ws = torch.full((binding.lib().moe_balance_loss_workspace_bytes(N, E),), 0xA5,
                    dtype=torch.uint8, device="cuda")  # no state from earlier calls is needed
    c = Guarded((E,), torch.int32)
    losses, counts, tokens = binding.moe_balance_loss(logits, ids, mask, counts=c.t, workspace=ws)
    assert binding.moe_read_device_status(ws) == 0
    c.check()
    clean = logits if mask is None else torch.where(mask[:, None], logits,
                                                    torch.zeros_like(logits))
    p, lse, f, T, want = balance64(clean, ids, mask, k)
    assert int(tokens) == T
    assert torch.equal(counts.long(), want)
    ref = losses64(p, lse, f, T)
    # a thread adds the rows of one block of 304 one after the other
    rows = N / 304 + 32
    tol = torch.stack([ref[0] * (P_REL + rows * 2.0 ** -24),
                       (2 * lse.abs() * (P_REL + 2.0 ** -22 * lse.abs())).sum() / max(T, 1)
                       + ref[1] * rows * 2.0 ** -24]) + 1e-30
    assert_within(losses, ref, tol, "losses")
    grad = torch.tensor([0.3, -0.02], dtype=F32, device="cuda")
    d = Guarded((N, E), logits.dtype)
    binding.moe_balance_loss_backward(logits, counts, tokens, k, grad, mask, dlogits=d.t)
    d.check()
    ref, tol = grad64(p, lse, f, T, grad)
    assert_within(d.t, ref, tol + HALF[logits.dtype] * (ref.abs() + tol) + 1e-38, "dlogits")
    if mask is not None:
        assert bool((d.t[~mask] == 0).all())
    return losses, counts, tokens


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (6, 2), (7, 3), (8, 8), (31, 4), (60, 4),
                                 (64, 6), (127, 8), (128, 8), (129, 10), (200, 5), (255, 1),
                                 (256, 8)])
@pytest.mark.parametrize("N", [1, 2, 37, 1000])
def test_balance_sizes(N, E, k, masked, dtype):
    check_balance(*balance_case(N, E, k, dtype, N * 1000 + E, masked), k)


# one cluster of 16 blocks (up to three passes), then several of 8
@pytest.mark.parametrize("N,E,k", [(2500, 256, 8), (5000, 128, 8), (12000, 60, 4), (3075, 255, 3),
                                   (6200, 128, 8), (40000, 128, 8), (100003, 60, 4),
                                   (300000, 6, 2)])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_many_tokens(N, E, k, masked):
    check_balance(*balance_case(N, E, k, F32, N, masked), k)


def test_balance_no_tokens():
    for N, mask in ((0, None), (5, torch.zeros(5, dtype=torch.bool, device="cuda"))):
        logits = torch.full((N, 12), float("nan"), device="cuda")
        ids = torch.zeros((N, 2), dtype=torch.int32, device="cuda")
        losses, counts, tokens = binding.moe_balance_loss(logits, ids, mask)
        assert losses.tolist() == [0.0, 0.0] and int(tokens) == 0
        assert counts.tolist() == [0] * 12
        d = binding.moe_balance_loss_backward(logits, counts, tokens, 2,
                                              torch.ones(2, device="cuda"), mask)
        assert d.shape == (N, 12) and bool((d == 0).all())


def test_balance_reports_ids_out_of_range():
    logits, ids, _ = balance_case(50, 16, 2, F32, 4, False)
    ids[7, 1] = 16
    ids[9, 0] = -5
    ws = torch.zeros(binding.lib().moe_balance_loss_workspace_bytes(50, 16), dtype=torch.uint8,
                     device="cuda")
    _, counts, _ = binding.moe_balance_loss(logits, ids, workspace=ws)
    assert binding.moe_read_device_status(ws) == 5
    assert int(counts.sum()) == 98
    ids[7, 1] = 15
    binding.moe_balance_loss(logits, ids, workspace=ws)
    assert binding.moe_read_device_status(ws) == 0


def test_balance_logits_at_any_element():
    """Rows that start on no 16-byte boundary (a slice of a larger tensor)."""
    for dtype in (F32, BF16):
        src, ids, _ = balance_case(77, 64, 4, dtype, 8, False)
        at = Guarded((77, 64), dtype, 1)
        at.t.copy_(src)
        check_balance(at.t, ids, None, 4)


def test_balance_gradient_against_differences():
    """Central differences of the losses in 64 bits, the load held fixed."""
    logits, ids, mask = balance_case(9, 10, 3, F32, 12, False)
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 1, 0, 1], dtype=torch.bool, device="cuda")
    _, counts, tokens = binding.moe_balance_loss(logits, ids, mask)
    grad = torch.tensor([0.7, 0.05], dtype=F32, device="cuda")
    got = binding.moe_balance_loss_backward(logits, counts, tokens, 3, grad, mask)
    _, _, f, T, _ = balance64(logits, ids, mask, 3)
    g64 = grad.double()

    def total(lg):
        p, lse, _, _, _ = balance64(lg, ids, mask, 3)
        return (g64 * losses64(p, lse, f, T)).sum()

    h = 2.0 ** -13
    for n in range(9):
        for e in range(10):
            up, down = logits.double().clone(), logits.double().clone()
            up[n, e] += h
            down[n, e] -= h
            diff = float((total(up) - total(down)) / (2 * h))
            # the difference's own error: h^2 / 6 times a third derivative
            # (below 10), and 2^-52 of the total's size over h
            tol = h * h / 6 * 10 + 2.0 ** -52 * 20 / h + 1e-5 * abs(diff) + 1e-7
            assert abs(float(got[n, e]) - diff) <= tol, (n, e)


def test_balance_same_bits_in_place_and_in_a_graph():
    logits, ids, mask = balance_case(5000, 128, 8, F32, 21, True)
    grad = torch.tensor([0.01, 0.001], dtype=F32, device="cuda")

    def both():
        a = binding.moe_balance_loss(logits, ids, mask)
        return (*a, binding.moe_balance_loss_backward(logits, a[1], a[2], 8, grad, mask))

    first = both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    graph.replay()
    again = logits.clone()
    binding.moe_balance_loss_backward(again, first[1], first[2], 8, grad, mask, dlogits=again)
    for a, b in zip(first, held):
        assert torch.equal(a, b)
    assert torch.equal(first[3], again)


# ------------------------------------------- other streams, far offsets


def test_norm_and_balance_on_another_stream_and_in_a_graph():
    g = gen(31)
    x, res = normal(g, 300, 2048).to(BF16), normal(g, 300, 2048).to(BF16)
    w = torch.ones(2048, dtype=BF16, device="cuda")
    out = torch.empty_like(res)
    logits, ids, mask = balance_case(3000, 64, 6, BF16, 2, True)
    grad = torch.tensor([0.5, 0.1], dtype=F32, device="cuda")

    def all_of_them():
        a = binding.moe_add_rmsnorm_fp8(x, res, w, want_normed=True, residual_out=out)
        b = binding.moe_quantize_fp8(x)
        c = binding.moe_balance_loss(logits, ids, mask)
        d = binding.moe_balance_loss_backward(logits, c[1], c[2], 6, grad, mask)
        return [t.float() for t in (*a, *b, *c, d)]

    first = all_of_them()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = all_of_them()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of_them()
    graph.replay()
    for a, b, c in zip(first, other, held):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("kind,O,residual", [("bf16", 8200, True), ("e4m3", 8001, False)])
def test_linear_past_2_31_outputs(kind, O, residual):
    """Outputs whose element offsets pass 32 bits, in tensor-map stores and in
    single values; sampled rows, the last ones among them."""
    N, K = 270000, 64
    x, w, scales = linear_case(N, K, O, kind, 77)
    r = normal(gen(78), N, O).to(BF16) if residual else None
    out = binding.moe_linear(x, w, residual=r, **scales)
    rows = torch.cat([torch.arange(0, N, 9973, device="cuda"),
                      torch.arange(N - 70, N, device="cuda")])
    part = {n: (t[rows] if n == "x_scale" else t) for n, t in scales.items()}
    ref, tol = linear_ref(x[rows], w, part, None, None if r is None else r[rows], "none", BF16)
    assert_within(out[rows], ref, tol, "far rows")


def test_rows_past_2_31_elements():
    N, H = 270000, 8200
    g = gen(5)
    x = torch.empty((N, H), dtype=BF16, device="cuda")
    for i in range(0, N, 30000):
        x[i:i + 30000] = normal(g, min(30000, N - i), H).to(BF16)
    q, s = binding.moe_quantize_fp8(x)
    rows = torch.cat([torch.arange(0, N, 9973, device="cuda"),
                      torch.arange(N - 70, N, device="cuda")])
    y = x[rows].double()
    check_e4m3(q[rows], s[rows], y, scale_of(y))


def test_balance_past_2_31_logits():
    N, E = (1 << 23) + 1001, 256
    logits = torch.empty((N, E), dtype=BF16, device="cuda")
    g = gen(6)
    for i in range(0, N, 1 << 20):
        logits[i:i + (1 << 20)] = normal(g, min(1 << 20, N - i), E).to(BF16)
    ids = torch.randint(0, E, (N, 1), generator=g, device="cuda", dtype=torch.int32)
    losses, counts, tokens = binding.moe_balance_loss(logits, ids)
    assert int(tokens) == N
    assert torch.equal(counts.long(), torch.bincount(ids[:, 0].long(), minlength=E))
    grad = torch.tensor([0.3, -0.02], dtype=F32, device="cuda")
    d = binding.moe_balance_loss_backward(logits, counts, tokens, 1, grad)
    rows = torch.cat([torch.arange(0, N, 99991, device="cuda"),
                      torch.arange(N - 70, N, device="cuda")])
    p, lse, _, _, _ = balance64(logits[rows], ids[rows], None, 1)
    ref, tol = grad64(p, lse, counts.double() / N, N, grad)
    assert_within(d[rows], ref, tol + HALF[BF16] * (ref.abs() + tol) + 1e-38, "far rows")
