"""The dense block's operators as they are used: together, captured in graphs, on
several streams, with extreme values, and their gradients against differences."""
import math

import pytest
import torch

from sparse_moe_ffn_gb300 import binding
from sparse_moe_ffn_gb300.block import DenseBlock, clip_step, dense_steps

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = 2.0 ** -8


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def weights(g, H, I):
    return (normal(g, I, H, std=H ** -0.5), normal(g, I, H, std=H ** -0.5),
            normal(g, H, I, std=I ** -0.5))


def make_block(g, H, I, activation="silu", bias=True):
    return DenseBlock(normal(g, H, std=0.1) + 1, normal(g, H, std=0.1) if bias else None,
                      *weights(g, H, I), activation)


def reference(block, x, residual, dout):
    """out and the gradients by autograd in 64 bits."""
    names = ["norm_weight", "norm_bias", "w_gate", "w_up", "w_down"]
    p = {n: getattr(block, n).double().requires_grad_() for n in names
         if getattr(block, n) is not None}
    r = (x.float() + residual.float()).to(BF16).double().requires_grad_()
    n = torch.nn.functional.layer_norm(r, r.shape[1:], p["norm_weight"], p.get("norm_bias"),
                                       block.eps)
    a = n @ p["w_gate"].T
    h = torch.nn.functional.silu(a) if block.activation == "silu" else \
        torch.nn.functional.gelu(a)
    out = (h * (n @ p["w_up"].T)) @ p["w_down"].T + r
    out.backward(dout.double())
    return out.detach(), r.grad, {n: t.grad for n, t in p.items()}


def off(got, ref):
    return float((got.double() - ref).square().mean().sqrt() / ref.square().mean().sqrt())


@pytest.mark.parametrize("N,H,I,act,bias", [(1, 64, 128, "silu", True), (3, 512, 256, "gelu", True),
                                            (70, 136, 520, "silu", False),
                                            (300, 256, 1024, "gelu", True),
                                            (2000, 512, 512, "silu", True)])
def test_block_forward_backward_and_clipping(N, H, I, act, bias):
    g = gen(N)
    block = make_block(g, H, I, act, bias)
    x, residual, dout = normal(g, N, H), normal(g, N, H, std=2.0), normal(g, N, H, std=0.1)
    out, dr, grads = reference(block, x, residual, dout)
    res = residual.clone()
    got, kept = block(x, res, keep=True)
    assert torch.equal(res, (x.float() + residual.float()).to(BF16))
    assert torch.equal(block(x, residual.clone()), got)  # serving gives the same
    got_dr, got_grads = block.backward(dout, kept)
    # roundings to bf16 on the way, each at most half a step of its value and
    # independent of the others: the normed row, h, out; in the backward pass the
    # normed row, gate, up, h or dgate and dup, the gradient
    assert off(got, out) <= 3 * HALF
    assert off(got_dr, dr) <= 6 * HALF
    assert set(got_grads) == set(grads)
    for n, t in got_grads.items():
        assert t.dtype is (F32 if n.startswith("norm") else BF16)
        assert off(t, grads[n]) <= 6 * HALF, n
    total = math.sqrt(sum(float(t.double().square().sum()) for t in got_grads.values()))
    before = {n: t.clone() for n, t in got_grads.items()}
    norm = clip_step(got_grads, 0.5 * total)
    assert abs(float(norm) - total) <= 2.0 ** -20 * total
    for n, t in got_grads.items():
        assert off(t, before[n].double() * 0.5) <= (2.0 ** -20 if t.dtype is F32 else 2 * HALF)


def test_steps_of_a_dense_block_run():
    norms = dense_steps(N=300, H=128, I=256, steps=3)
    assert len(norms) == 3 and all(math.isfinite(n) and n > 0 for n in norms)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_gradients_against_differences(act):
    """The directional difference of sum(dout * ffn(x)) in 64 bits against the
    kernel's gradients: five roundings of independent values, 5 x 2^-8 of the
    root of the sum of squares; the central difference with step 1e-4 is off by
    its third derivative, about 1e-8."""
    g = gen(7)
    N, H, I = 200, 128, 192
    wg, wu, wd = weights(g, H, I)
    x, dout = normal(g, N, H), normal(g, N, H)
    _, gate, up = binding.moe_gated_ffn(x, wg, wu, wd, act, keep=True)
    grads = binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate, up, act)
    vs = [torch.randn(t.shape, generator=g, device="cuda").double() for t in (x, wg, wu, wd)]

    def loss(e):
        x_, g_, u_, d_ = (t.double() + e * v for t, v in zip((x, wg, wu, wd), vs))
        a = x_ @ g_.T
        if act == "silu":
            a = a * torch.sigmoid(a)
        elif act == "gelu":
            a = a * torch.special.ndtr(a)
        else:
            a = a * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))
        return float((dout.double() * ((a * (x_ @ u_.T)) @ d_.T)).sum())

    slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
    parts = torch.cat([(t.double() * v).reshape(-1) for t, v in zip(grads, vs)])
    # a rounding error is random: the whole is off by a few times its root mean square
    assert abs(slope - float(parts.sum())) <= 5 * HALF * 5 * float(parts.square().sum().sqrt())


@pytest.mark.parametrize("N", [1, 2, 3, 40, 128, 129, 600])
def test_a_token_reaches_its_own_row_alone(N):
    g = gen(N)
    H, I = 256, 384
    wg, wu, wd = weights(g, H, I)
    x, res = normal(g, N, H), normal(g, N, H)
    clean, gate, up = binding.moe_gated_ffn(x, wg, wu, wd, residual=res, keep=True)
    bad = N // 2
    y = x.clone()
    y[bad, 3] = float("nan")
    out, gate2, up2 = binding.moe_gated_ffn(y, wg, wu, wd, residual=res, keep=True)
    rest = torch.arange(N, device="cuda") != bad
    assert bool(out[bad].isnan().all())
    for a, b in ((out, clean), (gate2, gate), (up2, up)):
        assert torch.equal(a[rest], b[rest])
    dout = normal(g, N, H)
    dx = binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate, up, want_dw=False)[0]
    dout[bad] = float("inf")
    got = binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate, up, want_dw=False)
    assert torch.equal(got[0][rest], dx[rest]) and got[1:] == (None, None, None)


def test_extreme_gates():
    """Where e^-v, v^2 or v^3 leave the range: the activation and its slope are
    those of the limits (identity matrices bring them out one by one)."""
    N = H = I = 64
    eye = torch.eye(H, dtype=BF16, device="cuda")
    zero = torch.zeros_like(eye)
    vals = torch.tensor([-3e38, -1e30, -1e15, -1e4, -200.0, -100.0, -88.5, -30.0, -10.0, -1e-30, 0.0,
                         1e-30, 10.0, 30.0, 88.5, 100.0, 200.0, 1e4, 1e15, 1e30, 3e38],
                        device="cuda").to(BF16)
    v = vals[torch.arange(N * I, device="cuda") % len(vals)].view(N, I)
    dout = normal(gen(1), N, H)
    up = torch.full_like(v, 0.5)
    for act in ("silu", "gelu", "gelu_tanh", "relu", "none"):
        vd = v.double()
        if act == "silu":
            s = torch.sigmoid(vd)
            a, d = vd * s, s + vd * s * torch.sigmoid(-vd)
        elif act == "gelu":
            c = torch.special.ndtr(vd)
            a, d = vd * c, c + vd * torch.exp(-vd * vd / 2) / math.sqrt(2 * math.pi)
        elif act == "gelu_tanh":
            k = 2 * math.sqrt(2 / math.pi)
            z = k * (vd + 0.044715 * vd ** 3)
            s = torch.sigmoid(z)
            a, d = vd * s, s + vd * s * torch.sigmoid(-z) * k * (1 + 0.134145 * vd * vd)
        elif act == "relu":
            a, d = vd.clamp(min=0), (vd > 0).double()
        else:
            a, d = vd, torch.ones_like(vd)
        a, d = a.nan_to_num(0.0), d.nan_to_num(0.0)  # inf * 0 of the formulas
        dgate = binding.moe_gated_ffn_backward(dout, eye, eye, zero, eye, v, up, act,
                                               want_dw=False)[0]
        dup = binding.moe_gated_ffn_backward(dout, eye, zero, eye, eye, v, up, act,
                                             want_dw=False)[0]
        for got, ref, mag in ((dgate, dout.double() * 0.5 * d, dout.double().abs()),
                              (dup, dout.double() * a, dout.double().abs() * vd.abs())):
            # two roundings (dgate or dup, dx), the description's 2^-20
            tol = 2.1 * HALF * ref.abs() + 2.0 ** -19 * mag.clamp(max=1e6) + 1e-37
            # dup is an operand in bf16: where dout * 3e38 passes 3.39e38 it is
            # infinite, and the row's product with the zeros of the other weights NaN
            over = ((dout.double() * a).abs() > 3.38e38).any(1, keepdim=True)
            assert int((~over).sum()) >= 8
            ok = ((got.double() - ref).abs() <= tol) | over
            assert bool(ok.all()), (act, v[~ok][:4], got[~ok][:4], ref[~ok][:4])


@pytest.mark.parametrize("N", [1, 64, 300])
@pytest.mark.parametrize("H,I", [(264, 1000), (256, 512)])
def test_arrays_on_16_bytes_only(N, H, I):
    """Rows that start on 16 but not on 32 bytes give the same bits."""
    g = gen(N + H)

    def shifted(t):
        flat = torch.empty(t.numel() + 8, dtype=BF16, device="cuda")
        flat[8:].copy_(t.reshape(-1))
        return flat[8:].view(t.shape)

    wg, wu, wd = weights(g, H, I)
    x, res, dout = normal(g, N, H), normal(g, N, H), normal(g, N, H)
    out, gate, up = binding.moe_gated_ffn(x, wg, wu, wd, residual=res, keep=True)
    first = binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate, up)
    x, res, dout, wg, wu, wd = map(shifted, (x, res, dout, wg, wu, wd))
    out2, gate2, up2 = binding.moe_gated_ffn(x, wg, wu, wd, residual=res, gate=shifted(gate),
                                             up=shifted(up), out=res)  # in place of the residual
    second = binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate2, up2, dx=shifted(x),
                                            dw_gate=shifted(wg), dw_up=shifted(wu),
                                            dw_down=shifted(wd))
    for a, b in zip((out, gate, up, *first), (out2, gate2, up2, *second)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("N", [1, 40, 300, 700])
def test_out_in_place_of_x(N):
    """out = x + FFN(x), written over x."""
    H, I = 512, 1024
    g = gen(N)
    wg, wu, wd = weights(g, H, I)
    x = normal(g, N, H)
    want, _, _ = binding.moe_gated_ffn(x, wg, wu, wd, residual=x)
    got, _, _ = binding.moe_gated_ffn(x, wg, wu, wd, residual=x, out=x)
    assert got is x and torch.equal(got, want)
    want, _, _ = binding.moe_gated_ffn(x, wg, wu, wd)
    binding.moe_gated_ffn(x, wg, wu, wd, out=x)
    assert torch.equal(x, want)


def step(block, x, residual, dout, bufs):
    """A training step into given buffers, without an allocation."""
    normed, mean, rstd = binding.moe_layernorm(
        x, block.norm_weight, block.norm_bias, residual, out=bufs["normed"],
        residual_out=bufs["r"], mean=bufs["mean"], rstd=bufs["rstd"])
    out, gate, up = binding.moe_gated_ffn(
        normed, block.w_gate, block.w_up, block.w_down, residual=bufs["r"], gate=bufs["gate"],
        up=bufs["up"], out=bufs["out"], workspace=bufs["ws"])
    dn, *_ = binding.moe_gated_ffn_backward(
        dout, normed, block.w_gate, block.w_up, block.w_down, gate, up, dx=bufs["dn"],
        dw_gate=bufs["dwg"], dw_up=bufs["dwu"], dw_down=bufs["dwd"], workspace=bufs["ws"])
    binding.moe_layernorm_backward(dn, bufs["r"], block.norm_weight, mean, rstd, dout,
                                   dx=bufs["dr"], dweight=bufs["dnw"], dbias=bufs["dnb"],
                                   workspace=bufs["ws"])
    binding.moe_grad_norm(bufs["set"], norm=bufs["norm"], workspace=bufs["ws"])
    binding.moe_clip_grads(bufs["set"], bufs["norm"], 0.25)


def buffers(N, H, I):
    def e(*s, dtype=BF16):
        return torch.empty(s, dtype=dtype, device="cuda")

    b = {"normed": e(N, H), "r": e(N, H), "mean": e(N, dtype=F32), "rstd": e(N, dtype=F32),
         "gate": e(N, I), "up": e(N, I), "out": e(N, H), "dn": e(N, H), "dwg": e(I, H),
         "dwu": e(I, H), "dwd": e(H, I), "dr": e(N, H), "dnw": e(H, dtype=F32),
         "dnb": e(H, dtype=F32), "norm": e(1, dtype=F32)}
    b["ws"] = e(max(binding.moe_gated_ffn_workspace_bytes(N, H, I),
                    binding.moe_gated_ffn_backward_workspace_bytes(N, H, I),
                    binding.moe_layernorm_backward_workspace_bytes(N, H),
                    binding.moe_grad_norm_workspace_bytes(5)), dtype=torch.uint8)
    b["set"] = binding.GradSet([b["dwg"], b["dwu"], b["dwd"], b["dnw"], b["dnb"]])
    return b


def results(bufs):
    return [bufs[n].clone() for n in ("out", "r", "dr", "dwg", "dwu", "dwd", "dnw", "dnb", "norm")]


@pytest.mark.parametrize("N,H,I", [(1, 512, 1024), (33, 256, 264), (700, 256, 2048)])
def test_step_captured_replayed_and_on_streams(N, H, I):
    g = gen(N)
    block = make_block(g, H, I)
    ins = [[normal(g, N, H) for _ in range(3)] for _ in range(2)]
    bufs = buffers(N, H, I)
    want = []
    for i in ins:
        step(block, *i, bufs)
        want.append(results(bufs))
    # one graph for both inputs, one workspace for all its calls
    held = [t.clone() for t in ins[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(block, *held, bufs)
    for i, w in zip((1, 0, 1), (want[1], want[0], want[1])):
        for h, t in zip(held, ins[i]):
            h.copy_(t)
        graph.replay()
        for a, b in zip(results(bufs), w):
            assert torch.equal(a, b)
    # two streams at once, buffers of their own, several times over
    other = buffers(N, H, I)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, i, b in zip(streams, ins, (bufs, other)):
            with torch.cuda.stream(s):
                step(block, *i, b)
    torch.cuda.synchronize()
    for b, w in zip((bufs, other), want):
        for x, y in zip(results(b), w):
            assert torch.equal(x, y)


def test_weights_written_right_before():
    """Early reads of the next step's weights see what the kernel before the call
    wrote: the down projection is filled anew before every call."""
    g = gen(3)
    for N in (1, 50, 300):
        H, I = 512, 4096
        wg, wu, _ = weights(g, H, I)
        x = normal(g, N, H)
        downs = [normal(g, H, I, std=I ** -0.5) for _ in range(3)]
        want = [binding.moe_gated_ffn(x, wg, wu, d)[0] for d in downs]
        torch.cuda.synchronize()
        live, out = torch.empty_like(downs[0]), torch.empty(6, N, H, dtype=BF16, device="cuda")
        ws = torch.empty(binding.moe_gated_ffn_workspace_bytes(N, H, I), dtype=torch.uint8,
                         device="cuda")
        for i in range(6):
            live.copy_(downs[i % 3])
            binding.moe_gated_ffn(x, wg, wu, live, out=out[i], workspace=ws)
        for i in range(6):
            assert torch.equal(out[i], want[i % 3])


def test_no_tokens():
    H, I = 64, 128
    wg, wu, wd = weights(gen(0), H, I)
    x = torch.empty(0, H, dtype=BF16, device="cuda")
    out, gate, up = binding.moe_gated_ffn(x, wg, wu, wd, keep=True)
    assert out.shape == (0, H) and gate.shape == up.shape == (0, I)
    dw = [torch.full_like(t, 7.0) for t in (wg, wu, wd)]
    dx, *got = binding.moe_gated_ffn_backward(x, x, wg, wu, wd, gate, up, dw_gate=dw[0],
                                              dw_up=dw[1], dw_down=dw[2])
    assert dx.shape == (0, H)
    for t in got:
        assert not bool(t.any())


def test_gradients_of_one_kind():
    g = gen(9)
    N, H, I = 150, 128, 136
    wg, wu, wd = weights(g, H, I)
    x, dout = normal(g, N, H), normal(g, N, H)
    _, gate, up = binding.moe_gated_ffn(x, wg, wu, wd, keep=True)
    both = binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate, up)
    no_dx = binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate, up, want_dx=False)
    no_dw = binding.moe_gated_ffn_backward(dout, x, wg, wu, wd, gate, up, want_dw=False)
    assert no_dx[0] is None and all(torch.equal(a, b) for a, b in zip(no_dx[1:], both[1:]))
    assert no_dw[1:] == (None, None, None) and torch.equal(no_dw[0], both[0])
