"""Refusals of the dense block's operators, on the host: every bad argument is
rejected before anything is enqueued."""
import ctypes

import pytest
import torch

from sparse_moe_ffn_gb300 import binding
from sparse_moe_ffn_gb300 import build as lib_build
from test_block_ops_devices_host import Library, Stand

OK, INVALID, SMALL, UNSUPPORTED = 0, 1, 2, 3
P = 0x10000  # 256-byte aligned, never dereferenced: validation fails first
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    lib_build.build()
    return binding.lib()


def test_gated_ffn_argument_errors(L):
    need = L.moe_gated_ffn_workspace_bytes(300, 64, 128)
    assert need >= 256 + 2 * 300 * 128
    assert L.moe_gated_ffn_workspace_bytes(-1, 64, 128) == 0
    assert L.moe_gated_ffn_workspace_bytes(4, 60, 128) == 0

    def call(x=P, wg=P, wu=P, wd=P, r=P, N=300, H=64, I=128, act=1, g=2 * P, u=3 * P, out=4 * P,
             ws=P, wsb=need):
        return L.moe_gated_ffn(x, wg, wu, wd, r, N, H, I, act, g, u, out, ws, wsb, None)

    assert call(N=-1) == INVALID
    for H in (0, -8, 60, 4):
        assert call(H=H) == INVALID, H
        assert call(I=H) == INVALID, H
    assert call(act=5) == INVALID and call(act=-1) == INVALID
    assert call(N=1 << 30) == UNSUPPORTED
    assert call(H=1 << 30) == UNSUPPORTED
    assert call(I=1 << 30) == UNSUPPORTED
    assert call(H=1 << 23, I=1 << 23) == UNSUPPORTED  # tiles of a weight's gradient
    assert call(N=1 << 23, I=1 << 23) == UNSUPPORTED
    for name in ("x", "wg", "wu", "wd", "out", "ws"):
        assert call(**{name: None}) == INVALID, name
    assert call(g=None) == INVALID and call(u=None) == INVALID
    assert call(u=2 * P) == INVALID and call(g=4 * P) == INVALID
    for name in ("x", "wg", "wu", "wd", "r", "g", "u", "out"):
        assert call(**{name: 7 * P + 8}) == INVALID, name
    assert b"aligned" in L.moe_last_error()
    assert call(ws=P + 64) == INVALID
    assert call(wsb=need - 1) == SMALL
    assert call(N=0, x=None, ws=None) == OK


def test_gated_ffn_backward_argument_errors(L):
    need = L.moe_gated_ffn_backward_workspace_bytes(300, 64, 128)
    assert need >= 256 + 3 * 2 * 300 * 128
    assert L.moe_gated_ffn_backward_workspace_bytes(300, 64, 0) == 0

    def call(dy=P, x=P, wg=P, wu=P, wd=P, g=P, u=P, N=300, H=64, I=128, act=1, dx=2 * P, dg=3 * P,
             du=4 * P, dd=5 * P, ws=P, wsb=need):
        return L.moe_gated_ffn_backward(dy, x, wg, wu, wd, g, u, N, H, I, act, dx, dg, du, dd, ws,
                                        wsb, None)

    assert call(N=-1) == INVALID
    assert call(H=12) == INVALID and call(I=12) == INVALID
    assert call(act=9) == INVALID
    assert call(N=1 << 30) == UNSUPPORTED
    for name in ("dy", "x", "wg", "wu", "wd", "g", "u", "ws"):
        assert call(**{name: None}) == INVALID, name
    for name in ("dg", "du", "dd"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: 2 * P}) == INVALID, name  # dx's
    assert call(du=3 * P) == INVALID and call(dd=4 * P) == INVALID
    for name in ("dy", "x", "wg", "wu", "wd", "g", "u", "dx", "dg", "du", "dd"):
        assert call(**{name: 7 * P + 8}) == INVALID, name
    assert call(ws=P + 128) == INVALID
    assert call(wsb=need - 1) == SMALL
    assert call(N=0, dy=None, dg=None, du=None, dd=None, ws=None) == OK


def test_layernorm_argument_errors(L):
    def call(x=P, r=P, w=P, b=P, bf16=1, N=4, H=64, eps=1e-5, ro=2 * P, out=3 * P, m=P, s=P):
        return L.moe_layernorm(x, r, w, b, bf16, N, H, eps, ro, out, m, s, None)

    assert call(N=-1) == INVALID
    assert call(H=0) == INVALID
    assert call(H=65537) == UNSUPPORTED
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    for name in ("x", "w", "out"):
        assert call(**{name: None}) == INVALID, name
    assert call(ro=3 * P) == INVALID  # out's
    for name in ("x", "r", "w", "b", "ro", "out"):
        assert call(**{name: 7 * P + 1}) == INVALID, name
        assert call(bf16=0, **{name: 7 * P + 2}) == INVALID, name
    for name in ("m", "s"):
        assert call(**{name: P + 2}) == INVALID, name
    assert call(N=0, x=None, out=None) == OK

    need = L.moe_layernorm_backward_workspace_bytes(1000, 64)
    assert need > 0 and need % 256 == 0
    assert L.moe_layernorm_backward_workspace_bytes(-1, 64) == 0
    assert L.moe_layernorm_backward_workspace_bytes(4, 70000) == 0

    def bwd(dy=P, x=P, w=P, m=P, s=P, dr=P, bf16=1, N=1000, H=64, dx=P, dw=P, db=P, ws=P, wsb=need):
        return L.moe_layernorm_backward(dy, x, w, m, s, dr, bf16, N, H, dx, dw, db, ws, wsb, None)

    assert bwd(N=-1) == INVALID
    assert bwd(H=0) == INVALID and bwd(H=65537) == UNSUPPORTED
    for name in ("dy", "x", "w", "m", "s", "ws"):
        assert bwd(**{name: None}) == INVALID, name
    for name in ("dy", "x", "w", "dr", "dx"):
        assert bwd(**{name: P + 1}) == INVALID, name
        assert bwd(bf16=0, **{name: P + 2}) == INVALID, name
    for name in ("m", "s", "dw", "db"):
        assert bwd(**{name: P + 2}) == INVALID, name
    assert bwd(ws=P + 8) == INVALID
    assert bwd(wsb=need - 1) == SMALL
    assert bwd(dx=None, dw=None, db=None, ws=None) == OK  # nothing is wanted
    assert bwd(N=0, dy=None, dw=None, db=None) == OK


def test_grad_clip_argument_errors(L):
    need = L.moe_grad_norm_workspace_bytes(2)
    assert need > 0 and L.moe_grad_norm_workspace_bytes(0) == need
    assert L.moe_grad_norm_workspace_bytes(-1) == 0
    assert L.moe_grad_norm_workspace_bytes((1 << 20) + 1) == 0
    sizes = (ctypes.c_int64 * 2)(100, 7)

    def both(ptr=(P, P), n=2, sizes=sizes, flags=b"\0\1", norm=P, ws=P, wsb=need, out=(P, P),
             out_flags=b"\0\1", max_norm=1.0, null=()):
        src = (ctypes.c_void_p * 2)(*ptr)
        dst = (ctypes.c_void_p * 2)(*out)
        args = [None if "src" in null else src, None if "sizes" in null else sizes,
                None if "flags" in null else flags, n]
        a = L.moe_grad_norm(*args, norm, ws, wsb, None)
        b = L.moe_clip_grads(*args, norm, max_norm, None if "dst" in null else dst,
                             None if "out_flags" in null else out_flags, None)
        return a, b

    assert both(n=-1) == (INVALID, INVALID)
    assert both(n=(1 << 20) + 1) == (UNSUPPORTED, UNSUPPORTED)
    for name in ("src", "sizes", "flags"):
        assert both(null=(name,)) == (INVALID, INVALID), name
    assert both(ptr=(P, 0)) == (INVALID, INVALID)
    assert both(ptr=(P + 2, P)) == (INVALID, INVALID)
    assert both(ptr=(P, P + 1)) == (INVALID, INVALID)
    assert both(sizes=(ctypes.c_int64 * 2)(100, -1)) == (INVALID, INVALID)
    assert both(sizes=(ctypes.c_int64 * 2)(100, (1 << 40) + 1)) == (INVALID, INVALID)
    assert both(norm=None) == (INVALID, INVALID) and both(norm=P + 2) == (INVALID, INVALID)

    def clip(**kw):
        src = (ctypes.c_void_p * 2)(P, P)
        dst = (ctypes.c_void_p * 2)(*kw.get("out", (P, P)))
        return L.moe_clip_grads(src, sizes, b"\0\1", 2, P, kw.get("max_norm", 1.0),
                                None if kw.get("no_out") else dst,
                                None if kw.get("no_flags") else b"\0\1", None)

    assert clip(no_out=True) == INVALID and clip(no_flags=True) == INVALID
    assert clip(out=(0, P)) == INVALID and clip(out=(P + 2, P)) == INVALID
    assert clip(max_norm=-1.0) == INVALID and clip(max_norm=float("nan")) == INVALID

    def norm(ws=P, wsb=need):
        return L.moe_grad_norm((ctypes.c_void_p * 2)(P, P), sizes, b"\0\1", 2, P, ws, wsb, None)

    assert norm(ws=None) == INVALID and norm(ws=P + 8) == INVALID
    assert norm(wsb=need - 1) == SMALL


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 64, dtype=BF16)
    v = torch.zeros(64, dtype=BF16)
    w = torch.zeros(128, 64, dtype=BF16)
    d = torch.zeros(64, 128, dtype=BF16)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_gated_ffn(x, w, w, d)
    with pytest.raises(ValueError, match="activation"):
        binding.moe_gated_ffn(x, w, w, d, "swish")
    with pytest.raises(ValueError, match="two dimensions"):
        binding.moe_gated_ffn(v, w, w, d)
    with pytest.raises(ValueError, match="two dimensions"):
        binding.moe_gated_ffn(x, v, w, d)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_gated_ffn_backward(x, x, w, w, d, x, x)
    with pytest.raises(ValueError, match="activation"):
        binding.moe_gated_ffn_backward(x, x, w, w, d, x, x, "swish")
    with pytest.raises(ValueError, match="bf16 or fp32"):
        binding.moe_layernorm(x.half(), v)
    with pytest.raises(ValueError, match="two dimensions"):
        binding.moe_layernorm(v, v)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_layernorm(x, v)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_layernorm_backward(x, x, v, f, f)
    with pytest.raises(ValueError, match="CUDA"):
        binding.moe_grad_norm([x])
    with pytest.raises(ValueError, match="at least one"):
        binding.moe_grad_norm([])


N, H, I = 4, 64, 128
FFN = dict(x=(BF16, N, H), w_gate=(BF16, I, H), w_up=(BF16, I, H), w_down=(BF16, H, I),
           gate=(BF16, N, I), up=(BF16, N, I), workspace=(torch.uint8, 1 << 20))


def ffn(**t):
    return binding.moe_gated_ffn(t["x"], t["w_gate"], t["w_up"], t["w_down"], residual=t["residual"],
                                 gate=t["gate"], up=t["up"], out=t["out"],
                                 workspace=t["workspace"])


def ffn_backward(**t):
    return binding.moe_gated_ffn_backward(
        t["dout"], t["x"], t["w_gate"], t["w_up"], t["w_down"], t["gate"], t["up"], dx=t["dx"],
        dw_gate=t["dw_gate"], dw_up=t["dw_up"], dw_down=t["dw_down"], workspace=t["workspace"])


def layernorm(**t):
    return binding.moe_layernorm(t["x"], t["weight"], t["bias"], t["residual"], out=t["out"],
                                 residual_out=t["residual_out"], mean=t["mean"], rstd=t["rstd"])


def layernorm_backward(**t):
    return binding.moe_layernorm_backward(t["dout"], t["x"], t["weight"], t["mean"], t["rstd"],
                                          t["dresidual"], dx=t["dx"], dweight=t["dweight"],
                                          dbias=t["dbias"], workspace=t["workspace"])


def grad_norm(**t):
    return binding.moe_grad_norm([t["a"], t["b"]], norm=t["norm"], workspace=t["workspace"])


def clip_grads(**t):
    return binding.moe_clip_grads([t["a"], t["b"]], t["norm"], 1.0, out=[t["c"], t["d"]])


CASES = {
    "ffn": (ffn, dict(FFN, residual=(BF16, N, H), out=(BF16, N, H))),
    "ffn backward": (ffn_backward, dict(FFN, dout=(BF16, N, H), dx=(BF16, N, H),
                                        dw_gate=(BF16, I, H), dw_up=(BF16, I, H),
                                        dw_down=(BF16, H, I))),
    "layernorm": (layernorm, dict(x=(F32, N, H), residual=(F32, N, H), weight=(F32, H),
                                  bias=(F32, H), out=(F32, N, H), residual_out=(F32, N, H),
                                  mean=(F32, N), rstd=(F32, N))),
    "layernorm backward": (layernorm_backward,
                           dict(dout=(BF16, N, H), x=(BF16, N, H), weight=(BF16, H),
                                mean=(F32, N), rstd=(F32, N), dresidual=(BF16, N, H),
                                dx=(BF16, N, H), dweight=(F32, H), dbias=(F32, H),
                                workspace=(torch.uint8, 1 << 20))),
    "grad norm": (grad_norm, dict(a=(BF16, 9), b=(F32, 3, 4), norm=(F32, 1),
                                  workspace=(torch.uint8, 1 << 20))),
    "clip": (clip_grads, dict(a=(BF16, 9), b=(F32, 3, 4), norm=(F32, 1), c=(F32, 9), d=(BF16, 12))),
}


class Placed(Stand):
    """Stand-ins that do not lie in one another."""
    places = 1

    def __init__(self, *spec, index=0):
        super().__init__(*spec, index=index)
        Placed.places += 1
        self.place = Placed.places << 20

    def data_ptr(self):
        return self.place


@pytest.fixture
def library(monkeypatch):
    fake = Library()
    monkeypatch.setattr(binding, "lib", lambda: fake)
    monkeypatch.setattr(binding, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    return fake


@pytest.mark.parametrize("name", CASES)
def test_operands_on_one_device(library, name, monkeypatch):
    call, specs = CASES[name]
    call(**{n: Placed(*s) for n, s in specs.items()})
    assert library.calls == 1
    for other in specs:  # each of them in turn elsewhere
        with pytest.raises(ValueError, match="cuda:"):
            call(**{n: Placed(*s, index=int(n == other)) for n, s in specs.items()})
    # all together elsewhere, with the current device unchanged
    with pytest.raises(ValueError, match="current device"):
        call(**{n: Placed(*s, index=1) for n, s in specs.items()})
    assert library.calls == 1
    monkeypatch.setattr(binding, "_current_device", lambda: 1)
    call(**{n: Placed(*s, index=1) for n, s in specs.items()})
    assert library.calls == 2


@pytest.mark.parametrize("name", ["ffn", "ffn backward", "layernorm", "layernorm backward"])
def test_shapes_and_types(library, name):
    call, specs = CASES[name]
    for other, spec in specs.items():
        if other == "workspace":
            continue
        wrong = [(torch.float16, *spec[1:])]
        if other not in ("x", "w_gate"):  # these say what the sizes are
            wrong.append((spec[0], *[n + 8 for n in spec[1:]]))
        for w in wrong:
            with pytest.raises(ValueError):
                call(**{n: Placed(*(w if n == other else s)) for n, s in specs.items()})
    assert library.calls == 0


class At(Stand):
    def __init__(self, dtype, n, place):
        super().__init__(dtype, n)
        self.place = place

    def data_ptr(self):
        return self.place


def test_clipped_gradients_lie_in_their_own_only():
    a, b = At(F32, 100, P), At(BF16, 100, P + 400)  # b right behind a
    binding.GradSet([a, b])
    binding.GradSet([a, b], [At(F32, 100, P), At(BF16, 100, 2 * P)])
    binding.GradSet([a, a], [At(F32, 100, 2 * P), At(F32, 100, 3 * P)])  # read twice
    binding.GradSet([], [])
    bad = [
        ([a, a], None),                                             # written twice
        ([a, At(F32, 100, P + 396)], None),                         # ends in the next
        ([a, b], [At(F32, 100, 2 * P), At(F32, 100, 2 * P + 200)]),  # outputs overlap
        ([a, b], [At(F32, 100, P + 4), At(BF16, 100, 2 * P)]),      # shifted in its own
        ([a, b], [At(BF16, 100, P), At(BF16, 100, 2 * P)]),         # its own, another type
        ([a, b], [At(F32, 100, P + 400), At(BF16, 100, 2 * P)]),    # in another gradient
        ([At(F32, 1000, P), At(F32, 4, 8 * P)], [At(F32, 1000, 2 * P), At(F32, 4, P + 800)]),
        ([At(F32, 1000, P), At(F32, 4, 8 * P)], [At(F32, 1000, 2 * P), At(F32, 4, 2 * P + 800)]),
    ]
    for grads, out in bad:
        with pytest.raises(ValueError, match="overlap"):
            binding.GradSet(grads, out)
    with pytest.raises(ValueError, match="as many"):
        binding.GradSet([a, b], [a])
    with pytest.raises(ValueError, match="100 values"):
        binding.GradSet([a], [At(F32, 99, 2 * P)])
    with pytest.raises(ValueError, match="bf16 or fp32"):
        binding.GradSet([At(torch.float16, 8, P)])
    with pytest.raises(ValueError, match="out tensors already"):
        binding.moe_clip_grads(binding.GradSet([a]), None, 1.0, out=[a])


def test_outputs_that_overlap_are_refused(L):
    """Each array 256 KB from the next, 300 x 64 and 300 x 128 of them used."""
    at = {n: (i + 1) << 18 for i, n in enumerate(
        "x wg wu wd r gate up out dy dx dg du dd w b ro m s dr dw db ws".split())}
    need = L.moe_gated_ffn_backward_workspace_bytes(300, 64, 128)

    def refused(function, names, **change):
        p = {**at, **{n: at[v] if isinstance(v, str) else v for n, v in change.items()}}
        status = getattr(L, function)(*(p.get(n, n) if isinstance(n, str) else n for n in names),
                                      None)
        return status == INVALID and b"overlap" in L.moe_last_error()

    def forward(**change):
        return refused("moe_gated_ffn", ["x", "wg", "wu", "wd", "r", 300, 64, 128, 1, "gate", "up",
                                         "out", "ws", need], **change)

    for name in ("wg", "wu", "wd"):
        assert forward(out=name), name
    for name in ("x", "wg", "wu", "wd", "r"):
        assert forward(gate=name) and forward(up=name), name
        assert forward(up=at[name] - 16), name
    assert forward(out=at["r"] + 128) and forward(out=at["x"] - 128)
    assert forward(up=at["gate"] + 300 * 128 * 2 - 16) and forward(out=at["up"] + 16)

    def backward(**change):
        return refused("moe_gated_ffn_backward", ["dy", "x", "wg", "wu", "wd", "gate", "up", 300,
                                                  64, 128, 1, "dx", "dg", "du", "dd", "ws", need],
                       **change)

    for name in ("dy", "x", "wg", "wu", "wd", "gate", "up"):
        for out in ("dx", "dg", "du", "dd"):
            assert backward(**{out: name}), (out, name)
    assert backward(dx=at["dy"] + 128) and backward(du=at["dg"] + 16)

    def norm(**change):
        return refused("moe_layernorm", ["x", "r", "w", "b", 1, 300, 64, 1e-5, "ro", "out", "m",
                                         "s"], **change)

    for out in ("out", "ro", "m", "s"):
        assert norm(**{out: "w"}) and norm(**{out: "b"}), out
    assert norm(out=at["x"] + 128) and norm(ro=at["r"] - 128) and norm(out=at["ro"] + 2)
    assert norm(m="x") and norm(s="m")

    def norm_backward(**change):
        return refused("moe_layernorm_backward", ["dy", "x", "w", "m", "s", "dr", 1, 300, 64, "dx",
                                                  "dw", "db", "ws", need], **change)

    for name in ("w", "m", "s"):
        assert norm_backward(dx=name), name
    for name in ("dy", "x", "dr", "w", "m", "s", "dx"):
        assert norm_backward(dw=name) and norm_backward(db=name), name
    assert norm_backward(dx=at["dy"] + 128) and norm_backward(db="dw")
