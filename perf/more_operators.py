"""Measured cases of the operators that train and serve a dense decoder block.

  ffn        the gated feed-forward block (act(x Wg^T) * (x Wu^T)) Wd^T onto a
             residual; train: forward that keeps both projections, then the
             gradients of x and of the three weights
  layernorm  residual add + layer norm with a row's mean and 1/std; train: then
             the gradients of x (onto the residual stream's own), of the weight
             and of the bias
  clip       the norm of a whole set of gradient tensors, then the set scaled so
             that its norm is max_norm at most

Each case is one pass a user makes.  ``run`` computes it in plain torch
operations, or with the library's entry points when ``own`` is set; ``exact``
computes it in 64 bits.
"""
import math
import random

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "fp32": F32}
EPS = 1e-5
ACTS = ("silu", "gelu", "gelu_tanh")


# ------------------------------------------------------------------ the cases

def _ffn(name, N, H, I, act="silu", train=False, residual=True):
    return dict(name=name, op="ffn", N=N, H=H, I=I, act=act, train=train, residual=residual)


def _layernorm(name, N, H, train, dtype="bf16", residual=True, bias=True):
    return dict(name=name, op="layernorm", N=N, H=H, train=train, dtype=dtype, residual=residual,
                bias=bias)


def _clip(name, layout, count=0, total=0, shape_seed=0, dtype="bf16", out="same"):
    return dict(name=name, op="clip", layout=layout, count=count, total=total,
                shape_seed=shape_seed, dtype=dtype, out=out)


def listed():
    return [
        # one new token of one sequence through a dense layer: weight streaming
        _ffn("ffn one token", 1, 2048, 8192),
        # a decode batch of 64 sequences
        _ffn("ffn decode", 64, 2048, 8192),
        # a prefill batch: tensor cores
        _ffn("ffn prefill", 8192, 2048, 8192),
        # a training step of a block as wide as one expert of the sparse layer
        _ffn("ffn train narrow", 2048, 2048, 768, train=True),
        # packed sequences of odd lengths, sizes that end inside every tile
        _ffn("ffn train ragged", 1021, 1000, 1400, "gelu_tanh", train=True, residual=False),
        # a training step of the wide block
        _ffn("ffn train", 8192, 2048, 8192, train=True),
        # one token enters a block: latency
        _layernorm("layernorm one token", 1, 2048, False),
        # a training batch through a block's norm, both ways: bandwidth
        _layernorm("layernorm train", 16384, 2048, True),
        # fp32 activations, rows of odd length
        _layernorm("layernorm train ragged", 1021, 1111, True, "fp32", False),
        # biases and norm weights, many small tensors: latency
        _clip("clip small tensors", "small", dtype="fp32"),
        # the gradients of one dense block
        _clip("clip dense block", "dense"),
        # the gradients of the sparse layer (128 experts), into fp32 for the optimizer
        _clip("clip sparse layer", "sparse", out="fp32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


MAX_FFN_FLOPS = 18 * 8192 * 2048 * 8192
MAX_FFN_WEIGHTS = 4096 * 12288
MAX_ROWS = 16384 * 2048
MAX_GRADS = 3 * 128 * 768 * 2048


def draw(rng):
    op = rng.choice(("ffn", "ffn", "layernorm", "clip"))
    if op == "ffn":
        train = rng.random() < 0.5
        while True:
            N = _log_int(rng, 1, 16384)
            H = max(64, _log_int(rng, 64, 4096) // 8 * 8)
            I = max(64, _log_int(rng, 64, 12288) // 8 * 8)
            if (18 if train else 6) * N * H * I <= MAX_FFN_FLOPS and H * I <= MAX_FFN_WEIGHTS:
                break
        c = _ffn("", N, H, I, rng.choice(ACTS), train, rng.random() < 0.5)
    elif op == "layernorm":
        while True:
            N, H = _log_int(rng, 1, 65536), _log_int(rng, 16, 16384)
            if rng.random() < 0.5:
                H = max(8, H // 8 * 8)
            if N * H <= MAX_ROWS:
                break
        c = _layernorm("", N, H, rng.random() < 0.7, rng.choice(("bf16", "fp32")),
                       rng.random() < 0.6, rng.random() < 0.7)
    else:
        count = _log_int(rng, 1, 60)
        c = _clip("", "mixed", count, _log_int(rng, max(count, 1000), MAX_GRADS // 4),
                  rng.randrange(1 << 30), rng.choice(("bf16", "fp32", "both")),
                  rng.choice(("same", "fp32")))
    del c["name"]
    return c


def _tensors(c):
    """(elements, type) of each gradient of a clip case."""
    if c["layout"] == "small":
        sizes = [n for _ in range(15) for n in (2048, 2048, 389, 8192)]
    elif c["layout"] == "dense":
        sizes = [8192 * 2048, 8192 * 2048, 2048 * 8192, 2048, 2048]
    elif c["layout"] == "sparse":
        sizes = [128 * 2048] + [128 * 768 * 2048] * 3 + [2048]
    else:
        # parts of a whole, a few of them large as weights are among biases
        r = random.Random(c["shape_seed"])
        parts = [math.exp(r.gauss(0.0, 2.0)) for _ in range(c["count"])]
        sizes = [max(1, int(p / sum(parts) * c["total"])) for p in parts]
    if c["dtype"] == "both":
        r = random.Random(c["shape_seed"] + 1)
        return [(n, r.choice((BF16, F32))) for n in sizes]
    return [(n, DTYPES[c["dtype"]]) for n in sizes]


# ------------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=F32) * std

    def empty(*shape, dtype=BF16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    s = {"case": c}
    if c["op"] == "ffn":
        N, H, I = c["N"], c["H"], c["I"]
        s["x"] = normal(N, H).to(BF16)  # a normed hidden state
        s["w_gate"] = normal(I, H, std=H ** -0.5).to(BF16)
        s["w_up"] = normal(I, H, std=H ** -0.5).to(BF16)
        s["w_down"] = normal(H, I, std=I ** -0.5).to(BF16)
        s["residual"] = normal(N, H, std=2.0).to(BF16) if c["residual"] else None
        s["out"] = empty(N, H)
        if c["train"]:
            s["dout"] = normal(N, H, std=0.01).to(BF16)
            s["gate"], s["up"] = empty(N, I), empty(N, I)
            s["dx"] = empty(N, H)
            s["dw_gate"], s["dw_up"], s["dw_down"] = empty(I, H), empty(I, H), empty(H, I)
        if own:
            from sparse_moe_ffn_gb300 import binding as b
            n = b.moe_gated_ffn_workspace_bytes(N, H, I)
            if c["train"]:
                n = max(n, b.moe_gated_ffn_backward_workspace_bytes(N, H, I))
            s["workspace"] = empty(n, dtype=torch.uint8)
    elif c["op"] == "layernorm":
        N, H, dtype = c["N"], c["H"], DTYPES[c["dtype"]]
        # a residual stream: larger than one layer's output, off zero, with a
        # few channels far above the others
        spread = 1.0 + 20.0 * (torch.rand(H, generator=g, device="cuda") < 0.005).float()
        s["x"] = (normal(N, H) * (1.0 if c["residual"] else spread) + 0.25).to(dtype)
        s["residual"] = (normal(N, H, std=4.0) * spread).to(dtype) if c["residual"] else None
        s["weight"] = (1.0 + normal(H, std=0.1)).to(dtype)
        s["bias"] = normal(H, std=0.1).to(dtype) if c["bias"] else None
        s["out"], s["mean"], s["rstd"] = empty(N, H, dtype=dtype), empty(N, dtype=F32), empty(
            N, dtype=F32)
        s["residual_out"] = empty(N, H, dtype=dtype) if c["residual"] else None
        if c["train"]:
            s["dout"] = normal(N, H, std=0.01).to(dtype)
            s["dresidual"] = normal(N, H, std=0.01).to(dtype) if c["residual"] else None
            s["dx"] = empty(N, H, dtype=dtype)
            s["dweight"] = empty(H, dtype=F32)
            s["dbias"] = empty(H, dtype=F32) if c["bias"] else None
            if own:
                from sparse_moe_ffn_gb300 import binding as b
                s["workspace"] = empty(b.moe_layernorm_backward_workspace_bytes(N, H),
                                       dtype=torch.uint8)
    else:
        tensors = _tensors(c)
        # gradients whose size differs from tensor to tensor; the norm of all is
        # a few times the one allowed
        s["grads"] = [normal(n, std=1e-3 * (1.0 + i % 5)).to(t) for i, (n, t) in enumerate(tensors)]
        s["max_norm"] = 1e-3 * math.sqrt(sum(n for n, _ in tensors))
        s["clipped"] = [empty(n, dtype=F32 if c["out"] == "fp32" else t) for n, t in tensors]
        s["norm"] = empty(1, dtype=F32)
        if own:
            from sparse_moe_ffn_gb300 import binding as b
            s["workspace"] = empty(b.moe_grad_norm_workspace_bytes(len(tensors)),
                                   dtype=torch.uint8)
            # a program whose gradients keep their buffers from step to step
            s["set"] = b.GradSet(s["grads"], out=s["clipped"])
    return s


# --------------------------------------------------------------- the plain form

def _act(v, act):
    """(act(v), its derivative)"""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-v))
        return v * s, s * (1.0 + v * (1.0 - s))
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))
        return v * cdf, cdf + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    a = math.sqrt(2.0 / math.pi)
    t = torch.tanh(a * (v + 0.044715 * v * v * v))
    return (0.5 * v * (1.0 + t),
            0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * a * (1.0 + 3.0 * 0.044715 * v * v))


def _plain_ffn(s):
    c = s["case"]
    x, wg, wu, wd = (s[n].float() for n in ("x", "w_gate", "w_up", "w_down"))
    gate, up = x @ wg.T, x @ wu.T
    a, slope = _act(gate, c["act"])
    h = a * up
    out = h @ wd.T
    if s["residual"] is not None:
        out = out + s["residual"].float()
    r = {"out": out.to(BF16)}
    if c["train"]:
        dout = s["dout"].float()
        dh = dout @ wd
        dgate, dup = dh * up * slope, dh * a
        r["dx"] = (dgate @ wg + dup @ wu).to(BF16)
        r["dw_gate"] = (dgate.T @ x).to(BF16)
        r["dw_up"] = (dup.T @ x).to(BF16)
        r["dw_down"] = (dout.T @ h).to(BF16)
    return r


def _plain_layernorm(s):
    c = s["case"]
    dtype = s["x"].dtype
    r = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dtype)
    rf, w = r.float(), s["weight"].float()
    mean = rf.mean(1, keepdim=True)
    d = rf - mean
    rstd = 1.0 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    n = d * rstd
    y = n * w
    if s["bias"] is not None:
        y = y + s["bias"].float()
    out = {"out": y.to(dtype), "mean": mean[:, 0], "rstd": rstd[:, 0],
           "residual": r if c["residual"] else None}
    if c["train"]:
        dy = s["dout"].float()
        t = dy * w
        dx = rstd * (t - t.mean(1, keepdim=True) - n * (t * n).mean(1, keepdim=True))
        if s["dresidual"] is not None:
            dx = dx + s["dresidual"].float()
        out["dx"] = dx.to(dtype)
        out["dweight"] = (dy * n).sum(0, dtype=torch.float64).float()  # sums over all tokens
        out["dbias"] = dy.sum(0, dtype=torch.float64).float() if c["bias"] else None
    return out


def _plain_clip(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")  # a long sum: 64 bits
    for t in s["grads"]:
        f = t.float()
        total = total + (f * f).sum(dtype=torch.float64)
    norm = torch.sqrt(total).float()
    factor = torch.where(norm <= s["max_norm"], torch.ones_like(norm), s["max_norm"] / norm)
    return {"norm": norm.reshape(1),
            "grads": [(t.float() * factor).to(o.dtype) for t, o in zip(s["grads"], s["clipped"])]}


# --------------------------------------------------------------- the library's

def _own_ffn(s):
    from sparse_moe_ffn_gb300 import binding as b
    c = s["case"]
    if not c["train"]:
        out, _, _ = b.moe_gated_ffn(s["x"], s["w_gate"], s["w_up"], s["w_down"],
                                    activation=c["act"], residual=s["residual"], out=s["out"],
                                    workspace=s["workspace"])
        return {"out": out}
    out, gate, up = b.moe_gated_ffn(s["x"], s["w_gate"], s["w_up"], s["w_down"],
                                    activation=c["act"], residual=s["residual"], gate=s["gate"],
                                    up=s["up"], out=s["out"], workspace=s["workspace"])
    dx, dwg, dwu, dwd = b.moe_gated_ffn_backward(
        s["dout"], s["x"], s["w_gate"], s["w_up"], s["w_down"], gate, up, activation=c["act"],
        dx=s["dx"], dw_gate=s["dw_gate"], dw_up=s["dw_up"], dw_down=s["dw_down"],
        workspace=s["workspace"])
    return {"out": out, "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}


def _own_layernorm(s):
    from sparse_moe_ffn_gb300 import binding as b
    c = s["case"]
    out, mean, rstd = b.moe_layernorm(s["x"], s["weight"], bias=s["bias"], residual=s["residual"],
                                      eps=EPS, out=s["out"], mean=s["mean"], rstd=s["rstd"],
                                      residual_out=s["residual_out"])
    r = {"out": out, "mean": mean, "rstd": rstd, "residual": s["residual_out"]}
    if c["train"]:
        x = s["x"] if s["residual"] is None else s["residual_out"]
        r["dx"], r["dweight"], r["dbias"] = b.moe_layernorm_backward(
            s["dout"], x, s["weight"], mean, rstd, dresidual=s["dresidual"], dx=s["dx"],
            dweight=s["dweight"], dbias=s["dbias"], want_dbias=c["bias"],
            workspace=s["workspace"])
    return r


def _own_clip(s):
    from sparse_moe_ffn_gb300 import binding as b
    norm = b.moe_grad_norm(s["set"], norm=s["norm"], workspace=s["workspace"])
    return {"norm": norm, "grads": b.moe_clip_grads(s["set"], norm, s["max_norm"])}


def run(state):
    op = state["case"]["op"]
    if op == "ffn":
        return _own_ffn(state) if own else _plain_ffn(state)
    if op == "layernorm":
        return _own_layernorm(state) if own else _plain_layernorm(state)
    return _own_clip(state) if own else _plain_clip(state)


# ------------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "ffn":
        N, H, I = c["N"], c["H"], c["I"]
        b = 2 * (3 * H * I + 2 * N * H + (N * H if c["residual"] else 0))
        if c["train"]:  # dout read, dx and the weights' gradients written
            b += 2 * (2 * N * H + 3 * H * I)
        return {"bytes": b, "flops": (18 if c["train"] else 6) * N * H * I}
    if c["op"] == "layernorm":
        N, H, size = c["N"], c["H"], 4 if c["dtype"] == "fp32" else 2
        # x and the residual read, the sum and the output written; a loss lies
        # between the passes, so the second one reads the sum again
        per = 4 if c["residual"] else 2
        if c["train"]:
            per += 4 if c["residual"] else 3
        return {"bytes": N * H * per * size + 8 * N + 2 * size * H,
                "flops": N * H * (20 if c["train"] else 8)}
    sizes = _tensors(c)
    read = sum(n * (2 if t is BF16 else 4) for n, t in sizes)
    total = sum(n for n, _ in sizes)
    written = 4 * total if c["out"] == "fp32" else read
    # the norm is known once everything was read: what the L2 does not hold
    # until then is read again
    again = read if read > 100e6 else 0
    return {"bytes": read + again + written, "flops": 3 * total}


# ----------------------------------------------------------------------- exact

def exact(case, seed):
    """The case's outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    if case["op"] == "ffn":
        x, wg, wu, wd = (s[n].double() for n in ("x", "w_gate", "w_up", "w_down"))
        g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        if case["act"] == "silu":
            sg = torch.sigmoid(g)
            a, slope = g * sg, torch.addcmul(sg, g * sg, 1 - sg)
        elif case["act"] == "gelu":
            cdf = torch.special.ndtr(g)
            a = g * cdf
            slope = cdf + g * torch.exp(-g.square() / 2) * (2 * math.pi) ** -0.5
        else:
            # (1 + tanh z) / 2 is the logistic function of 2 z
            k = 2 * math.sqrt(2 / math.pi)
            sg = torch.sigmoid(k * (g + 0.044715 * g.pow(3)))
            a = g * sg
            slope = sg + g * sg * (1 - sg) * k * (1 + 0.134145 * g.square())
        h = a * u
        y = torch.mm(h, wd.t())
        if case["residual"]:
            y += s["residual"].double()
        out = {"out": y}
        if case["train"]:
            dy = s["dout"].double()
            out["dw_down"] = torch.mm(dy.t(), h)
            dh = torch.mm(dy, wd)
            dg, du = dh * u * slope, dh * a
            out["dx"] = torch.addmm(torch.mm(du, wu), dg, wg)
            out["dw_gate"], out["dw_up"] = torch.mm(dg.t(), x), torch.mm(du.t(), x)
        return out
    if case["op"] == "layernorm":
        r = s["x"].double()
        if case["residual"]:
            r = r + s["residual"].double()
        total = r
        r = r.to(DTYPES[case["dtype"]]).double()  # the operator normalises the stored sum
        mean = r.sum(dim=1) / case["H"]
        dev = r - mean.unsqueeze(1)
        rstd = (dev.square().sum(dim=1) / case["H"] + EPS).rsqrt()
        n = dev * rstd.unsqueeze(1)
        w = s["weight"].double().unsqueeze(0)
        y = n * w
        if case["bias"]:
            y = y + s["bias"].double()
        out = {"out": y, "mean": mean, "rstd": rstd, "residual": total if case["residual"] else None}
        if case["train"]:
            dy = s["dout"].double()
            t = dy * w
            along = torch.einsum("nh,nh->n", t, n) / case["H"]
            dx = (t - t.sum(dim=1, keepdim=True) / case["H"] - n * along.unsqueeze(1))
            dx = dx * rstd.unsqueeze(1)
            if case["residual"]:
                dx = dx + s["dresidual"].double()
            out["dx"] = dx
            out["dweight"] = torch.einsum("nh,nh->h", dy, n)
            out["dbias"] = dy.sum(dim=0) if case["bias"] else None
        return out
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t, dtype=torch.float64)) ** 2
                               for t in s["grads"]))
    factor = min(1.0, s["max_norm"] / norm) if norm > 0 else 1.0
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
            "grads": [t.double() * factor for t in s["grads"]]}
