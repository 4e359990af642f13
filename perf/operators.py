"""Measured cases of the operators around the sparse FFN layer of a decoder.

  norm      residual add + RMSNorm with an e4m3 output and a scale per token
            (and the bf16 output that the router reads)
  quantize  rows to e4m3 with a scale per row (weights at load, activations
            between two 8-bit products)
  linear    x W^T with scales, bias, activation and residual in the epilogue,
            from bf16 or e4m3 operands, to bf16 or fp32
  balance   per-expert counts, load-balance loss and router z-loss, and (train)
            their gradient with respect to the router logits

Each case is one call a user makes (the training case: forward, then
backward).  ``run`` computes it in plain torch operations, or with the
library's entry points when ``own`` is set; ``exact`` computes it in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100  # the smallest scale: an all-zero row quantises to zeros
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu")
EPS = 1e-6


# ------------------------------------------------------------------ the cases

def _norm(name, N, H, gemma=False, normed=True, residual=True):
    return dict(name=name, op="norm", N=N, H=H, gemma=gemma, normed=normed, residual=residual)


def _quantize(name, N, H):
    return dict(name=name, op="quantize", N=N, H=H)


def _linear(name, N, K, O, kind, act="none", bias=True, residual=False, out="bf16"):
    return dict(name=name, op="linear", N=N, K=K, O=O, kind=kind, act=act, bias=bias,
                residual=residual, out=out)


def _balance(name, N, E, k, train, dtype="fp32", masked=False):
    return dict(name=name, op="balance", N=N, E=E, k=k, train=train, dtype=dtype, masked=masked)


def listed():
    return [
        # one new token of one sequence enters the layer: latency
        _norm("norm one token", 1, 2048),
        # a prefill batch enters the layer: bandwidth
        _norm("norm prefill", 8192, 2048),
        # the weights of a projection converted at load
        _quantize("quantize weights", 8192, 2048),
        # a ragged batch of activations between two 8-bit products
        _quantize("quantize ragged", 1021, 4104),
        # router logits of a decode batch, kept in fp32
        _linear("linear router decode", 64, 2048, 128, "bf16", bias=False, out="fp32"),
        # one token through an 8-bit projection: weight streaming
        _linear("linear e4m3 one token", 1, 2048, 8192, "e4m3", act="silu"),
        # a mid-sized ragged batch through a bf16 projection onto the residual
        _linear("linear bf16 ragged", 333, 1000, 1111, "bf16", act="gelu", residual=True),
        # the up projection of a prefill batch in 8 bits
        _linear("linear e4m3 prefill", 8192, 2048, 8192, "e4m3", act="silu"),
        # the down projection of a prefill batch in bf16, added to the residual
        _linear("linear bf16 prefill", 8192, 8192, 2048, "bf16", residual=True),
        # load statistics of one decode step
        _balance("balance decode", 64, 128, 8, False),
        # a training step: losses, counts and the gradient of the logits
        _balance("balance train", 131072, 128, 8, True),
        # packed sequences with padding tokens, dropped slots, disabled experts
        _balance("balance train ragged", 4099, 60, 4, True, "bf16", True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log_mult(rng, lo, hi, m):
    return max(m, _log_int(rng, lo, hi) // m * m)


MAX_FLOPS = 2.0 * 8192 * 2048 * 8192
MAX_ELEMENTS = 8192 * 2048


def draw(rng):
    op = rng.choice(("norm", "quantize", "linear", "linear", "linear", "balance", "balance"))
    if op in ("norm", "quantize"):
        while True:
            N, H = _log_int(rng, 1, 16384), _log_mult(rng, 64, 8192, 8)
            if N * H <= MAX_ELEMENTS:
                break
        if op == "quantize":
            c = _quantize("", N, H)
        else:
            c = _norm("", N, H, rng.random() < 0.3, rng.random() < 0.5, rng.random() < 0.8)
    elif op == "linear":
        kind = rng.choice(("bf16", "e4m3"))
        while True:
            N = _log_int(rng, 1, 16384)
            K = _log_mult(rng, 64, 8192, 16 if kind == "e4m3" else 8)
            O = _log_int(rng, 6, 8192)
            if rng.random() < 0.5:
                O = max(8, O // 8 * 8)
            if 2.0 * N * K * O <= MAX_FLOPS:
                break
        c = _linear("", N, K, O, kind, rng.choice(ACTS), rng.random() < 0.7, rng.random() < 0.5,
                    "fp32" if rng.random() < 0.25 else "bf16")
    else:
        while True:
            N, E = _log_int(rng, 1, 262144), _log_int(rng, 4, 256)
            if N * E <= 131072 * 128:
                break
        c = _balance("", N, E, rng.randint(1, min(E, 10)), rng.random() < 0.6,
                     rng.choice(("fp32", "bf16")), rng.random() < 0.4)
    del c["name"]
    return c


# ------------------------------------------------------------------- the inputs

def _rows_e4m3(t):
    """(e4m3 rows, fp32 scale per row) of a 2-D tensor, as loaded weights come."""
    s = (t.float().abs().amax(1) / E4M3_MAX).clamp(min=SCALE_MIN)
    return (t.float() / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(F8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=F32) * std

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda", dtype=F32)

    s = {"case": c}
    if c["op"] == "norm":
        N, H = c["N"], c["H"]
        # a residual stream: larger than one layer's output, with a few
        # channels far above the others
        spread = 1.0 + 20.0 * (uniform(H) < 0.005).float()
        s["x"] = normal(N, H).to(BF16)
        s["residual"] = (normal(N, H, std=4.0) * spread).to(BF16) if c["residual"] else None
        s["weight"] = (normal(H, std=0.1) + (0.0 if c["gemma"] else 1.0)).to(BF16)
        s["residual_out"] = torch.empty((N, H), dtype=BF16, device="cuda")
        s["q"] = torch.empty((N, H), dtype=F8, device="cuda")
        s["scale"] = torch.empty(N, dtype=F32, device="cuda")
        s["normed"] = torch.empty((N, H), dtype=BF16, device="cuda") if c["normed"] else None
    elif c["op"] == "quantize":
        N, H = c["N"], c["H"]
        s["x"] = normal(N, H, std=0.02).to(BF16)
        s["q"] = torch.empty((N, H), dtype=F8, device="cuda")
        s["scale"] = torch.empty(N, dtype=F32, device="cuda")
    elif c["op"] == "linear":
        N, K, O = c["N"], c["K"], c["O"]
        x, w = normal(N, K).to(BF16), normal(O, K, std=0.02).to(BF16)
        if c["kind"] == "e4m3":
            s["x"], s["x_scale"] = _rows_e4m3(x)
            s["w"], s["w_scale"] = _rows_e4m3(w)
        else:
            s["x"], s["w"], s["x_scale"], s["w_scale"] = x, w, None, None
        s["bias"] = normal(O, std=0.1).to(BF16) if c["bias"] else None
        s["residual"] = normal(N, O).to(BF16) if c["residual"] else None
        dtype = F32 if c["out"] == "fp32" else BF16
        s["out"] = torch.empty((N, O), dtype=dtype, device="cuda")
        s["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
    else:
        N, E, k = c["N"], c["E"], c["k"]
        # router logits: one unit of spread a token, a bias an expert
        logits = normal(N, E) + normal(E, std=0.3)
        mask = None
        if c["masked"]:
            off = uniform(E) < 0.05  # disabled experts
            off[0] = False
            logits = logits.masked_fill(off[None, :], float("-inf"))
            mask = uniform(N) >= 0.1  # padding tokens take no part
        ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        if c["masked"]:
            ids = ids.masked_fill(uniform(N, k) < 0.02, -1)  # dropped slots
            # tokens with no expert left
            logits = logits.masked_fill((uniform(N) < 0.002)[:, None], float("-inf"))
        s["logits"] = logits.to(F32 if c["dtype"] == "fp32" else BF16).contiguous()
        s["ids"], s["mask"] = ids.contiguous(), mask
        s["grad"] = torch.tensor([0.01, 0.001], dtype=F32, device="cuda")  # the losses' weights
        s["losses"] = torch.empty(2, dtype=F32, device="cuda")
        s["counts"] = torch.empty(E, dtype=torch.int32, device="cuda")
        s["tokens"] = torch.empty(1, dtype=torch.int32, device="cuda")
        s["dlogits"] = torch.empty_like(s["logits"]) if c["train"] else None
    return s


# --------------------------------------------------------------- the plain form

def _act(v, act):
    if act == "silu":
        return v / (1.0 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if act == "relu":
        return torch.clamp(v, min=0.0)
    return v


def _plain_e4m3(y):
    scale = (y.abs().amax(1) / E4M3_MAX).clamp(min=SCALE_MIN)
    return (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(F8), scale


def _plain_norm(s):
    c = s["case"]
    r = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(BF16)
    rf = r.float()
    w = s["weight"].float() + (1.0 if c["gemma"] else 0.0)
    y = rf * torch.rsqrt((rf * rf).mean(1, keepdim=True) + EPS) * w
    q, scale = _plain_e4m3(y)
    return {"residual": r, "q": q, "scale": scale,
            "normed": y.to(BF16) if c["normed"] else None}


def _plain_linear(s):
    c = s["case"]
    acc = s["x"].float() @ s["w"].float().T
    if s["x_scale"] is not None:
        acc = acc * s["x_scale"][:, None] * s["w_scale"][None, :]
    if s["bias"] is not None:
        acc = acc + s["bias"].float()
    acc = _act(acc, c["act"])
    if s["residual"] is not None:
        acc = acc + s["residual"].float()
    return acc.to(s["out"].dtype)


def _plain_balance(s):
    c = s["case"]
    N, E, k = c["N"], c["E"], c["k"]
    lg = s["logits"].float()
    m = s["mask"] if s["mask"] is not None else torch.ones(N, dtype=torch.bool, device=lg.device)
    top = lg.amax(1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    e = torch.exp(lg - top)
    total = e.sum(1, keepdim=True)
    some = total > 0
    p = torch.where(some, e / total, torch.zeros_like(e)) * m[:, None]
    lse = torch.where(some, top + torch.log(total), torch.zeros_like(top)) * m[:, None]
    ids = s["ids"].long()
    ids = torch.where((ids >= 0) & (ids < E) & m[:, None], ids, torch.full_like(ids, E))
    counts = torch.zeros(E + 1, dtype=torch.int64, device=lg.device)
    counts = counts.scatter_add_(0, ids.reshape(-1), torch.ones_like(ids).reshape(-1))[:E]
    T = m.sum()
    inv = 1.0 / T.double().clamp(min=1)  # the sums over tokens are long: 64 bits
    f = counts.double() * inv / k
    losses = torch.stack([E * (f * p.sum(0, dtype=torch.float64) * inv).sum(),
                          (lse.double() ** 2).sum() * inv]).float()
    out = {"losses": losses, "counts": counts.int(), "tokens": T.int().reshape(1)}
    if c["train"]:
        # sum_e p_e = 1: the mean share 1/E is taken off f, which leaves the
        # difference from the weighted mean as it is, without its cancellation
        d = (f - 1.0 / E).float()
        u = d - (p * d).sum(1, keepdim=True)
        inv = inv.float()
        out["dlogits"] = (p * inv * (s["grad"][0] * E * u + 2.0 * s["grad"][1] * lse)).to(
            s["logits"].dtype)
    return out


# --------------------------------------------------------------- the library's

def _own_norm(s):
    from sparse_moe_ffn_gb300 import binding as b
    c = s["case"]
    q, scale, normed = b.moe_add_rmsnorm_fp8(
        s["x"], s["residual"], s["weight"], eps=EPS, gemma=c["gemma"], q=s["q"],
        scale=s["scale"], normed=s["normed"], residual_out=s["residual_out"])
    return {"residual": s["residual_out"], "q": q, "scale": scale, "normed": normed}


def _own_linear(s):
    from sparse_moe_ffn_gb300 import binding as b
    return b.moe_linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"],
                        activation=s["case"]["act"], x_scale=s["x_scale"],
                        w_scale=s["w_scale"], out=s["out"], workspace=s["workspace"])


def _own_balance(s):
    from sparse_moe_ffn_gb300 import binding as b
    c = s["case"]
    losses, counts, tokens = b.moe_balance_loss(s["logits"], s["ids"], mask=s["mask"],
                                                losses=s["losses"], counts=s["counts"],
                                                tokens=s["tokens"])
    out = {"losses": losses, "counts": counts, "tokens": tokens}
    if c["train"]:
        out["dlogits"] = b.moe_balance_loss_backward(s["logits"], counts, tokens, c["k"],
                                                     s["grad"], mask=s["mask"],
                                                     dlogits=s["dlogits"])
    return out


def run(state):
    op = state["case"]["op"]
    if not own:
        if op == "norm":
            return _plain_norm(state)
        if op == "quantize":
            q, scale = _plain_e4m3(state["x"].float())
            return {"q": q, "scale": scale}
        return _plain_linear(state) if op == "linear" else _plain_balance(state)
    if op == "norm":
        return _own_norm(state)
    if op == "quantize":
        from sparse_moe_ffn_gb300 import binding as b
        q, scale = b.moe_quantize_fp8(state["x"], q=state["q"], scale=state["scale"])
        return {"q": q, "scale": scale}
    return _own_linear(state) if op == "linear" else _own_balance(state)


# ------------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] in ("norm", "quantize"):
        N, H = c["N"], c["H"]
        if c["op"] == "quantize":
            return {"bytes": N * H * 3 + 4 * N, "flops": 3 * N * H}
        # x read, the sum and the e4m3 written; residual read; bf16 written
        per = 2 + 2 + 1 + (2 if c["residual"] else 0) + (2 if c["normed"] else 0)
        return {"bytes": N * H * per + 4 * N + 2 * H, "flops": 8 * N * H}
    if c["op"] == "linear":
        N, K, O = c["N"], c["K"], c["O"]
        b = (N * K + O * K) * (1 if c["kind"] == "e4m3" else 2)
        b += 4 * (N + O) if c["kind"] == "e4m3" else 0
        b += N * O * ((4 if c["out"] == "fp32" else 2) + (2 if c["residual"] else 0))
        b += 2 * O if c["bias"] else 0
        return {"bytes": b, "flops": 2 * N * K * O}
    N, E, k = c["N"], c["E"], c["k"]
    size = 4 if c["dtype"] == "fp32" else 2
    b = N * E * size + 4 * N * k + 4 * E + (N if c["masked"] else 0)
    return {"bytes": b + (N * E * size if c["train"] else 0),
            "flops": N * E * (12 if c["train"] else 6)}


# ----------------------------------------------------------------------- exact

def exact(case, seed):
    """The case's outputs from the definitions, in 64 bits (8-bit values before
    their rounding to e4m3)."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double()
        scale = torch.maximum(x.abs().max(dim=1).values / E4M3_MAX,
                              torch.tensor(SCALE_MIN, dtype=torch.float64, device=x.device))
        return {"q": x / scale.unsqueeze(1), "scale": scale}
    if op == "norm":
        total = s["x"].double()
        if case["residual"]:
            total = total + s["residual"].double()
        r = total.to(BF16).double()  # the operator normalises the stored residual
        rms = (r.pow(2).sum(dim=1) / case["H"] + EPS).sqrt()
        gain = s["weight"].double()
        if case["gemma"]:
            gain = gain + 1
        y = r / rms.unsqueeze(1) * gain
        scale = torch.maximum(y.abs().max(dim=1).values / E4M3_MAX,
                              torch.tensor(SCALE_MIN, dtype=torch.float64, device=y.device))
        return {"residual": total, "q": y / scale.unsqueeze(1), "scale": scale,
                "normed": y if case["normed"] else None}
    if op == "linear":
        x, w = s["x"].double(), s["w"].double()
        if case["kind"] == "e4m3":
            x = x * s["x_scale"].double().unsqueeze(1)
            w = w * s["w_scale"].double().unsqueeze(1)
        y = torch.mm(x, w.t())
        if case["bias"]:
            y += s["bias"].double()
        if case["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif case["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif case["act"] == "gelu_tanh":
            # (1 + tanh(z)) / 2 is the logistic function of 2 z
            y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y.pow(3)))
        elif case["act"] == "relu":
            y = torch.where(y > 0, y, torch.zeros_like(y))
        if case["residual"]:
            y += s["residual"].double()
        return y
    # balance: only the tokens that take part, in their own order
    N, E, k = case["N"], case["E"], case["k"]
    lg = s["logits"].double()
    rows = torch.arange(N, device=lg.device) if s["mask"] is None else s["mask"].nonzero()[:, 0]
    T = rows.numel()
    part = lg[rows]
    lse = torch.logsumexp(part, dim=1)
    lse = lse.masked_fill(torch.isinf(lse), 0.0)
    p = torch.exp(part - lse.unsqueeze(1))
    ids = s["ids"][rows].reshape(-1).long()
    counts = torch.bincount(ids[ids >= 0], minlength=E)
    f = counts.double() / max(k * T, 1)
    out = {"losses": torch.stack([E * torch.dot(f, p.sum(dim=0) / max(T, 1)),
                                  lse.square().sum() / max(T, 1)]),
           "counts": None, "tokens": None}
    if case["train"]:
        a, z = 0.01, 0.001
        a, z = (float(v) for v in torch.tensor([a, z], dtype=F32))
        d = torch.zeros_like(lg)
        d[rows] = p * (a * E / max(T, 1) * (f.unsqueeze(0) - torch.mv(p, f).unsqueeze(1))
                       + 2.0 * z / max(T, 1) * lse.unsqueeze(1))
        out["dlogits"] = d
    return out
