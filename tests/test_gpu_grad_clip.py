"""The norm of a set of tensors and its clipping on the GPU against 64 bits.

Tolerances count roundings: fp32 squares of at most 32 values (33 roundings, and
2^-60 for what underflow takes), sums in 64 bits, one rounding of the norm, half
the relative error by the root; factor: a division, a product, the output's."""
import math

import pytest
import torch

from sparse_moe_ffn_gb300 import binding

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
NORM_REL = 33 / 2 * 2.0 ** -24 + 2.0 ** -23


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def tensors(g, sizes, dtypes, std=1.0):
    return [(torch.randn(n, generator=g, device="cuda") * std).to(t) for n, t in zip(sizes, dtypes)]


def norm64(ts):
    return math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in ts))


def check(grads, max_norm, out_dtypes=None, offset=0):
    ref = norm64(grads)
    norm = binding.moe_grad_norm(grads)
    assert norm.shape == (1,) and norm.dtype is F32
    assert abs(float(norm) - ref) <= NORM_REL * ref
    keep = [t.clone() for t in grads]
    out, flats = None, []
    if out_dtypes is not None:
        out = []
        for t, d in zip(grads, out_dtypes):
            flat = torch.full((t.numel() + 64 + offset,), float("nan"), dtype=d, device="cuda")
            flats.append(flat)
            out.append(flat[32 + offset:32 + offset + t.numel()].view(t.shape))
    got = binding.moe_clip_grads(grads, norm, max_norm, out=out)
    factor = 1.0 if float(norm) <= max_norm else max_norm / float(norm)
    for i, (k, o) in enumerate(zip(keep, got)):
        v = k.double() * factor
        tol = (HALF[o.dtype] + (0 if factor == 1.0 else 3 * 2.0 ** -24)) * v.abs() + 1e-40
        assert bool(((o.double() - v).abs() <= tol).all()), i
        if out is not None:
            assert torch.equal(grads[i], k)
            n = k.numel()
            assert bool(flats[i][:32 + offset].isnan().all())
            assert bool(flats[i][32 + offset + n:].isnan().all())
        else:
            assert o is grads[i]


SETS = {
    "one value": ([1], [F32]),
    "one small": ([7], [BF16]),
    "one chunk": ([8192], [BF16]),
    "a chunk and one": ([8193], [F32]),
    "odd": ([1, 3, 8191, 8200, 33, 65537], [BF16, F32, BF16, F32, BF16, BF16]),
    "with empty ones": ([0, 5, 0, 0, 9000, 0], [F32, BF16, BF16, F32, F32, BF16]),
    "many": ([1 + 37 * i % 5000 for i in range(64)], [BF16, F32] * 32),
    "more": ([1 + 37 * i % 5000 for i in range(300)], [BF16, F32, F32] * 100),
    "tables": ([1 + 91 * i % 700 for i in range(1500)], [BF16, BF16, F32] * 500),
    "large": ([20_000_003, 5, 4_000_000], [BF16, F32, F32]),
}


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("form", ["in place", "same", "fp32", "bf16"])
def test_sets(name, form):
    sizes, dtypes = SETS[name]
    grads = tensors(gen(len(sizes)), sizes, dtypes)
    out = {"in place": None, "same": dtypes, "fp32": [F32] * len(sizes),
           "bf16": [BF16] * len(sizes)}[form]
    check(grads, 0.25 * math.sqrt(sum(sizes)), out)


@pytest.mark.parametrize("name", ["odd", "many"])
@pytest.mark.parametrize("out", [None, "same"])
def test_below_the_limit(name, out):
    sizes, dtypes = SETS[name]
    grads = tensors(gen(1), sizes, dtypes)
    check(grads, 1e6, None if out is None else dtypes)


@pytest.mark.parametrize("offset", [1, 2, 5])
def test_tensors_that_start_anywhere(offset):
    g = gen(offset)
    grads = [t[offset:] for t in tensors(g, [9000, 70001, 40], [BF16, F32, BF16])]
    check(grads, 10.0, [F32, BF16, BF16], offset=offset)
    check(grads, 10.0)


@pytest.mark.parametrize("shape", [(3, 5, 7), (64, 128), (2, 2048, 16)])
def test_shapes(shape):
    g = gen(3)
    t = torch.randn(shape, generator=g, device="cuda")
    norm = binding.moe_grad_norm([t])
    out = binding.moe_clip_grads([t], norm, 1.0, out=[torch.empty(t.numel(), device="cuda")])
    assert out[0].dim() == 1 and torch.allclose(out[0], t.reshape(-1) / norm, rtol=1e-6)


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-25, 1e-19, 1e18, 1e25, 3e36])
@pytest.mark.parametrize("n", [5, 100_000])
def test_values_whose_squares_leave_fp32(scale, n):
    """fp32 squares of these overflow or vanish; their sum does not."""
    t = (torch.rand(n, generator=gen(n), device="cuda") + 0.5) * scale
    # subnormal values: torch's product may round on their grid; the reference
    # is of what is stored
    ref = norm64([t])
    got = float(binding.moe_grad_norm([t]))
    if ref > torch.finfo(F32).max:  # 100000 values of 3e36 have norm 9.9e38: no fp32 value
        assert got == math.inf
        return
    assert abs(got - ref) <= NORM_REL * ref + 2.0 ** -149
    mixed = [t, torch.zeros(1000, device="cuda"), torch.ones(3, device="cuda")]
    ref = norm64(mixed)
    assert abs(float(binding.moe_grad_norm(mixed)) - ref) <= NORM_REL * ref


def test_zeros_nan_and_infinities():
    z = [torch.zeros(10_000, device="cuda"), torch.zeros(5, dtype=BF16, device="cuda")]
    norm = binding.moe_grad_norm(z)
    assert float(norm) == 0.0
    binding.moe_clip_grads(z, norm, 0.0)
    assert not any(bool(t.any()) for t in z)
    ones = torch.ones(10_000, device="cuda")
    for bad in (float("nan"), float("inf"), -float("inf")):
        t = ones.clone()
        t[777] = bad
        norm = binding.moe_grad_norm([ones, t])
        assert math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf
        out = binding.moe_clip_grads([ones, t], norm, 1.0, out=[torch.empty_like(t) for _ in "ab"])
        if math.isnan(bad):
            assert bool(out[0].isnan().all())
        else:
            assert bool((out[0] == 0).all()) and bool(out[1][777].isnan())
    binding.moe_clip_grads([ones], torch.full((1,), 5.0, device="cuda"), 0.0)
    assert not bool(ones.any())


def test_no_tensors_and_empty_ones():
    e = [torch.empty(0, device="cuda"), torch.empty(0, dtype=BF16, device="cuda")]
    norm = binding.moe_grad_norm(e)
    assert float(norm) == 0.0
    assert binding.moe_clip_grads(e, norm, 1.0)[0] is e[0]
    assert binding.moe_clip_grads([], norm, 1.0) == []


def test_handle_keeps_the_tensors_and_sees_their_values():
    grads = tensors(gen(0), [3000, 17], [BF16, F32])
    kept = binding.GradSet(grads)
    for scale in (1.0, 3.0):
        for t in grads:
            t.mul_(scale)
        ref = norm64(grads)
        assert abs(float(binding.moe_grad_norm(kept)) - ref) <= NORM_REL * ref


def test_same_bits_streams_and_graphs():
    g = gen(4)
    grads = tensors(g, [3_000_001, 77, 500_000], [BF16, F32, F32])
    kept = binding.GradSet(grads, [torch.empty_like(t) for t in grads])
    norm, ws = torch.empty(1, device="cuda"), torch.empty(
        binding.moe_grad_norm_workspace_bytes(3), dtype=torch.uint8, device="cuda")

    def both():
        binding.moe_grad_norm(kept, norm=norm, workspace=ws)
        return binding.moe_clip_grads(kept, norm, 5.0)

    first = [t.clone() for t in both()]
    n0 = norm.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for t in kept.out:
        t.zero_()
    norm.zero_()
    graph.replay()
    assert torch.equal(norm, n0)
    for a, b in zip(first, kept.out):
        assert torch.equal(a, b)
    grads[0].mul_(2.0)  # the graph reads the tensors, not what they held
    graph.replay()
    ref = norm64(grads)
    assert abs(float(norm) - ref) <= NORM_REL * ref
