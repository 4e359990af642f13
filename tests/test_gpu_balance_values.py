"""The balance loss and its gradient on logits far from zero: experts disabled
with a large finite value instead of -inf, and single huge logits."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
STEP = 2.0 ** -24  # half a step of fp32, relative to the value
HALF = {F32: STEP, BF16: 2.0 ** -8}
# e^(x - top): the exponential is off by 2 + 1.16 |x - top| steps, and what is
# further down than e^-20 adds nothing; the sum, the quotient and the division:
# 14 more half steps
P_REL = (2 * 26 + 14) * STEP
FILLS = [-1e9, -1e10, -1e11, -1e15, -1e20, -1e30, -1e38, "lowest", 1e10, 1e11, 1e30]


def value_of(fill, dtype):
    v = torch.finfo(dtype).min if fill == "lowest" else fill
    return float(torch.tensor(v, dtype=dtype))


def normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def check(logits, k, grad=(0.3, -0.02)):
    """Losses and gradient against 64 bits; the row's largest logit is taken
    off first there too (1e30 + ln E is 1e30 even in 64 bits)."""
    N, E = logits.shape
    ids = (torch.arange(N * k, device="cuda", dtype=torch.int32) % E).view(N, k)
    losses, counts, tokens = binding.moe_balance_loss(logits, ids)
    g = torch.tensor(grad, dtype=F32, device="cuda")
    got = binding.moe_balance_loss_backward(logits, counts, tokens, k, g).double()

    lg = logits.double()
    top = lg.amax(1, keepdim=True)
    e = torch.exp(lg - top)
    p = e / e.sum(1, keepdim=True)
    lse = top[:, 0] + torch.log(e.sum(1))
    slots = torch.bincount(ids.reshape(-1).long(), minlength=E)
    assert torch.equal(counts.long(), slots)
    f = slots.double() / (k * N)
    # a lane adds at most 64 rows here, then 5 lanes, 16 warps and 3 joins; the
    # products with the counts and their sum over the experts: 24
    sums = (64 + 5 + 16 + 3 + 24) * STEP
    balance = float(E * (f * p.sum(0)).sum() / N)
    assert abs(float(losses[0]) - balance) <= balance * (P_REL + sums)
    z = float((lse * lse).sum())
    if z > torch.finfo(F32).max * 1.001:
        assert float(losses[1]) == float("inf")  # the sum passes fp32
    else:
        dl = P_REL + 4 * STEP * lse.abs()
        dz = float((2 * lse.abs() * dl + dl * dl).sum()) + z * sums
        assert abs(float(losses[1]) - z / N) <= dz / N

    d = f - 1.0 / E
    g0, g1 = float(g[0]) * E / N, 2 * float(g[1]) / N
    around = (p * d.abs()).sum(1, keepdim=True)
    u = d - (p * d).sum(1, keepdim=True)
    want = p * (g0 * u + g1 * lse[:, None])
    du = (P_REL + 16 * STEP) * around + 4 * STEP * (d.abs() + around)
    dl = (P_REL + 4 * STEP * lse.abs())[:, None]
    tol = (P_REL + 8 * STEP) * want.abs() + p * (abs(g0) * du + abs(g1) * dl)
    tol = tol + 4 * STEP * p * (abs(g0) * u.abs() + abs(g1) * lse.abs()[:, None])
    tol = tol + HALF[logits.dtype] * (want.abs() + tol) + 1e-12 * (abs(g0) + abs(g1))
    assert bool(got.isfinite().all())
    assert bool(((got - want).abs() <= tol).all())
    return losses


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("N,E,k", [(1, 128, 8), (5, 7, 3), (64, 128, 8), (70, 60, 4), (300, 255, 2),
                                   (40, 1, 1)])
def test_rows_of_one_large_value(N, E, k, fill, dtype):
    v = value_of(fill, dtype)
    check(torch.full((N, E), v, dtype=dtype, device="cuda"), k)
    mixed = normal(N + E, N, E).to(dtype)
    mixed[::3] = v  # among ordinary rows
    check(mixed, k)
    check(mixed, k, grad=(0.5, 0.0))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("fill", FILLS)
def test_some_logits_large(fill, dtype):
    """Disabled experts beside ordinary ones, and one huge logit."""
    v = value_of(fill, dtype)
    some = normal(1, 90, 64).to(dtype)
    some[:, 5:40] = v
    some[7, :] = v
    some[8, 63] = 1e10
    some[9, 0] = -1e10
    check(some, 6)


@pytest.mark.parametrize("fill", [-1e10, -1e11, "lowest"])
def test_large_values_in_many_tokens(fill):
    """Several clusters, and the second kernel."""
    lg = normal(2, 40000, 128)
    lg[::17] = value_of(fill, F32)
    check(lg, 8, grad=(0.3, 0.0))


@pytest.mark.parametrize("centre", [0.0, 1e3, 2.0 ** 20, -(2.0 ** 20) - 1, 3e6, -1e7])
def test_logits_around_a_far_centre(centre):
    """Rows that differ by a few around a value far from zero keep their
    probabilities."""
    check(normal(3, 130, 128) * 2 + centre, 4)
