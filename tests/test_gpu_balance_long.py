"""The balance losses over millions of tokens: the error of a sum does not grow
with their number."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24  # half a step of fp32, relative to the value
N, E, k = (1 << 22) + 77, 254, 2


@pytest.mark.parametrize("rows", ["same", "random"])
def test_losses_of_many_tokens(rows):
    """Rows that are all alike round the same way at every addition: summed one
    after the other in fp32, the 2048 rows of a lane come out 2.9e-5 too far
    (with p = 1/254 and lse = log 254)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    logits = torch.zeros((N, E), dtype=torch.bfloat16, device="cuda")
    chunks = [slice(i, min(i + (1 << 18), N)) for i in range(0, N, 1 << 18)]
    if rows == "random":
        for c in chunks:
            logits[c] = torch.randn(logits[c].shape, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, E, (N, k), generator=g, device="cuda", dtype=torch.int32)
    ids[::3] = 11  # an uneven load
    losses, counts, tokens = binding.moe_balance_loss(logits, ids)
    p, z = torch.zeros(E, dtype=torch.float64, device="cuda"), 0.0
    for c in chunks:
        lg = logits[c].double()
        p += torch.softmax(lg, 1).sum(0)
        z += float(torch.logsumexp(lg, 1).square().sum())
    slots = torch.bincount(ids.reshape(-1).long(), minlength=E)
    assert torch.equal(counts.long(), slots) and int(tokens) == N
    want = float(E * (slots.double() / (k * N) * p).sum() / N), z / N
    # a lane adds at most 64 rows on their own, then 5 lanes, 8 warps and 3 joins;
    # the products with the counts and their sum over the experts: 24
    sums = (64 + 5 + 8 + 3 + 24) * STEP
    # equal logits: the exponentials are 1, then a quotient; else the
    # exponentials' steps within e^-20 of the largest
    p_rel = (4 if rows == "same" else 2 * 26 + 14) * STEP
    lse = want[1] ** 0.5
    d = p_rel + 4 * STEP * lse
    assert abs(float(losses[0]) - want[0]) <= want[0] * (p_rel + sums)
    assert abs(float(losses[1]) - want[1]) <= 2 * 1.01 * lse * d + want[1] * sums


# more than 16 passes, with rows of 1, 8, 16 and 32 lanes
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,E,k", [(4300001, 7, 2), (600003, 60, 4), (300001, 128, 8),
                                   (200003, 256, 8)])
def test_long_batches_of_every_width(N, E, k, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(E)
    logits = torch.randn((N, E), generator=g, device="cuda").to(dtype)
    ids = torch.randint(0, E, (N, k), generator=g, device="cuda", dtype=torch.int32)
    mask = torch.rand(N, generator=g, device="cuda") > 0.25
    logits[~mask] = float("nan")
    losses, counts, tokens = binding.moe_balance_loss(logits, ids, mask)
    p, z, T = torch.zeros(E, dtype=torch.float64, device="cuda"), 0.0, int(mask.sum())
    for i in range(0, N, 1 << 20):
        lg = logits[i:i + (1 << 20)][mask[i:i + (1 << 20)]].double()
        p += torch.softmax(lg, 1).sum(0)
        z += float(torch.logsumexp(lg, 1).square().sum())
    slots = torch.bincount(ids[mask].reshape(-1).long(), minlength=E)
    assert torch.equal(counts.long(), slots) and int(tokens) == T
    want = float(E * (slots.double() / (k * T) * p).sum() / T), z / T
    # as above; each row's lse, at most log E + 6 here, is off by d
    sums, p_rel = (64 + 5 + 8 + 3 + 24) * STEP, (2 * 26 + 14) * STEP
    d = p_rel + 4 * STEP * 12
    assert abs(float(losses[0]) - want[0]) <= want[0] * (p_rel + sums)
    assert abs(float(losses[1]) - want[1]) <= 2 * want[1] ** 0.5 * d + d * d + want[1] * sums
