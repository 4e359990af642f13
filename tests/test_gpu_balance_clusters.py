"""The balance loss on a device without room for clusters of 16 blocks: one
cluster of 8 takes the same batches in more passes."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24  # half a step of fp32, relative to the value


@pytest.fixture
def portable_only():
    binding.lib().moe_selftest_portable_clusters(1)
    yield
    binding.lib().moe_selftest_portable_clusters(0)


# from just past one pass of 8 blocks to the largest batch of one cluster
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,E,k", [(1025, 128, 8), (6144, 128, 8), (4099, 60, 4), (3072, 255, 3),
                                   (98304, 8, 2), (98301, 7, 3)])
def test_one_cluster_of_8(portable_only, N, E, k, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    logits = (torch.randn(N, E, generator=g, device="cuda") * 1.5).to(dtype)
    ids = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
    mask = torch.rand(N, generator=g, device="cuda") > 0.2
    assert binding.lib().moe_balance_loss_workspace_bytes(N, E) == 256  # one cluster
    before = binding.lib().moe_kernel_launch_count()
    losses, counts, tokens = binding.moe_balance_loss(logits, ids, mask)
    assert binding.lib().moe_kernel_launch_count() == before + 1
    slots = torch.bincount(ids[mask].reshape(-1).long(), minlength=E)
    T = int(mask.sum())
    assert torch.equal(counts.long(), slots) and int(tokens) == T
    lg = logits[mask].double()
    lse = torch.logsumexp(lg, 1)
    balance = float(E * (slots.double() / (k * T) * torch.softmax(lg, 1).sum(0)).sum() / T)
    z = float(lse.square().sum())
    # a lane adds at most 64 rows, then 5 lanes, 16 warps and 3 joins; the
    # products with the counts and their sum over the experts: 24; exponentials
    # within e^-20 of the largest: 2 * 26 half steps, and 14
    sums, p_rel = (64 + 5 + 16 + 3 + 24) * STEP, (2 * 26 + 14) * STEP
    assert abs(float(losses[0]) - balance) <= balance * (p_rel + sums)
    dz = float((2 * lse.abs() * (p_rel + 4 * STEP * lse.abs())).sum()) * 1.001 + z * sums
    assert abs(float(losses[1]) - z / T) <= dz / T


def test_the_wider_cluster_returns():
    """Afterwards calls take the cluster that they took before."""
    logits = torch.randn(4000, 128, device="cuda")
    ids = torch.topk(logits, 8, dim=1).indices.to(torch.int32)
    first = binding.moe_balance_loss(logits, ids)
    binding.lib().moe_selftest_portable_clusters(1)
    other = binding.moe_balance_loss(logits, ids)
    binding.lib().moe_selftest_portable_clusters(0)
    again = binding.moe_balance_loss(logits, ids)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert torch.equal(first[1], other[1]) and torch.equal(first[2], other[2])
