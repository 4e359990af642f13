"""dweight and dbias over many rows: the roundings of their sums stay few however
many rows there are.

The statistics are given as mean 0 and 1/std 1 with x = 1, so that dweight and dbias
are both the sum of dout; dout is 1 + 2^-13 - 2^-23 everywhere, of which a single
fp32 sum loses the part behind the 1 once it is past 2048: 4096 rows come out 2^-14
of their sum too small.  In runs of 128 rows a sum takes 128 roundings; then, by
kernel, the runs of a part (64 of up to 8192 rows) or a block's rows (8), eight
parts by each other in fp32, and the result's one.  A rounding is off by at most
2^-24 of the magnitudes' sum, which is the sum itself here.
"""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding

pytestmark = pytest.mark.gpu

F32 = torch.float32
C = 1 + 2.0 ** -13 - 2.0 ** -23
TOL = (128 + 64 + 8 + 8 + 1) * 2.0 ** -24


def sums(N, H, shift=0):
    def full(v, *shape):
        flat = torch.full((shift + torch.Size(shape).numel(),), v, device="cuda")
        return flat[shift:].view(shape)

    x, dy = full(1.0, N, H), full(C, N, H)
    w, mean, rstd = full(1.0, H), torch.zeros(N, device="cuda"), torch.ones(N, device="cuda")
    _, dw, db = binding.moe_layernorm_backward(dy, x, w, mean, rstd, want_dx=False)
    for got in (dw, db):
        assert float((got.double() / (N * C) - 1).abs().max()) <= TOL


@pytest.mark.parametrize("N,H,shift", [(10_000_001, 8, 0), (10_000_001, 7, 0), (1_300_001, 100, 0),
                                       (200_003, 1000, 1), (700_001, 1024, 0), (160_001, 4096, 0),
                                       (80_003, 4001, 0)])
def test_sums_in_registers(N, H, shift):
    sums(N, H, shift)


@pytest.mark.parametrize("N,H,shift", [(8192, 65535, 0), (8001, 65536, 1), (16384, 65536, 0),
                                       (16003, 40001, 0)])
def test_sums_of_their_own_pass(N, H, shift):
    sums(N, H, shift)


@pytest.mark.parametrize("N,H", [(130, 16), (40_003, 64), (400_000, 64), (90_001, 4000),
                                 (3000, 4104)])
def test_every_row_counts_once(N, H):
    """Whole numbers: exact in fp32 whatever the order."""
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    dy = torch.randint(-2, 3, (N, H), generator=g, device="cuda").to(F32)
    x = torch.randint(-2, 3, (N, H), generator=g, device="cuda").to(F32)
    w, mean, rstd = torch.ones(H, device="cuda"), torch.zeros(N, device="cuda"), torch.ones(
        N, device="cuda")
    for dtype in (F32, torch.bfloat16):
        _, dw, db = binding.moe_layernorm_backward(dy.to(dtype), x.to(dtype), w.to(dtype), mean, rstd,
                                                   want_dx=False)
        assert torch.equal(dw.double(), (dy.double() * x.double()).sum(0))
        assert torch.equal(db.double(), dy.double().sum(0))
