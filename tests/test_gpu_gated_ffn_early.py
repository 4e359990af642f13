"""Weights written right before a call, by a copy or by one of the library's own
kernels (whose dependents may start before it ends): the kernels that read weights
ahead of their wait for the kernel before see what was written."""
import pytest
import torch

from sparse_moe_ffn_gb300 import binding
from test_gpu_gated_ffn import BF16, gen, normal

pytestmark = pytest.mark.gpu


def write(how, src, dst):
    if how == "copy":
        for s, d in zip(src, dst):
            d.copy_(s)
    else:  # a factor of 1: the values as they are
        one = torch.ones(1, device="cuda")
        binding.moe_clip_grads(src, one, 1.0, out=dst)


@pytest.mark.parametrize("how", ["copy", "own kernel"])
@pytest.mark.parametrize("N,H,I", [(1, 512, 4096), (2, 4096, 512), (50, 512, 4096), (128, 2048, 768),
                                   (300, 512, 4096), (512, 1024, 2816), (700, 512, 1024)])
def test_forward_and_backward(N, H, I, how):
    g = gen(N)
    x, dout = normal(g, N, H), normal(g, N, H, std=0.1)
    gate, up = normal(g, N, I), normal(g, N, I)
    sets = [(normal(g, I, H, std=H ** -0.5), normal(g, I, H, std=H ** -0.5),
             normal(g, H, I, std=I ** -0.5)) for _ in range(3)]
    calls = {
        "forward": lambda w, ws: binding.moe_gated_ffn(x, *w, "silu", workspace=ws)[:1],
        "backward": lambda w, ws: binding.moe_gated_ffn_backward(dout, x, *w, gate, up,
                                                                 workspace=ws),
        "dx": lambda w, ws: binding.moe_gated_ffn_backward(dout, x, *w, gate, up, want_dw=False,
                                                           workspace=ws)[:1],
    }
    need = max(binding.moe_gated_ffn_workspace_bytes(N, H, I),
               binding.moe_gated_ffn_backward_workspace_bytes(N, H, I))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for name, call in calls.items():
        want = [call(w, None) for w in sets]
        torch.cuda.synchronize()
        live = [torch.empty_like(t) for t in sets[0]]
        got = []
        for i in range(9):
            write(how, sets[i % 3], live)
            got.append(call(live, ws))
        for i, outs in enumerate(got):
            for a, b in zip(outs, want[i % 3]):
                assert torch.equal(a, b), (name, i)
    assert torch.equal(live[0], sets[2][0])
    assert live[0].dtype is BF16
