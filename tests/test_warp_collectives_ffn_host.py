"""The gated feed-forward kernels' `.aligned` instructions come right after a warp
barrier (test_warp_collectives_host.py says why), read from the sources."""
import re

import pytest

from test_warp_collectives_host import lines_of


@pytest.mark.parametrize("name", ["gated_ffn.cu", "ffn_split.cu"])
def test_tensor_memory_is_read_and_freed_by_whole_warps(name):
    before = ""
    for i, code in lines_of(name):
        if re.search(r"\btmem_(load32|dealloc(_2cta)?)\(", code):
            assert before == "__syncwarp();", f"{name}:{i}"
        before = code


@pytest.mark.parametrize("name", ["gated_ffn.cu", "ffn_split.cu", "grad_clip.cu"])
def test_cluster_barriers_take_lanes_as_they_come(name):
    assert not [i for i, code in lines_of(name) if "barrier.cluster" in code]
