"""Instructions that a whole warp has to execute together (`.aligned`) come
right after a warp barrier in the kernels whose lanes branch on their own: a
`.aligned` instruction that lanes reach apart is undefined, and whether they do
is up to the compiler.  Read from the sources, as no run can show it."""
import os
import re

import pytest

from sparse_moe_ffn_gb300.build import CSRC

KERNELS = ["linear_split.cu", "linear_pair.cu", "balance.cu"]


def lines_of(name):
    """(number, code) of the lines that hold code, without comments."""
    with open(os.path.join(CSRC, name)) as f:
        for i, line in enumerate(f, 1):
            code = re.sub(r"//.*", "", line).strip()
            if code:
                yield i, code


@pytest.mark.parametrize("name", KERNELS)
def test_cluster_barriers_take_lanes_as_they_come(name):
    assert not [i for i, code in lines_of(name) if "barrier.cluster" in code]
    header = [code for _, code in lines_of("cluster.cuh") if "barrier.cluster" in code]
    assert header and not [code for code in header if ".aligned" in code]


@pytest.mark.parametrize("name", KERNELS)
def test_tensor_memory_is_read_and_freed_by_whole_warps(name):
    before = ""
    for i, code in lines_of(name):
        if re.search(r"\btmem_(load32|dealloc(_2cta)?)\(", code):
            assert before == "__syncwarp();", f"{name}:{i}"
        before = code
