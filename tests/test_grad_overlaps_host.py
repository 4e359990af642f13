"""moe_clip_grads and moe_grad_norm refuse tensors that lie in one another, on the
host.  Every call here is refused, for its overlap or, where there is none, for
the negative max_norm that is looked at afterwards."""
import ctypes
import random

import pytest

from sparse_moe_ffn_gb300 import binding
from sparse_moe_ffn_gb300 import build as lib_build

INVALID = 1
P = 1 << 20
NORM = 1 << 40


@pytest.fixture(scope="module")
def L():
    lib_build.build()
    return binding.lib()


def clip(L, grads, out, norm=NORM):
    """grads, out: (address, values, bf16) each; whether an overlap is refused."""
    n = len(grads)
    src = (ctypes.c_void_p * n)(*(g[0] for g in grads))
    dst = (ctypes.c_void_p * n)(*(o[0] for o in out))
    sizes = (ctypes.c_int64 * n)(*(g[1] for g in grads))
    status = L.moe_clip_grads(src, sizes, bytes(g[2] for g in grads), n, norm, -1.0, dst,
                              bytes(o[2] for o in out), None)
    assert status == INVALID
    message = L.moe_last_error()
    assert (b"overlap" in message) != (message.startswith(b"max_norm"))
    return b"overlap" in message


def test_overlaps_of_two_tensors(L):
    a, b = (P, 100, 0), (P + 400, 100, 1)  # b right behind a
    far = [(2 * P, 100, 0), (3 * P, 100, 1)]
    assert not clip(L, [a, b], [a, b])
    assert not clip(L, [a, b], far)
    assert not clip(L, [b, a], [far[1], far[0]])
    assert not clip(L, [a, a], [far[0], (3 * P, 100, 0)])  # read twice
    assert not clip(L, [a, (P + 200, 50, 0)], far)          # read in one another
    assert not clip(L, [a, (0, 0, 0)], [a, (P, 0, 1)])      # an empty one
    assert clip(L, [a, a], [a, a])                          # written twice
    assert clip(L, [a, (P + 396, 100, 0)], [a, (P + 396, 100, 0)])
    assert clip(L, [a, b], [far[0], (2 * P + 200, 100, 1)])
    assert clip(L, [a, b], [(P + 4, 100, 0), far[1]])       # shifted in its own
    assert clip(L, [a, b], [(P, 100, 1), far[1]])           # its own, another type
    assert clip(L, [b, a], [(P + 400, 100, 0), far[0]])
    assert clip(L, [a, b], [(P + 400, 100, 0), far[1]])     # in another gradient
    assert clip(L, [(P, 1000, 0), (8 * P, 4, 0)], [(2 * P, 1000, 0), (P + 800, 4, 0)])
    assert clip(L, [(P, 1000, 0), (8 * P, 4, 0)], [(2 * P, 1000, 0), (2 * P + 800, 4, 0)])


def test_the_norm_in_a_tensor(L):
    a = (P, 100, 0)
    assert clip(L, [a], [a], norm=P + 396) and not clip(L, [a], [a], norm=P + 400)
    assert clip(L, [a], [(2 * P, 100, 0)], norm=2 * P)
    assert not clip(L, [a], [(2 * P, 100, 0)], norm=P)  # read twice
    need = L.moe_grad_norm_workspace_bytes(1)
    for at in (P, P + 396):
        status = L.moe_grad_norm((ctypes.c_void_p * 1)(P), (ctypes.c_int64 * 1)(100), b"\0", 1, at,
                                 1 << 30, need, None)
        assert status == INVALID and b"norm overlaps tensor 0" in L.moe_last_error()


def overlapping(grads, out):
    """The same by comparing all pairs."""
    def span(t):
        return t[0], t[0] + t[1] * (2 if t[2] else 4)

    def cross(a, b):
        return a[0] < b[1] and b[0] < a[1]

    n = len(grads)
    for i in range(n):
        for j in range(n):
            if i != j and cross(span(out[i]), span(out[j])):
                return True
            own = i == j and grads[i][0] == out[i][0] and grads[i][2] == out[i][2]
            if not own and cross(span(out[i]), span(grads[j])):
                return True
    return False


@pytest.mark.parametrize("n", [1, 3, 40, 300])
def test_sets_in_any_order(L, n):
    rng = random.Random(n)
    found = set()
    for _ in range(60):
        places = [P + 4 * rng.randrange(60 * n * n) for _ in range(2 * n)]
        grads = [(places[i], rng.randrange(1, 12), rng.randrange(2)) for i in range(n)]
        out = [(places[n + i], g[1], rng.randrange(2)) if rng.random() < 0.5 else g
               for i, g in enumerate(grads)]
        refused = clip(L, grads, out)
        assert refused == overlapping(grads, out)
        found.add(refused)
    assert n == 1 or len(found) == 2
