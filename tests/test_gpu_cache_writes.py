"""The KV cache writer where its work list and its lengths can go wrong (marked
gpu): codes, scales and lengths are exact values and have to be equal."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import attention as ref
from test_gpu_attention import D, World, bf16, rounded

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


def ints(a):
    return torch.tensor([int(x) for x in a], dtype=torch.int32, device="cuda")


def rows(s, n, H):
    return rounded(s.g.standard_normal((n, 2, H, D)))


def append(w12, s, x, off, **kw):
    k, v = (bf16(x[:, i].reshape(len(x), -1)) for i in range(2))
    return w12.w12_kv_append(s.cache, s.rope, k, v, ints(off), s.ws, **kw)


@pytest.mark.parametrize("off,served", [
    ([0, 40, 8, 48, 70], [0, 3]),              # 1: backwards; 2: behind it, over rows of 0
    ([0, 70, 0, 70, 70], [0, 3]),              # 2 would need as many blocks again as the grid has
    ([30, 10, 20, 30, 70], [3]),               # 3 starts where the largest offset before it was
    ([-5, 10, 30, 50, 71], [1, 2]),
])
def test_offsets_out_of_order(w12, off, served):
    """Requests behind a larger offset are refused, the others served, and the next append on the workspace is whole."""
    s = World(w12, [3, 30, 64, 5], 2, 32, room=200, seed=20)
    x = rows(s, 70, 2)
    append(w12, s, x, off)
    for r in served:
        ref.kv_write(s.host, r, x[off[r]:off[r + 1], 0], x[off[r]:off[r + 1], 1], s.cos, s.sin)
    s.same()
    assert s.ws.status() == w12.W12_E_INVAL
    good = [0, 20, 20, 41, 70]
    append(w12, s, x, good)
    for r in range(4):
        ref.kv_write(s.host, r, x[good[r]:good[r + 1], 0], x[good[r]:good[r + 1], 1], s.cos, s.sin)
    s.same()
    assert s.ws.status() == 0


def test_offsets_out_of_order_among_many_requests(w12):
    """The same over more requests than a warp has lanes, the faults on both sides of a warp's end."""
    n = 75
    s = World(w12, [0] * n, 1, 32, room=130, seed=21)
    off = np.arange(n + 1) * 3
    off[32] = 200                              # 31 takes the rows of 32 .. 66 as well
    off[70] = 10                               # 69 runs backwards, 70 over rows served before
    x = rows(s, int(off[-1]), 1)
    append(w12, s, x, off)
    high = np.maximum.accumulate(off)
    for r in range(n):
        if off[r] <= off[r + 1] and off[r] == high[r]:
            ref.kv_write(s.host, r, x[off[r]:off[r + 1], 0], x[off[r]:off[r + 1], 1], s.cos, s.sin)
    s.same()
    assert s.ws.status() == w12.W12_E_INVAL


@pytest.mark.parametrize("length", [INT_MAX, INT_MAX - 1, INT_MAX - 60, -1, -2 ** 31])
@pytest.mark.parametrize("commit", [False, True])
def test_lengths_out_of_range(w12, length, commit):
    """A request whose length is no length is refused and changes nothing for those behind it."""
    s = World(w12, [4, 4, 4, 33], 1, 32, room=200, seed=22)
    s.host["len"][1] = length
    s.upload()
    off = np.asarray([0, 2, 66, 68, 70], np.int32)
    x = rows(s, 70, 1)
    if commit:
        parent = np.arange(70) - 1
        parent[off[:-1]] = -1
        depth = np.concatenate([np.arange(b - a) for a, b in zip(off, off[1:])])
        tree = w12.DeviceTree.from_arrays(ints(parent), torch.from_numpy(depth.astype(np.uint8)).cuda(),
                                          ints(np.repeat(np.arange(4), np.diff(off))), ints(off))
        acc = [1, 30, 67, 69]
        k, v = (bf16(x[:, i].reshape(70, -1)) for i in range(2))
        w12.w12_kv_commit(s.cache, s.rope, tree, 4, ints(acc), k, v, s.ws)
    else:
        append(w12, s, x, off)
    for r in (0, 2, 3):
        ref.kv_write(s.host, r, x[off[r]:off[r + 1], 0], x[off[r]:off[r + 1], 1], s.cos, s.sin)
    s.same()
    assert s.ws.status() == w12.W12_E_INVAL
