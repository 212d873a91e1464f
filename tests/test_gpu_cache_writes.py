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


def counters(s):
    """The writer's words of the workspace: its arrivals."""
    return s.ws.buf[256:256 + 2048].view(torch.int32).tolist()


@pytest.mark.parametrize("n,top,H,bt", [(70, 900, 1, 128), (48, 1400, 3, 128), (90, 700, 2, 32), (300, 150, 1, 64)])
def test_in_place_over_several_waves(w12, n, top, H, bt):
    """More CTAs than the SMs hold at once, the lengths written where they are read: two appends and a commit on one
    workspace."""
    g = np.random.default_rng(n)
    s = World(w12, [int(x) for x in g.integers(0, 2 * bt, n)], H, bt, room=2 * top + 1, seed=n)
    for _ in range(2):
        cnt = g.integers(0, top, n)
        off = np.concatenate([[0], np.cumsum(cnt)])
        x = rows(s, int(off[-1]), H)
        append(w12, s, x, off)
        for r in range(n):
            ref.kv_write(s.host, r, x[off[r]:off[r + 1], 0], x[off[r]:off[r + 1], 1], s.cos, s.sin)
        s.same()
        assert not any(counters(s))
    t = chains(w12, n, 1)
    x = rows(s, n, H)
    w12.w12_kv_commit(s.cache, s.rope, t, n, ints(range(n)), bf16(x[:, 0].reshape(n, -1)), bf16(x[:, 1].reshape(n, -1)), s.ws)
    for r in range(n):
        ref.kv_write(s.host, r, x[r:r + 1, 0], x[r:r + 1, 1], s.cos, s.sin)
    s.same()
    assert not any(counters(s)) and s.ws.status() == 0


def chains(w12, n, each):
    """n requests of one chain of `each` rows."""
    j = np.tile(np.arange(each), n)
    parent = np.where(j == 0, -1, np.arange(n * each) - 1)
    return w12.DeviceTree.from_arrays(ints(parent), torch.from_numpy(j.astype(np.uint8)).cuda(), ints(np.repeat(np.arange(n), each)),
                                      ints(np.arange(n + 1) * each))


@pytest.mark.parametrize("n,each,H,bt", [(500, 1, 4, 128), (60, 8, 8, 32), (15, 34, 16, 32), (128, 4, 8, 64)])
def test_in_place_commits_of_many_requests(w12, n, each, H, bt):
    """More CTAs without a block of their own than with one; many lengths change the number of blocks that the same rows
    would touch behind them."""
    g = np.random.default_rng(n)
    s = World(w12, [int(x) for x in g.integers(0, 2 * bt, n)], H, bt, room=4 * each + 1, seed=23)
    t = chains(w12, n, each)
    for _ in range(3):
        x = rows(s, n * each, H)
        acc = np.arange(n) * each + g.integers(0, each, n)
        k, v = (bf16(x[:, i].reshape(n * each, -1)) for i in range(2))
        w12.w12_kv_commit(s.cache, s.rope, t, n, ints(acc), k, v, s.ws)
        for r in range(n):
            path = range(r * each, acc[r] + 1)
            ref.kv_write(s.host, r, x[path, 0], x[path, 1], s.cos, s.sin)
        s.same()
        assert not any(counters(s)) and s.ws.status() == 0


def test_in_place_is_as_apart(w12):
    """A long append of many requests, the lengths in place and apart: the same caches."""
    n, H, bt = 24, 8, 128
    g = np.random.default_rng(24)
    lens, cnt = g.integers(0, 300, n), g.integers(500, 4000, n)
    off = np.concatenate([[0], np.cumsum(cnt)])
    per = -(-int((lens + cnt).max()) // bt)
    x = [torch.randn(int(off[-1]), H * D, device="cuda").bfloat16() for _ in range(2)]
    table = torch.arange(n * per, dtype=torch.int32, device="cuda").view(n, per)
    ws = w12.Workspace(1, 0, 0, n)
    got = []
    for apart in (True, False):
        c = w12.KvCache.empty(n * per, H, bt, table)
        c.len.copy_(ints(lens))
        out = w12.w12_kv_append(c, None, x[0], x[1], ints(off), ws, len_out=torch.empty_like(c.len) if apart else None)
        got.append((c.k, c.v, c.k_scale, c.v_scale, out))
    assert got[0][4].tolist() == (lens + cnt).tolist() and all(torch.equal(a, b) for a, b in zip(*got))
    assert ws.status() == 0


@pytest.mark.parametrize("bt", [32, 64, 128])
def test_every_rotated_width(w12, bt):
    """Append and commit at every number of rotated dimensions, whose tables lie in shared memory."""
    for rot in range(0, 129, 8):
        s = World(w12, [bt - 3, 5], 2, bt, rot, bool(rot & 8), room=2 * bt + 8, seed=rot)
        off = [0, 7, 7 + bt]
        x = rows(s, off[-1], 2)
        append(w12, s, x, off)
        for r in range(2):
            ref.kv_write(s.host, r, x[off[r]:off[r + 1], 0], x[off[r]:off[r + 1], 1], s.cos, s.sin, bool(rot & 8))
        s.same()
        x = rows(s, 8, 2)
        k, v = (bf16(x[:, i].reshape(8, -1)) for i in range(2))
        w12.w12_kv_commit(s.cache, s.rope, chains(w12, 2, 4), 2, ints([3, 6]), k, v, s.ws)
        for r, path in enumerate((range(4), range(4, 7))):
            ref.kv_write(s.host, r, x[path, 0], x[path, 1], s.cos, s.sin, bool(rot & 8))
        s.same()
        assert s.ws.status() == 0


def test_no_rows(w12):
    """An append without rows, whatever strides an empty tensor has, reports the lengths as they are."""
    s = World(w12, [5, 40], 2, 32, seed=25)
    none = torch.empty(0, dtype=torch.bfloat16, device="cuda")
    for k in (none.view(0, 2 * D), none.as_strided((0, 2 * D), (0, 0)), none.as_strided((0, 2 * D), (1, 7))):
        out = w12.w12_kv_append(s.cache, s.rope, k, k, ints([0, 0, 0]), s.ws, len_out=torch.full_like(s.cache.len, -5))
        s.same()
        assert out.tolist() == [5, 40] and s.ws.status() == 0
