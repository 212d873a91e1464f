"""GPU parity of the KV cache writer and the tree attention through the C ABI,
against the 64-bit forms in oracle/attention.py (marked gpu).

Cache codes, scales and lengths are exact values: they have to be equal.
Attention outputs are held to the bound that the oracle derives for each of
them from the roundings the kernel may make (see tree_attention there)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import attention as ref
from speculative_decoding_tree_w12_gb300 import synth

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


def bf16(a):
    return torch.from_numpy(synth.f32_to_bf16_bits(np.asarray(a, np.float32)).view(np.int16)).cuda().view(torch.bfloat16)


def rounded(a):
    return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(np.asarray(a, np.float32)))


def tables(rot, n):
    if rot == 0:
        return None, None
    f = 10000.0 ** (-np.arange(rot // 2) / (rot / 2))
    a = np.arange(n)[:, None] * f
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


class World:
    """A cache filled through the oracle, on the host and on the GPU."""

    def __init__(self, w12, lens, H, bt, rot=128, adjacent=False, room=40, seed=0, junk=0x7F, n_pos=None):
        g = np.random.default_rng(seed)
        self.g, self.w12, self.H, self.bt, self.adjacent = g, w12, H, bt, adjacent
        n = len(lens)
        need = [-(-(x + room) // bt) for x in lens]
        nb = sum(need) + 2
        order = g.permutation(nb)
        table = np.full((n, max(need)), -1, np.int32)       # entries past a request's blocks are no blocks
        at = 0
        for r, m in enumerate(need):
            table[r, :m] = order[at:at + m]
            at += m
        self.cos, self.sin = tables(rot, n_pos or max(lens) + room)
        self.host = dict(k=np.full((nb, H, bt, D), junk, np.uint8), v=np.full((nb, H, D, bt), junk, np.uint8),
                         k_scale=np.full((nb, H), np.nan, np.float32), v_scale=np.full((nb, H), np.nan, np.float32),
                         table=table, len=np.zeros(n, np.int32))
        for r, x in enumerate(lens):
            ref.kv_write(self.host, r, rounded(g.standard_normal((x, H, D))), rounded(g.standard_normal((x, H, D))),
                         self.cos, self.sin, adjacent)
        self.upload()
        c = lambda a: torch.from_numpy(a).cuda()
        self.rope = w12.Rope(c(self.cos), c(self.sin), adjacent) if rot else None
        self.ws = w12.Workspace(1, 0, 0, n)

    def upload(self):
        c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        h = self.host
        self.cache = self.w12.KvCache(c(h["k"]), c(h["v"]), c(h["k_scale"]), c(h["v_scale"]), c(h["table"]), c(h["len"]))

    def same(self):
        torch.cuda.synchronize()
        for name in ("k", "v", "k_scale", "v_scale", "len"):
            got, want = getattr(self.cache, name).cpu().numpy(), self.host[name]
            assert np.array_equal(got, want, equal_nan=name.endswith("scale")), name


def make_tree(g, rows, chain=False):
    parent, depth, req, off = [], [], [], [0]
    for r, n in enumerate(rows):
        base = len(parent)
        for j in range(n):
            p = -1 if j == 0 else (len(parent) - 1 if chain else base + int(g.integers(0, j)))
            if p >= 0 and depth[p] >= 33:
                p = base
            parent.append(p)
            depth.append(0 if p < 0 else depth[p] + 1)
            req.append(r)
        off.append(len(parent))
    return (np.asarray(parent, np.int32), np.asarray(depth, np.uint8), np.asarray(req, np.int32), np.asarray(off, np.int32))


def dev_tree(w12, t, token=None):
    c = lambda a: torch.from_numpy(a).cuda()
    return w12.DeviceTree.from_arrays(c(t[0]), c(t[1]), c(t[2]), c(t[3]), token=None if token is None else c(token))


# ---------------------------------------------------------------------------
# cache
# ---------------------------------------------------------------------------

APPENDS = [
    # lengths before, new tokens, heads, block, rotated dimensions, adjacent pairs
    ([0], [1], 1, 64, 128, False),
    ([5], [1], 2, 32, 128, False),
    ([63], [2], 2, 64, 128, True),
    ([0, 1, 31, 32, 33], [33, 0, 1, 32, 95], 3, 32, 64, False),
    ([127, 128, 129], [1, 300, 127], 1, 128, 32, True),
    ([10, 0], [0, 0], 2, 64, 128, False),
    ([7] * 40, list(range(40)), 1, 32, 0, False),
]


@pytest.mark.parametrize("lens,new,H,bt,rot,adjacent", APPENDS)
def test_append(w12, lens, new, H, bt, rot, adjacent):
    s = World(w12, lens, H, bt, rot, adjacent, room=max(new) + 1, seed=3)
    T = sum(new)
    x = rounded(s.g.standard_normal((T, 2, H, D)) * np.exp(s.g.uniform(-3, 3, (T, 1, H, 1))))
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    fused = bf16(x.reshape(T, 2 * H * D))
    fused = torch.cat([torch.zeros(T, 8, dtype=torch.bfloat16, device="cuda"), fused], 1)     # rows of a wider buffer
    w12.w12_kv_append(s.cache, s.rope, fused[:, 8:8 + H * D], fused[:, 8 + H * D:], torch.from_numpy(off).cuda(), s.ws)
    for r in range(len(lens)):
        rows = x[off[r]:off[r + 1]]
        ref.kv_write(s.host, r, rows[:, 0], rows[:, 1], s.cos, s.sin, adjacent)
    s.same()
    assert s.ws.status() == 0


@pytest.mark.parametrize("bt,rot,adjacent", [(32, 128, False), (64, 64, True), (128, 0, False), (128, 128, False)])
def test_append_long(w12, bt, rot, adjacent):
    """Enough tokens and heads that a CTA takes several heads of a block."""
    lens, new, H = [5, 0, 77], [4001, 6000, 33], 16
    s = World(w12, lens, H, bt, rot, adjacent, room=6001, seed=4)
    x = rounded(s.g.standard_normal((sum(new), 2, H, D)) * np.exp(s.g.uniform(-3, 3, (sum(new), 1, H, 1))))
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v = (bf16(x[:, i].reshape(-1, H * D)) for i in range(2))
    w12.w12_kv_append(s.cache, s.rope, k, v, torch.from_numpy(off).cuda(), s.ws)
    for r in range(len(lens)):
        rows = x[off[r]:off[r + 1]]
        ref.kv_write(s.host, r, rows[:, 0], rows[:, 1], s.cos, s.sin, adjacent)
    s.same()
    assert s.ws.status() == 0


@pytest.mark.parametrize("bt", [32, 128])
def test_growing_block(w12, bt):
    """One token at a time through a block, each larger than the ones before:
    every append rounds the codes again under the larger scale."""
    s = World(w12, [0], 2, bt, room=bt, seed=5)
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for i in range(20):
        x = rounded(s.g.standard_normal((1, 2, 2, D)) * 1.7 ** i * 1e-3)
        w12.w12_kv_append(s.cache, s.rope, bf16(x[:, 0].reshape(1, -1)), bf16(x[:, 1].reshape(1, -1)), off, s.ws)
        ref.kv_write(s.host, 0, x[:, 0], x[:, 1], s.cos, s.sin)
        s.same()


def test_zeros_tiny_huge_and_not_finite(w12):
    s = World(w12, [3], 1, 64, rot=0, room=64, seed=6)
    x = np.zeros((5, 1, D), np.float32)
    x[1, 0, :4] = [1e-30, -1e-38, 2.0 ** -41, 2.0 ** -42]
    x[2, 0, :4] = [np.inf, -np.inf, np.nan, 3.0]
    x[3, 0, :2] = [3e38, -3e38]
    for rows in (x[:2], x[2:3], x[3:4], x[4:5]):
        n = len(rows)
        off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        w12.w12_kv_append(s.cache, None, bf16(rows.reshape(n, -1)), bf16(rows.reshape(n, -1)), off, s.ws)
        ref.kv_write(s.host, 0, rounded(rows), rounded(rows), None, None)
        torch.cuda.synchronize()
        for name in ("k", "v"):
            got, want = getattr(s.cache, name).cpu().numpy(), s.host[name]
            assert np.array_equal(ref.E4M3[got], ref.E4M3[want], equal_nan=True)
            assert np.array_equal(getattr(s.cache, name + "_scale").cpu().numpy(), s.host[name + "_scale"], equal_nan=True)


@pytest.mark.parametrize("rows,chain,bt", [([1], True, 64), ([34], True, 32), ([9, 1, 30, 2], False, 32), ([8] * 24, False, 64),
                                           ([300], False, 128)])
def test_commit(w12, rows, chain, bt):
    g = np.random.default_rng(8)
    lens = [int(x) for x in g.integers(0, 150, len(rows))]
    s = World(w12, lens, 2, bt, seed=9)
    t = make_tree(g, rows, chain)
    R = len(t[0])
    acc = np.asarray([t[3][r + 1] - 1 for r in range(len(rows))], np.int32)
    x = rounded(g.standard_normal((R, 2, 2, D)))
    out = torch.empty(len(rows), dtype=torch.int32, device="cuda")
    w12.w12_kv_commit(s.cache, s.rope, dev_tree(w12, t), len(rows), torch.from_numpy(acc).cuda(),
                      bf16(x[:, 0].reshape(R, -1)), bf16(x[:, 1].reshape(R, -1)), s.ws, len_out=out)
    for r, a in enumerate(acc):
        path = ref.root_path(t[0], int(a))
        ref.kv_write(s.host, r, x[path, 0], x[path, 1], s.cos, s.sin)
    torch.cuda.synchronize()
    assert out.cpu().tolist() == s.host["len"].tolist() and s.cache.len.cpu().tolist() == lens
    s.cache.len.copy_(out)
    s.same()
    assert s.ws.status() == 0


def test_cache_refusals_on_the_device(w12):
    """Offsets, lengths and blocks out of range leave their request as it was and the others served."""
    cases = [("block outside the pool", lambda s: s.host["table"].__setitem__((1, 0), 10 ** 6)),
             ("negative length", lambda s: s.host["len"].__setitem__(1, -1)),
             ("past the table", lambda s: s.host["len"].__setitem__(1, s.host["table"].shape[1] * 32 - 1))]
    for what, spoil in cases:
        s = World(w12, [4, 4, 4], 1, 32, seed=1)
        spoil(s)
        s.upload()
        x = rounded(s.g.standard_normal((6, 2, 1, D)))
        off = np.asarray([0, 2, 4, 6], np.int32)
        w12.w12_kv_append(s.cache, s.rope, bf16(x[:, 0].reshape(6, -1)), bf16(x[:, 1].reshape(6, -1)),
                          torch.from_numpy(off).cuda(), s.ws)
        for r in (0, 2):
            ref.kv_write(s.host, r, x[off[r]:off[r + 1], 0], x[off[r]:off[r + 1], 1], s.cos, s.sin)
        s.same()
        assert s.ws.status() == w12.W12_E_INVAL, what
        assert s.ws.status() == 0
    s = World(w12, [4, 4], 1, 32, seed=1)
    t = make_tree(s.g, [3, 3])
    x = rounded(s.g.standard_normal((6, 2, 1, D)))
    w12.w12_kv_commit(s.cache, s.rope, dev_tree(w12, t), 2, torch.tensor([4, 3], dtype=torch.int32, device="cuda"),
                      bf16(x[:, 0].reshape(6, -1)), bf16(x[:, 1].reshape(6, -1)), s.ws)
    ref.kv_write(s.host, 1, x[3:4, 0], x[3:4, 1], s.cos, s.sin)
    s.same()
    assert s.ws.status() == w12.W12_E_INVAL


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

ATTENDS = [
    # cached tokens, rows per request, heads, group, block, rotated dimensions, adjacent, chain
    ([0], [1], 1, 1, 64, 128, False, True),
    ([1], [1], 1, 5, 32, 128, False, True),
    ([127], [1], 2, 4, 64, 128, False, True),
    ([128], [3], 2, 5, 128, 64, True, False),
    ([129], [7], 1, 3, 32, 128, False, False),
    ([1000], [32], 2, 5, 64, 128, False, False),
    ([0, 1, 33, 500, 64], [1, 4, 1, 9, 2], 2, 5, 32, 32, True, False),
    ([300] * 24, [8] * 24, 1, 5, 64, 128, False, False),
    ([700], [34], 1, 2, 128, 0, False, True),
    ([200, 90], [100, 60], 1, 5, 64, 128, False, False),
    ([257], [5], 1, 64, 64, 128, False, False),
    ([5000], [2], 1, 8, 32, 128, False, True),
]


def inputs(g, R, H, G, s, q_std=2.0):
    x = g.standard_normal((R, (G + 2) * H, D))
    x[:, :G * H] *= q_std
    x = rounded(x)
    fused = bf16(x.reshape(R, -1))
    return x[:, :G * H], x[:, G * H:(G + 1) * H], x[:, (G + 1) * H:], \
        (fused[:, :G * H * D], fused[:, G * H * D:(G + 1) * H * D], fused[:, (G + 1) * H * D:])


def attend(w12, s, t, dev, H, G, n_req, **kw):
    aws = w12.AttentionWorkspace(len(t[0]), H * G, H, n_req)
    aws.buf.fill_(0xFF)                       # the scratch needs no initialisation
    out = w12.w12_tree_attention(s.cache, s.rope, dev_tree(w12, t), n_req, *dev, s.ws, aws, **kw)
    torch.cuda.synchronize()
    return out


def close(out, want, slack):
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    worst = (np.abs(got - want) / np.maximum(slack, 1e-30)).max()
    assert worst <= 1.0, worst


@pytest.mark.parametrize("lens,rows,H,G,bt,rot,adjacent,chain", ATTENDS)
def test_attention(w12, lens, rows, H, G, bt, rot, adjacent, chain):
    s = World(w12, lens, H, bt, rot, adjacent, seed=11)     # slots past each length hold NaN codes
    t = make_tree(s.g, rows, chain)
    q, k, v, dev = inputs(s.g, len(t[0]), H, G, s)
    out = attend(w12, s, t, dev, H, G, len(lens))
    assert s.ws.status() == 0
    close(out, *ref.tree_attention(s.host, t[0], t[1], t[2], q, k, v, s.cos, s.sin, adjacent, D ** -0.5))
    again = attend(w12, s, t, dev, H, G, len(lens))
    assert torch.equal(out, again)


def _many(n, seed):
    g = np.random.default_rng(seed)
    return [int(x) for x in g.integers(0, 5000, n)], [int(x) for x in g.integers(1, 5, n)]


# enough tiles that the split counts segments and columns: few long requests whose
# rows need several groups, some without tokens; more requests than a warp has lanes
LONG = [([9000, 3001, 0, 12345, 700], [8, 12, 2, 1, 30], 4, 5, 64), _many(40, 1) + (2, 4, 32), ([40000], [3], 2, 8, 128),
        _many(70, 2) + (1, 8, 64)]


@pytest.mark.parametrize("lens,rows,H,G,bt", LONG)
def test_attention_long(w12, lens, rows, H, G, bt):
    s = World(w12, lens, H, bt, 64, False, seed=16)
    t = make_tree(s.g, rows)
    q, k, v, dev = inputs(s.g, len(t[0]), H, G, s)
    out = attend(w12, s, t, dev, H, G, len(lens))
    assert s.ws.status() == 0
    close(out, *ref.tree_attention(s.host, t[0], t[1], t[2], q, k, v, s.cos, s.sin, False, D ** -0.5))
    assert torch.equal(out, attend(w12, s, t, dev, H, G, len(lens)))


def test_attention_scales_and_sinks(w12):
    """Blocks whose scales differ by 2^20, a key every row attends to most, and a large softmax scale."""
    s = World(w12, [600], 1, 64, rot=0, seed=12)
    b = s.host["table"][0]
    s.host["k_scale"][b[3]] *= 2.0 ** 3
    s.host["v_scale"][b[2]] *= 2.0 ** 10
    s.host["v_scale"][b[5]] *= 2.0 ** -10
    s.host["v"][b[6]] = 0                                   # a block of zeros under the least scale
    s.host["v_scale"][b[6]] = 2.0 ** -32
    s.upload()
    t = make_tree(s.g, [6])
    q, k, v, dev = inputs(s.g, 6, 1, 5, s)
    for scale in (D ** -0.5, 0.5):
        close(attend(w12, s, t, dev, 1, 5, 1, scale=scale),
              *ref.tree_attention(s.host, t[0], t[1], t[2], q, k, v, None, None, False, scale))


def test_rows_off_the_path_and_stale_slots_cannot_reach_an_output(w12):
    s = World(w12, [100, 70], 1, 32, seed=13)
    t = make_tree(s.g, [6, 6])
    q, k, v, dev = inputs(s.g, 12, 1, 5, s)
    clean = attend(w12, s, t, dev, 1, 5, 2)
    on_path = ref.root_path(t[0], 5)
    off = [j for j in range(6) if j not in on_path]
    assert off
    dev[1][off] = float("nan")
    dev[2][off] = float("inf")
    dirty = attend(w12, s, t, dev, 1, 5, 2)
    keep = [i for i in range(12) if not set(ref.root_path(t[0], i)) & set(off)]
    assert 5 in keep and torch.equal(clean[keep], dirty[keep])
    assert not torch.isfinite(dirty[off].float()).all()
    assert s.ws.status() == 0


def test_zero_values_and_extreme_queries(w12):
    s = World(w12, [200], 1, 64, seed=14)
    s.host["v"][:] = 0
    s.upload()
    t = make_tree(s.g, [3])
    q, k, v, dev = inputs(s.g, 3, 1, 2, s)
    dev[2].zero_()
    assert (attend(w12, s, t, dev, 1, 2, 1) == 0).all()
    s = World(w12, [200], 1, 64, rot=0, seed=15)
    t = make_tree(s.g, [3])
    q, k, v, dev = inputs(s.g, 3, 1, 2, s)
    dev[0].zero_()                                          # all scores equal
    q[:] = 0
    close(attend(w12, s, t, dev, 1, 2, 1), *ref.tree_attention(s.host, t[0], t[1], t[2], q, k, v, None, None, False, 0.1))
    dev[0].fill_(2.0 ** -100)                               # scores that are all but equal
    close(attend(w12, s, t, dev, 1, 2, 1), *ref.tree_attention(s.host, t[0], t[1], t[2], q, k, v, None, None, False, 0.1))


@pytest.mark.parametrize("G", [1, 5, 16])
def test_attention_wait_times_out_cleanly(w12, G):
    """CTA 0 never copies a key (test hook): the scores' wait runs out after
    50 ms, every warp stops, tensor memory is released, the status word reads
    W12_E_TIMEOUT, and the same call without the hook matches the 64-bit form."""
    s = World(w12, [3000], 1, 64, rot=0, seed=17)
    t = make_tree(s.g, [4])
    q, k, v, dev = inputs(s.g, 4, 1, G, s)
    w12.debug_set(1, 50_000_000)
    try:
        attend(w12, s, t, dev, 1, G, 1)
        torch.cuda.synchronize()
        assert s.ws.status() == w12.W12_E_TIMEOUT
    finally:
        w12.debug_set(0, 0)
    out = attend(w12, s, t, dev, 1, G, 1)
    assert s.ws.status() == 0
    close(out, *ref.tree_attention(s.host, t[0], t[1], t[2], q, k, v, None, None, False, D ** -0.5))


def test_attention_device_checks(w12):
    def spoil_parent(s, t):
        t[0][4] = 5

    def spoil_req(s, t):
        t[2][3] = 9

    def spoil_len(s, t):
        s.host["len"][1] = s.host["table"].shape[1] * 32 + 1

    def spoil_block(s, t):
        s.host["table"][1, 0] = -5

    for spoil in (spoil_parent, spoil_req, spoil_len, spoil_block):
        s = World(w12, [50, 60], 1, 32, seed=16)
        t = make_tree(s.g, [3, 3], chain=True)
        q, k, v, dev = inputs(s.g, 6, 1, 2, s)
        spoil(s, t)
        s.upload()
        out = attend(w12, s, t, dev, 1, 2, 2)
        assert s.ws.status() == w12.W12_E_INVAL, spoil.__name__
        want, slack = ref.tree_attention({**s.host, "len": np.asarray([50, 0])}, t[0], t[1], np.zeros(6, np.int32), q, k, v,
                                         s.cos, s.sin, False, D ** -0.5) if spoil is not spoil_parent else (None, None)
        if want is not None:
            close(out[:3], want[:3], slack[:3])


def test_on_another_stream(w12):
    s = World(w12, [400, 9], 2, 64, seed=17)
    t = make_tree(s.g, [5, 6])
    q, k, v, dev = inputs(s.g, 11, 2, 4, s)
    want = attend(w12, s, t, dev, 2, 4, 2)
    side = torch.cuda.Stream()
    aws, tree = w12.AttentionWorkspace(11, 8, 2, 2), dev_tree(w12, t)
    torch.cuda.synchronize()
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):                  # and inside a graph
        w12.w12_tree_attention(s.cache, s.rope, tree, 2, *dev, s.ws, aws, out=out)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
