"""Host tests of the KV cache, tree attention and sampled verification: the
64-bit forms pinned by hand, and the refusals of the entry points (every bad
argument is turned away before any launch, so no GPU is needed)."""
from __future__ import annotations

import ctypes as C

import numpy as np
import pytest

from oracle import attention as ref


# ---------------------------------------------------------------------------
# the 64-bit forms
# ---------------------------------------------------------------------------

def test_e4m3_round_trip_and_ties():
    codes = np.arange(256, dtype=np.uint8)
    fin = (codes & 127) != 127
    back = ref.e4m3_encode(ref.E4M3[fin])
    assert np.array_equal(ref.E4M3[back], ref.E4M3[fin])
    assert ref.E4M3[126] == 448 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[8] == 2.0 ** -6
    # halfway cases go to the even mantissa
    assert ref.E4M3[ref.e4m3_encode(1.0625)] == 1.0 and ref.E4M3[ref.e4m3_encode(1.1875)] == 1.25
    assert ref.E4M3[ref.e4m3_encode(2.0 ** -10)] == 0.0 and ref.E4M3[ref.e4m3_encode(3 * 2.0 ** -10)] == 2.0 ** -8


def test_block_scale():
    for top, want in ((448.0, 1.0), (448.5, 2.0), (224.0, 0.5), (1.75, 2.0 ** -8), (0.0, 2.0 ** -32), (1e-30, 2.0 ** -32)):
        assert ref.block_scale(top) == want


def test_turn_keeps_pair_norms_and_composes():
    g = np.random.default_rng(0)
    a = np.arange(20)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    cos, sin = np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)
    x = g.standard_normal(128).astype(np.float32)
    for adjacent in (False, True):
        y = ref.turn(x, 7, cos, sin, adjacent)
        assert np.array_equal(y[64:], x[64:])
        i = np.arange(32)
        p, q = (2 * i, 2 * i + 1) if adjacent else (i, i + 32)
        assert np.allclose(y[p] ** 2 + y[q] ** 2, x[p] ** 2 + x[q] ** 2, rtol=1e-5)
        assert np.allclose(ref.turn(y, 5, cos, sin, adjacent), ref.turn(x, 12, cos, sin, adjacent), atol=1e-5)


def test_attention_of_one_key_is_its_value():
    cache = dict(k=np.zeros((1, 1, 32, 128), np.uint8), v=np.zeros((1, 1, 128, 32), np.uint8),
                 k_scale=np.ones((1, 1), np.float32), v_scale=np.ones((1, 1), np.float32),
                 table=np.zeros((1, 1), np.int32), len=np.zeros(1, np.int32))
    v = np.arange(128, dtype=np.float32).reshape(1, 1, 128)
    out, _ = ref.tree_attention(cache, np.asarray([-1]), np.asarray([0]), np.asarray([0]), np.ones((1, 2, 128), np.float32),
                                np.ones((1, 1, 128), np.float32), v, None, None, False, 0.1)
    assert np.array_equal(out[0, 0], v[0, 0]) and np.array_equal(out[0, 1], v[0, 0])


def test_rejection_sampling_gives_the_target_distribution():
    """One child drawn from q, then accepted, or replaced from the residual: summed over the draws, that is p."""
    p = np.asarray([0.1, 0.5, 0.2, 0.2])
    q = np.asarray([0.4, 0.1, 0.25, 0.25])
    got = np.zeros(4)
    n = 400
    for x in range(4):
        for ua in (np.arange(n) + 0.5) / n:
            if ua * q[x] < p[x]:
                got[x] += q[x] / n
            else:
                rest = np.maximum(p - q, 0)
                got += q[x] / n * rest / rest.sum()
                for us in (0.1, 0.9):
                    may = ref.sample_row(p, [x], q, [ua], us, 0.0)
                    assert len(may) == 1 and rest[next(iter(may))] > 0
    assert np.abs(got - p).max() < 2.0 / n


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


A = 0x10000          # never dereferenced: every call below is refused on the host
INVAL, UNSUPPORTED, WORKSPACE = -1, -2, -6


def good(w12):
    cache = w12.KvCacheC(2, 128, 64, 16, 4, A, A, A, A, A, A)
    rope = w12.RopeC(128, 0, 1000, A, A)
    tree = w12.TreeC(4, A, A, A, A, A, A, A)
    return cache, rope, tree


def test_append_and_commit_refusals(w12):
    L = w12.lib()
    nbytes = int(L.w12_workspace_bytes(1, 0, 0, 3))

    def append(cache, rope, n_req=3, k=A, ks=256, v=A, vs=256, rows=5, off=A, out=A, ws=A, wsb=nbytes):
        return L.w12_kv_append(C.byref(cache) if cache else None, C.byref(rope) if rope else None, n_req, k, ks, v, vs, rows,
                               off, out, ws, wsb, None)

    def commit(cache, rope, tree, acc=A, **kw):
        a = dict(n_req=3, k=A, ks=256, v=A, vs=256, out=A, ws=A, wsb=nbytes)
        a.update(kw)
        return L.w12_kv_commit(C.byref(cache), C.byref(rope), C.byref(tree) if tree else None, a["n_req"], acc, a["k"], a["ks"],
                               a["v"], a["vs"], a["out"], a["ws"], a["wsb"], None)

    cache, rope, tree = good(w12)
    for kw, want in ((dict(n_req=0), INVAL), (dict(n_req=513), UNSUPPORTED), (dict(k=None), INVAL), (dict(k=A + 2), INVAL),
                     (dict(ks=248), INVAL), (dict(vs=260), INVAL), (dict(v=A + 8), INVAL), (dict(rows=-1), INVAL),
                     (dict(off=None), INVAL), (dict(out=None), INVAL), (dict(ws=None), WORKSPACE), (dict(ws=A + 16), WORKSPACE),
                     (dict(wsb=nbytes - 1), WORKSPACE)):
        assert append(cache, rope, **kw) == want, kw
    assert append(None, rope) == INVAL
    for field, value, want in (("head_dim", 64, UNSUPPORTED), ("head_dim", 0, UNSUPPORTED), ("block_tokens", 16, UNSUPPORTED),
                               ("block_tokens", 48, UNSUPPORTED), ("n_kv_heads", 0, INVAL), ("n_kv_heads", 2000, UNSUPPORTED),
                               ("n_blocks", 0, INVAL), ("max_blocks", 0, INVAL), ("k", None, INVAL), ("v", A + 4, INVAL),
                               ("k_scale", None, INVAL), ("block_table", None, INVAL), ("len", None, INVAL),
                               ("n_blocks", 2 ** 31 - 1, UNSUPPORTED), ("max_blocks", 2 ** 31 - 1, UNSUPPORTED)):
        c, _, _ = good(w12)
        setattr(c, field, value)
        assert append(c, rope) == want, field
        assert commit(c, rope, tree) == want, field
    for field, value, want in (("rot_dim", 3, INVAL), ("rot_dim", -2, INVAL), ("rot_dim", 130, UNSUPPORTED), ("max_pos", 0, INVAL),
                               ("cos", None, INVAL), ("sin", None, INVAL)):
        _, r, _ = good(w12)
        setattr(r, field, value)
        assert append(cache, r) == want, field
    assert commit(cache, rope, None) == INVAL
    assert commit(cache, rope, tree, acc=None) == INVAL
    assert commit(cache, rope, w12.TreeC(0, A, A, A, A, A, A, A)) == INVAL
    assert commit(cache, rope, w12.TreeC(513, A, A, A, A, A, A, A)) == UNSUPPORTED
    assert commit(cache, rope, w12.TreeC(4, None, A, A, A, A, A, A)) == INVAL


def test_attention_refusals(w12):
    L = w12.lib()
    nbytes = int(L.w12_workspace_bytes(1, 0, 0, 3))
    abytes = int(L.w12_attn_workspace_bytes(4, 10, 2, 3))
    assert abytes > 0
    for bad in ((0, 10, 2, 3), (513, 10, 2, 3), (4, 10, 3, 3), (4, 130, 2, 3), (4, 1, 2, 3), (4, 10, 0, 3), (4, 10, 2, 0),
                (4, 10, 2, 513)):
        assert L.w12_attn_workspace_bytes(*bad) == 0, bad

    def call(cache=None, rope=None, tree=None, **kw):
        c, r, t = good(w12)
        a = dict(n_req=3, heads=10, q=A, qs=1280, k=A, ks=256, v=A, vs=256, scale=0.1, out=A, ws=A, wsb=nbytes, aws=A, awsb=abytes)
        a.update(kw)
        return L.w12_tree_attention(C.byref(cache or c), C.byref(rope or r), C.byref(tree or t), a["n_req"], a["heads"], a["q"],
                                    a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["scale"], a["out"], a["ws"], a["wsb"], a["aws"],
                                    a["awsb"], None)

    for kw, want in ((dict(n_req=0), INVAL), (dict(heads=9), INVAL), (dict(heads=1), INVAL), (dict(heads=130), UNSUPPORTED),
                     (dict(q=None), INVAL), (dict(q=A + 2), INVAL), (dict(qs=1272), INVAL), (dict(qs=1284), INVAL),
                     (dict(k=None), INVAL), (dict(vs=128), INVAL), (dict(scale=0.0), INVAL), (dict(scale=-1.0), INVAL),
                     (dict(scale=float("nan")), INVAL), (dict(scale=float("inf")), INVAL), (dict(out=None), INVAL),
                     (dict(out=A + 8), INVAL), (dict(ws=None), WORKSPACE), (dict(wsb=10), WORKSPACE), (dict(aws=None), WORKSPACE),
                     (dict(aws=A + 64), WORKSPACE), (dict(awsb=abytes - 1), WORKSPACE)):
        assert call(**kw) == want, kw
    assert call(tree=w12.TreeC(4, A, A, A, None, A, A, A)) == INVAL
    assert call(tree=w12.TreeC(0, A, A, A, A, A, A, A)) == INVAL
    assert call(cache=w12.KvCacheC(2, 96, 64, 16, 4, A, A, A, A, A, A)) == UNSUPPORTED
    assert call(rope=w12.RopeC(129, 0, 10, A, A)) == INVAL


def test_sampling_refusals(w12):
    L = w12.lib()
    nbytes = int(L.w12_workspace_bytes(1, 0, 0, 3))
    top = int(L.w12_sample_max_vocab())
    assert top >= 262144

    def call(dist=None, tree=True, **kw):
        d = dist or dict()
        s = dict(logits=A, logits_f32=1, vocab=1000, logits_stride=1000, temperature=None, draft_p=None, draft_stride=0,
                 u_accept=None, u_sample=A)
        s.update(d)
        a = dict(n_req=3, p_max=4, row=A, logp=None, tok=A, length=A, node=None, ws=A, wsb=nbytes)
        a.update(kw)
        t = w12.TreeC(4, A, A, A, A, A, A, A) if tree is True else tree
        return L.w12_tree_verify_sampled(C.byref(w12.SamplingC(*s.values())), C.byref(t), a["n_req"], a["p_max"], a["row"], a["logp"],
                                         a["tok"], a["length"], a["node"], a["ws"], a["wsb"], None)

    for kw, want in ((dict(n_req=0), INVAL), (dict(n_req=513), UNSUPPORTED), (dict(p_max=-1), INVAL), (dict(p_max=34), UNSUPPORTED),
                     (dict(row=None), INVAL), (dict(tok=None), INVAL), (dict(length=None), INVAL), (dict(ws=None), WORKSPACE),
                     (dict(wsb=nbytes - 1), WORKSPACE)):
        assert call(**kw) == want, kw
    for d, want in ((dict(logits=None), INVAL), (dict(logits=A + 2), INVAL), (dict(logits=A + 1, logits_f32=0), INVAL),
                    (dict(vocab=0), INVAL), (dict(logits_stride=999), INVAL), (dict(u_sample=None), INVAL),
                    (dict(draft_p=A, draft_stride=1000), INVAL), (dict(draft_p=A, u_accept=A, draft_stride=999), INVAL),
                    (dict(draft_p=A + 2, u_accept=A, draft_stride=1000), INVAL),
                    (dict(vocab=top + 1, logits_stride=top + 1), UNSUPPORTED)):
        assert call(d) == want, d
    assert call(tree=w12.TreeC(4, A, A, A, None, A, A, A)) == INVAL
    assert call(tree=w12.TreeC(4, A, None, A, A, A, A, A)) == INVAL
    assert L.w12_tree_verify_sampled(None, C.byref(w12.TreeC(4, A, A, A, A, A, A, A)), 3, 4, A, None, A, A, None, A, nbytes,
                                     None) == INVAL


def test_binding_refuses_tensors_it_cannot_pass(w12):
    torch = pytest.importorskip("torch")
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)
    args = lambda: [z(3, 2, 64, 128), z(3, 2, 128, 64), z(3, 2, dt=torch.float32), z(3, 2, dt=torch.float32),
                    z(2, 2, dt=torch.int32), z(2, dt=torch.int32)]
    w12.KvCache(*args())
    for i, bad in ((1, z(3, 2, 64, 128)), (2, z(3, 2)), (4, z(2, 2, dt=torch.int64)), (5, z(3, dt=torch.int32)),
                   (0, z(3, 2, 128, 64).transpose(2, 3))):
        a = args()
        a[i] = bad
        with pytest.raises(ValueError):
            w12.KvCache(*a)
    with pytest.raises(ValueError):
        w12.Rope(z(4, 8, dt=torch.float32), z(4, 9, dt=torch.float32))
    with pytest.raises(ValueError):
        w12.SampleRows(z(2, 8, dt=torch.float16), z(2, dt=torch.float32))
    with pytest.raises(ValueError):
        w12.SampleRows(z(2, 8, dt=torch.float32), z(2, dt=torch.float32), draft_p=z(2, 8, dt=torch.float32))
    with pytest.raises(ValueError):
        w12.DeviceTree.from_arrays(z(3, dt=torch.int32), z(3, dt=torch.int32), z(3, dt=torch.int32), z(2, dt=torch.int32))


def test_rope_refusals(w12):
    L, n = w12.lib(), None
    A = 1 << 20
    nbytes = L.w12_workspace_bytes(1, 0, 0, 2)
    cache = w12.KvCacheC(2, 128, 64, 8, 4, A, A, A, A, A, A)

    def call(**kw):
        r = dict(rot_dim=64, adjacent=0, max_pos=100, cos=A, sin=A)
        r.update(kw)
        return L.w12_kv_append(C.byref(cache), C.byref(w12.RopeC(*r.values())), 2, A, 256, A, 256, 4, A, A, A, nbytes, n)

    for kw, want in ((dict(rot_dim=-8), INVAL), (dict(rot_dim=7), INVAL), (dict(max_pos=0), INVAL), (dict(cos=None), INVAL),
                     (dict(sin=None), INVAL), (dict(cos=A + 4), INVAL), (dict(sin=A + 8), INVAL), (dict(rot_dim=12), UNSUPPORTED),
                     (dict(rot_dim=136), UNSUPPORTED)):
        assert call(**kw) == want, kw


def test_sampling_scratch(w12):
    L = w12.lib()
    A = 1 << 20
    nbytes = L.w12_workspace_bytes(1, 0, 0, 3)
    top = L.w12_sample_max_vocab()
    assert L.w12_sample_scratch_bytes(0, 10) == L.w12_sample_scratch_bytes(513, 10) == L.w12_sample_scratch_bytes(1, 0) == 0
    assert L.w12_sample_scratch_bytes(1, top + 1) == 0
    sizes = [L.w12_sample_scratch_bytes(r, v) for r, v in ((1, 1), (2, 1), (2, 5000), (512, 5000), (512, top))]
    assert sizes == sorted(sizes) and sizes[0] > 0
    tree = w12.TreeC(4, A, A, A, A, A, A, A)
    for scratch, rows in ((None, 4), (A + 8, 4), (A, 3)):
        d = w12.SamplingC(A, 1, 1000, 1000, None, None, 0, None, A, scratch, rows)
        assert L.w12_tree_sample(C.byref(d), C.byref(tree), 3, A, None, A, nbytes, None) == WORKSPACE, (scratch, rows)
