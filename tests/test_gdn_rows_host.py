"""Host tests of the recurrent layer over rows and of the norms: the 64-bit form against the tree's, and the refusals of the
entry points (every bad argument is turned away before any launch, so no GPU is needed)."""
from __future__ import annotations

import ctypes as C

import numpy as np
import pytest

import oracle
from speculative_decoding_tree_w12_gb300 import synth


def test_a_sequence_is_a_chain():
    """gdn_sequence on one request's rows is gdn_tree_path and gdn_commit on a chain of them."""
    R, H = 9, 2
    x = synth.gdn_inputs(R, 1, H, 128, seed=3)
    t = oracle.Tree(R=R, parent=np.arange(-1, R - 1, dtype=np.int32), token=np.zeros(R, np.int32), depth=np.arange(R, dtype=np.uint8),
                    req=np.zeros(R, np.int32), score=np.zeros(R, np.float32), rank=np.zeros(R, np.uint8),
                    req_row_off=np.asarray([0, R], np.int32))
    o, S, top = oracle.gdn_sequence(x.S0, x.q, x.k, x.v, x.alpha, x.beta, t.req_row_off)
    assert np.allclose(o, oracle.gdn_tree_path(x.S0, x.q, x.k, x.v, x.alpha, x.beta, t), rtol=0, atol=1e-12)
    assert np.allclose(S, oracle.gdn_commit(x.S0, x.k, x.v, x.alpha, x.beta, t, np.asarray([R - 1])), rtol=0, atol=1e-12)
    assert (top[0] >= np.sqrt((S[0] ** 2).sum(-1)).max(-1)).all()


def test_shared_heads_and_requests():
    """Value heads of one key head see the same keys; requests do not see one another; empty ones keep their state."""
    x = synth.gdn_inputs(10, 3, 4, 128, seed=4)
    q, k = x.q[:, :2], x.k[:, :2]
    o, S, _ = oracle.gdn_sequence(x.S0, q, k, x.v, x.alpha, x.beta, [0, 6, 6, 10])
    o1, S1, _ = oracle.gdn_sequence(x.S0[2:], q[6:], k[6:], x.v[6:], x.alpha[6:], x.beta[6:], [0, 4])
    assert np.array_equal(o[6:], o1) and np.array_equal(S[2], S1[0]) and np.array_equal(S[1], x.S0[1].astype(np.float64))
    full = [np.repeat(t, 2, 1) for t in (q, k)]
    assert np.array_equal(oracle.gdn_sequence(x.S0, *full, x.v, x.alpha, x.beta, [0, 6, 6, 10])[0], o)


def test_a_unit_key_at_full_strength_stores_its_value():
    one = np.zeros((1, 1, 128), np.uint16)
    one[0, 0, 7] = 0x3F80
    v = synth.f32_to_bf16_bits(np.arange(128, dtype=np.float32).reshape(1, 1, 128))
    o, S, _ = oracle.gdn_sequence(np.ones((1, 1, 128, 128), np.float32), one, one, v, np.ones((1, 1)), np.ones((1, 1)), [0, 1])
    assert np.array_equal(o[0, 0], np.arange(128)) and np.array_equal(S[0, 0, :, 7], np.arange(128)) and (S[0, 0, :, 6] == 1).all()


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


def rows(w12, **kw):
    f = dict(n_heads=4, n_qk_heads=2, head_dim=128, n_rows=10, q=A, k=A, v=A, q_stride=256, k_stride=256, v_stride=512, alpha=A, beta=A,
             scratch=0, scratch_bytes=0)
    f.update(kw)
    return w12.GdnRowsC(*(f[n] for n, _ in w12.GdnRowsC._fields_))


BAD_ROWS = [
    (dict(n_heads=0), INVAL), (dict(n_qk_heads=0), INVAL), (dict(n_rows=-1), INVAL), (dict(head_dim=64), UNSUPPORTED),
    (dict(n_qk_heads=3), UNSUPPORTED), (dict(n_heads=65536, v_stride=65536 * 128), UNSUPPORTED), (dict(q=0), INVAL), (dict(k=0), INVAL),
    (dict(v=0), INVAL), (dict(alpha=0), INVAL), (dict(beta=0), INVAL), (dict(q=A + 8), INVAL), (dict(k=A + 2), INVAL), (dict(v=A + 8), INVAL),
    (dict(alpha=A + 2), INVAL), (dict(q_stride=248), INVAL), (dict(k_stride=260), INVAL), (dict(v_stride=504), INVAL),
    (dict(v_stride=1 << 38), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", BAD_ROWS, ids=str)
def test_rows_refused(w12, kw, want):
    r = rows(w12, **kw)
    big = C.c_size_t(1 << 30)
    assert w12.lib().w12_gdn_prefill(C.byref(r), 2, A, A, A, A, A, big, None) == want
    assert w12.lib().w12_gdn_step(C.byref(r), A, A, A, None) == want


def test_prefill_refused(w12):
    r, big = rows(w12), C.c_size_t(1 << 30)
    call = lambda n=2, off=A, S0=A, state=A, o=A, ws=A, nb=big, rr=C.byref(r): w12.lib().w12_gdn_prefill(rr, n, off, S0, state, o, ws, nb, None)
    for kw, want in ((dict(n=0), INVAL), (dict(n=513), UNSUPPORTED), (dict(off=None), INVAL), (dict(state=None), INVAL), (dict(o=None), INVAL),
                     (dict(S0=A + 8), INVAL), (dict(S0=A + 16), INVAL), (dict(state=A + 4), INVAL), (dict(state=A + 16), INVAL), (dict(o=A + 4), INVAL), (dict(ws=None), WORKSPACE),
                     (dict(ws=A + 16), WORKSPACE), (dict(nb=C.c_size_t(64)), WORKSPACE), (dict(rr=None), INVAL)):
        assert call(**kw) == want, kw


def test_scratch_refused(w12):
    """Scratch is checked where one is given: its alignment, and its size where a call of such rows would use it."""
    L, big = w12.lib(), C.c_size_t(1 << 30)
    call = lambda **kw: L.w12_gdn_prefill(C.byref(rows(w12, **kw)), 1, A, A, A, A, A, big, None)
    need = L.w12_gdn_scratch_bytes(4, 5000)
    assert need > 0 and L.w12_gdn_scratch_bytes(4, 100) == 0
    assert L.w12_gdn_scratch_bytes(0, 5000) == 0 and L.w12_gdn_scratch_bytes(4, 0) == 0 and L.w12_gdn_scratch_bytes(65536, 5000) == 0
    assert call(n_rows=5000, scratch=A + 16, scratch_bytes=need) == INVAL
    assert call(n_rows=5000, scratch=A, scratch_bytes=need - 1) == WORKSPACE
    assert call(n_rows=5000, scratch=A, scratch_bytes=0) == WORKSPACE


def test_step_refused(w12):
    step = w12.lib().w12_gdn_step
    assert step(None, A, A, A, None) == INVAL
    assert step(C.byref(rows(w12)), A, None, A, None) == INVAL
    assert step(C.byref(rows(w12)), A, A, None, None) == INVAL
    assert step(C.byref(rows(w12, n_rows=65536)), A, A, A, None) == UNSUPPORTED
    assert step(C.byref(rows(w12, n_rows=0, q=0, k=0, v=0, alpha=0, beta=0)), None, None, None, None) == 0


def test_gdn_norm_refused(w12):
    f = w12.lib().w12_gdn_norm
    call = lambda o=A, R=3, H=2, d=128, z=A, zs=256, w=A, eps=1e-6, x=A + 4096, xs=256: f(o, R, H, d, z, zs, w, eps, 0, x, xs, None)
    for kw, want in ((dict(o=None), INVAL), (dict(o=A + 8), INVAL), (dict(R=-1), INVAL), (dict(H=0), INVAL), (dict(d=64), UNSUPPORTED),
                     (dict(R=1 << 30, H=4, zs=512, xs=512), UNSUPPORTED), (dict(z=A + 8), INVAL), (dict(zs=248), INVAL), (dict(zs=260), INVAL),
                     (dict(w=None), INVAL), (dict(w=A + 4), INVAL), (dict(eps=0.0), INVAL), (dict(eps=float("nan")), INVAL),
                     (dict(eps=float("inf")), INVAL), (dict(x=None), INVAL), (dict(x=A + 8), INVAL), (dict(xs=128), INVAL),
                     (dict(x=A, zs=264), INVAL), (dict(o=A + 4096), INVAL)):
        assert call(**kw) == want, kw
    assert call(R=0, o=None, x=None) == 0


def test_block_norm_refused(w12):
    def call(**kw):
        f = dict(n_rows=3, h_f32=0, n=256, h=A, h_stride=256, h_out=2 * A, h_out_stride=256, y=3 * A, y_stride=256, post=4 * A, scale=1.0,
                 pre=5 * A, eps=1e-6, x=6 * A, x_stride=256)
        f.update(kw)
        return w12.lib().w12_block_norm(C.byref(w12.ResidualC(*(f[n] for n, _ in w12.ResidualC._fields_))), None)

    for kw, want in ((dict(n_rows=-1), INVAL), (dict(n=0), INVAL), (dict(n=252), UNSUPPORTED), (dict(n=16392), UNSUPPORTED), (dict(h=None), INVAL),
                     (dict(h=A + 8), INVAL), (dict(h_stride=248), INVAL), (dict(h_stride=260), INVAL), (dict(h_f32=1, h_stride=258), INVAL),
                     (dict(h_out=None), INVAL), (dict(h_out=A + 2), INVAL), (dict(h_out_stride=0), INVAL), (dict(h_out=A, h_out_stride=264), INVAL),
                     (dict(y=A + 2), INVAL), (dict(y_stride=128), INVAL), (dict(post=A + 2), INVAL), (dict(pre=A + 2), INVAL), (dict(x=None), INVAL),
                     (dict(x=A + 2), INVAL), (dict(x_stride=250), INVAL), (dict(x=3 * A, x_stride=264), INVAL), (dict(x=A), INVAL),
                     (dict(x=2 * A), INVAL), (dict(y=2 * A), INVAL), (dict(eps=0.0), INVAL), (dict(scale=float("nan")), INVAL), (dict(scale=float("inf")), INVAL),
                     (dict(y=None, pre=None, post=None), INVAL), (dict(y=None), INVAL)):
        assert call(**kw) == want, kw
    assert call(n_rows=0) == 0
    assert w12.lib().w12_block_norm(None, None) == INVAL


def test_residual_bytes(w12):
    """The binding's packed arguments are the C structure's bytes."""
    values = (3, 1, 256, A, 264, 2 * A, 272, 3 * A, 280, 4 * A, 0.5, 5 * A, 1e-6, 6 * A, 288)
    packed = w12._residual(*values)
    assert len(packed) == C.sizeof(w12.ResidualC)
    r = w12.ResidualC.from_buffer_copy(packed)
    for (name, _), v in zip(w12.ResidualC._fields_, values):
        assert getattr(r, name) == (pytest.approx(v) if isinstance(v, float) else v), name


def test_binding_turns_host_and_misshapen_tensors_away(w12):
    torch = pytest.importorskip("torch")
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    f = lambda *s: torch.zeros(s)
    good = (b(3, 256), b(3, 256), b(3, 512), f(3, 4), f(3, 4))
    layer = w12.GdnRows(*good)
    for i, t in ((0, b(3, 200)), (0, b(3, 384)), (0, b(2, 256)), (0, f(3, 256)), (1, b(3, 512)), (2, b(3, 256)), (2, b(512, 3).T), (3, f(3, 8)[:, :4]),
                 (4, f(3, 2)), (3, b(3, 4))):
        with pytest.raises(ValueError):
            w12.GdnRows(*good[:i], t, *good[i + 1:])
    off = torch.zeros(2, dtype=torch.int32)
    for offsets in (off, off[:1], off[:0]):
        with pytest.raises(ValueError):
            w12.w12_gdn_prefill(layer, offsets, None)
    with pytest.raises(ValueError):
        w12.w12_gdn_step(layer)
    with pytest.raises(ValueError):
        w12.w12_gdn_norm(f(2, 2, 128), b(128))
    with pytest.raises(ValueError):
        w12.w12_block_norm(b(2, 64), b(2, 64), pre=b(64))
