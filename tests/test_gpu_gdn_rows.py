"""The recurrent layer over prompts (w12_gdn_prefill) and single tokens
(w12_gdn_step) against the token-by-token form in 64 bits.

Tolerances.  With keys and queries of unit norm and gates and strengths in
[0, 1] no value in between exceeds B = max(||S[v]|| + |v|), and the update does not
enlarge an error.  A value comes from sums of up to 3 * 128 FP32 products, each
rounded by 2^-23 of B at most: 4.6e-5 B in the worst case for a run of 64 rows, of
which the gates here keep a few alive: 1e-4 B.  Over a whole
output the roundings' signs are independent: sqrt(384) * 2^-23 = 2.3e-6 of its
2-norm a run, 2^-17 with the runs kept alive.  The step's sums have 128 terms and it is one token:
2^-19 of both."""
from __future__ import annotations

import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

D = 128
WORST, NORM = 1e-4, 2.0 ** -17
STEP = 2.0 ** -19


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


class Case:
    """Rows of a layer with `gap` rows in front of, between and behind the requests, which hold NaN."""

    def __init__(self, w12, counts, H, Hk, seed=0, s0=True, gap=0, fused=True, alpha=None, beta=None, key=None):
        g = torch.Generator().manual_seed(seed)
        new = lambda *s: torch.randn(s, generator=g)
        self.counts, self.H, self.Hk, n = counts, H, Hk, len(counts)
        off = [gap]
        for c in counts:
            off.append(off[-1] + c)
        self.T = off[-1] + gap
        unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()
        k = unit(new(self.T, Hk, D) + 0.5 * new(Hk, D)) if key is None else key(new(self.T, Hk, D))
        self.q, self.k, self.v = unit(new(self.T, Hk, D)).bfloat16(), k.bfloat16(), new(self.T, H, D).bfloat16()
        self.alpha = torch.rand(self.T, H, generator=g) * 0.3 + 0.7 if alpha is None else alpha(self.T, H, g)
        self.beta = torch.rand(self.T, H, generator=g) if beta is None else beta(self.T, H, g)
        self.S0 = new(n, H, D, D) * 0.05 if s0 else None
        inside = torch.zeros(self.T, dtype=torch.bool)
        inside[off[0]:off[-1]] = True
        for t in (self.q, self.k, self.v, self.alpha, self.beta):
            t[~inside] = float("nan")
        self.inside, self.off = inside, np.asarray(off, np.int32)
        parts = [t.flatten(1) for t in (self.q, self.k, self.v)]
        if fused:
            row = torch.cat([torch.zeros(self.T, 8).bfloat16()] + parts, 1).cuda()   # rows of an odd multiple of 16 bytes
            w = [p.shape[1] for p in parts]
            parts = row[:, 8:].split(w, 1)
        else:
            parts = [p.cuda() for p in parts]
        self.rows = w12.GdnRows(*parts, self.alpha.cuda(), self.beta.cuda())
        self.row_off = torch.from_numpy(self.off).cuda()
        self.ws = w12.Workspace(1, 0, 0, n)

    def run(self, w12, **kw):
        S0 = self.S0.cuda() if self.S0 is not None else None
        out = torch.full((self.T, self.H, D), 7.0, device="cuda")
        got = w12.w12_gdn_prefill(self.rows, self.row_off, self.ws, S0=S0, out=out, **kw)
        torch.cuda.synchronize()
        assert self.ws.status() == 0
        return got

    def exact(self):
        bits = lambda t: t.contiguous().view(torch.int16).numpy().view(np.uint16)
        f = lambda t: None if t is None else t.numpy()
        return oracle.gdn_sequence(f(self.S0), bits(self.q), bits(self.k), bits(self.v), f(self.alpha), f(self.beta), self.off)

    def check(self, out, state, worst=WORST, norm=NORM):
        o, S, top = self.exact()
        out, state = out.cpu().double().numpy(), state.cpu().double().numpy()
        assert (out[~self.inside.numpy()] == 7.0).all()
        for r in range(len(self.counts)):
            a, b = self.off[r], self.off[r + 1]
            for got, ref in ((out[a:b].transpose(1, 0, 2), o[a:b].transpose(1, 0, 2)), (state[r], S[r])):   # [H]...
                for h in range(self.H):
                    e = got[h] - ref[h]
                    assert np.isfinite(got[h]).all()
                    if e.size and top[r, h]:
                        assert np.abs(e).max() <= worst * top[r, h], (r, h, np.abs(e).max() / top[r, h])
                    if e.size > D:
                        assert np.linalg.norm(e) <= norm * max(np.linalg.norm(ref[h]), 1e-30), (r, h)


COUNTS = [[1], [2], [63], [64], [65], [128], [129], [300], [0], [5, 0, 70, 1], [64, 64, 64], [0, 0, 33], [1] * 9, [190, 3, 64, 0, 129]]


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("H,Hk,s0", [(1, 1, True), (4, 2, False), (3, 3, True), (6, 1, True)])
def test_prompts(w12, counts, H, Hk, s0):
    c = Case(w12, counts, H, Hk, seed=len(counts) * 100 + sum(counts) + H, s0=s0, gap=3 if H == 6 else 0, fused=H != 3)
    c.check(*c.run(w12))


def test_rows_of_others_hold_nan(w12):
    """The rows in front and behind hold NaN; 37 and 64 rows of a run are theirs."""
    c = Case(w12, [27, 64, 100], 2, 1, seed=3, gap=70)
    c.check(*c.run(w12))


def test_a_request_of_nan_reaches_no_other(w12):
    """A NaN in one request's rows stays in its request and head, and reaches no run of 64 rows before its own."""
    counts, H = [100, 200, 90], 3
    c = Case(w12, counts, H, 3, seed=4)
    clean, cs = c.run(w12)
    row = 100 + 130
    c.rows.k[row, D:2 * D] = float("nan")             # head 1, the request's third run
    out, state = c.run(w12)
    bad = torch.zeros(c.T, H, dtype=torch.bool, device="cuda")
    bad[100 + 128:300, 1] = True
    assert torch.equal(out[~bad], clean[~bad]) and out[row:300, 1].isnan().all()
    keep = torch.ones(3, H, dtype=torch.bool, device="cuda")
    keep[1, 1] = False
    assert torch.equal(state[keep], cs[keep]) and state[1, 1].isnan().all()


GATES = dict(
    zero=lambda T, H, g: (torch.rand(T, H, generator=g) > 0.1).float(),                    # forgets everything now and then
    tiny=lambda T, H, g: torch.rand(T, H, generator=g).pow(40),                            # products far below the least float
    one=lambda T, H, g: torch.ones(T, H),
    fast=lambda T, H, g: torch.rand(T, H, generator=g) * 1e-3,
)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("strength", ["some", "zero", "one"])
def test_gates_and_strengths(w12, gate, strength):
    beta = dict(some=None, zero=lambda T, H, g: torch.zeros(T, H), one=lambda T, H, g: torch.ones(T, H))[strength]
    c = Case(w12, [150, 64], 2, 2, seed=5, alpha=GATES[gate], beta=beta)
    c.check(*c.run(w12))


def test_equal_keys(w12):
    """Every key of a head the same unit vector, written at full strength: only the last value is remembered."""
    c = Case(w12, [200], 2, 1, seed=6, key=lambda x: torch.nn.functional.one_hot(torch.full(x.shape[:2], 5), D).float(),
             alpha=GATES["one"], beta=lambda T, H, g: torch.ones(T, H))
    out, state = c.run(w12)
    c.check(out, state)
    assert torch.allclose(state[0, :, :, 5], c.v[-1].cuda().float(), atol=1e-5)


def test_values_of_any_size(w12):
    """Values and states of 2^60 and 2^-60: three BF16 pieces have the range of FP32."""
    for e in (60, -60):
        c = Case(w12, [130], 2, 2, seed=7)
        c.v, c.S0 = (c.v.float() * 2.0 ** e).bfloat16(), c.S0 * 2.0 ** e
        c.rows.v.copy_(c.v.reshape(c.T, -1))
        c.check(*c.run(w12))


def test_in_place_and_split_anywhere(w12):
    """A prompt taken in two parts, the second in place, ends like the whole one."""
    c = Case(w12, [170], 4, 2, seed=8)
    o, S, top = c.exact()
    for cut in (1, 63, 64, 100, 169):
        out = torch.empty(170, 4, D, device="cuda")
        state = c.S0.cuda()
        for part in ((0, cut), (cut, 170)):
            off = torch.tensor(part, dtype=torch.int32, device="cuda")
            w12.w12_gdn_prefill(c.rows, off, c.ws, S0=state, state=state, out=out)
        torch.cuda.synchronize()
        assert c.ws.status() == 0
        assert np.abs(out.cpu().double().numpy() - o).max() <= WORST * top.max()
        assert np.abs(state.cpu().double().numpy() - S).max() <= WORST * top.max()


def test_a_request_does_not_depend_on_its_batch(w12):
    c = Case(w12, [70, 129, 5], 2, 2, seed=9)
    out, state = c.run(w12)
    again, state2 = c.run(w12)
    assert torch.equal(out, again) and torch.equal(state, state2)
    off = torch.tensor([70, 199], dtype=torch.int32, device="cuda")
    alone, s1 = w12.w12_gdn_prefill(c.rows, off, c.ws, S0=c.S0[1:2].cuda().contiguous())
    assert torch.equal(alone[70:199], out[70:199]) and torch.equal(s1[0], state[1])


def test_offsets_that_make_no_sense(w12):
    """Descending offsets, or ones outside the rows: that request is left as it was, the others are served."""
    c = Case(w12, [10, 20, 30, 40], 2, 2, seed=10)
    good, gs = c.run(w12)
    S0 = c.S0.cuda()
    for off, bad in (([0, 10, 5, 60, 100], (1,)), ([-1, 10, 30, 60, 100], (0,)), ([0, 10, 30, 60, 101], (3,))):
        out, state = torch.full_like(good, 7.0), torch.full_like(S0, 9.0)
        w12.w12_gdn_prefill(c.rows, torch.tensor(off, dtype=torch.int32, device="cuda"), c.ws, S0=S0, state=state, out=out)
        torch.cuda.synchronize()
        assert c.ws.status() == w12.W12_E_INVAL
        for r in range(4):
            if r in bad:
                assert (state[r] == 9.0).all()
            elif (off[r], off[r + 1]) == (c.off[r], c.off[r + 1]):
                end = min(off[r + 1], off[2])              # (rows that another request's offsets take in as well are anyone's)
                assert torch.equal(state[r], gs[r]) and (r >= 2 or torch.equal(out[off[r]:end], good[off[r]:end]))
                assert r < 2 or torch.equal(out[off[r]:off[r + 1]], good[off[r]:off[r + 1]])
    out, state = c.run(w12)
    assert torch.equal(out, good) and torch.equal(state, gs)


def test_no_rows_at_all(w12):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    rows = w12.GdnRows(z(0, 2 * D), z(0, 2 * D), z(0, 4 * D), torch.zeros(0, 4, device="cuda"), torch.zeros(0, 4, device="cuda"))
    ws = w12.Workspace(1, 0, 0, 2)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    S0 = torch.randn(2, 4, D, D, device="cuda")
    out, state = w12.w12_gdn_prefill(rows, off, ws, S0=S0)
    _, zero = w12.w12_gdn_prefill(rows, off, ws)
    out1, none = w12.w12_gdn_step(rows)
    torch.cuda.synchronize()
    assert ws.status() == 0
    assert torch.equal(state, S0) and out.shape == (0, 4, D) and not zero.any() and none.shape[0] == 0 and out1.shape[0] == 0


def test_a_wait_that_runs_out(w12):
    """CTA (0, 0) never copies its first rows (test hook): every role gives up, the state is left alone, and the same
    call without the hook is right."""
    c = Case(w12, [150, 40], 2, 2, seed=11)
    S0 = c.S0.cuda()
    w12.debug_set(1, 50_000_000)
    try:
        state = torch.full_like(S0, 9.0)
        w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=S0, state=state)
        torch.cuda.synchronize()
        assert c.ws.status() == w12.W12_E_TIMEOUT
        assert (state[0, 0] == 9.0).all() and not (state[0, 1] == 9.0).any()
    finally:
        w12.debug_set(0, 0)
    c.check(*c.run(w12))


def test_captured_and_on_another_stream(w12):
    c = Case(w12, [100, 64], 2, 1, seed=12)
    want, ws_ = c.run(w12)
    S0 = c.S0.cuda()
    out, state = torch.zeros_like(want), torch.zeros_like(S0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=S0, state=state, out=out)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(state, ws_)
    out.zero_()
    state.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=S0, state=state, out=out)
    assert not out.any()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(state, ws_)


def test_rows_far_apart(w12):
    """Row strides that put the last rows beyond 2^31 elements."""
    T, stride = 150, 1 << 24
    c = Case(w12, [T], 2, 1, seed=13, fused=False)
    big = torch.empty((T - 1) * stride + 1024, dtype=torch.bfloat16, device="cuda")
    views = [big[at:].as_strided((T, t.shape[1]), (stride, 1)) for at, t in ((0, c.rows.q), (128, c.rows.k), (512, c.rows.v))]
    for view, t in zip(views, (c.rows.q, c.rows.k, c.rows.v)):
        view.copy_(t)
    c.rows = w12.GdnRows(*views, c.rows.alpha, c.rows.beta)
    c.check(*c.run(w12))


# ---------------------------------------------------------------------------
# single tokens
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n,H,Hk,s0", [(1, 1, 1, True), (1, 32, 16, True), (3, 4, 2, False), (7, 6, 1, True), (40, 3, 3, True)])
def test_steps(w12, n, H, Hk, s0):
    c = Case(w12, [1] * n, H, Hk, seed=20 + n, s0=s0, fused=H != 3)
    S0 = c.S0.cuda() if s0 else None
    out, state = w12.w12_gdn_step(c.rows, S0=S0)
    c.check(out, state, STEP, STEP)
    if s0:
        o2, s2 = w12.w12_gdn_step(c.rows, S0=S0, state=S0)     # in place
        assert s2 is S0 and torch.equal(o2, out) and torch.equal(s2, state)
    # the prompt's kernel on the same rows
    o3, s3 = c.run(w12)
    c.check(o3, s3)


def test_a_gate_of_zero_in_a_step(w12):
    c = Case(w12, [1] * 4, 2, 2, seed=31, alpha=lambda T, H, g: torch.zeros(T, H))
    out, state = w12.w12_gdn_step(c.rows, S0=c.S0.cuda())
    c.check(out, state, STEP, STEP)


def test_prompt_then_steps_then_tree(w12):
    """A prompt, three single tokens and a drafted chain (w12_gdn_tree_verify, w12_gdn_commit) in a row, captured as one
    graph, against one pass over all tokens in 64 bits."""
    H, P, K = 2, 90, 5
    c = Case(w12, [P + 3 + K] * 2, H, H, seed=32, fused=False)
    n = P + 3 + K
    i32 = lambda a, dt=torch.int32: torch.tensor(a, dtype=dt, device="cuda")
    pick = lambda idx: w12.GdnRows(*(t[idx].contiguous() for t in (c.rows.q, c.rows.k, c.rows.v, c.rows.alpha, c.rows.beta)))
    prompt = pick(torch.cat([torch.arange(P), n + torch.arange(P)]))
    steps = [pick(torch.tensor([P + i, n + P + i])) for i in range(3)]
    idx = torch.cat([torch.arange(P + 3, n), n + torch.arange(P + 3, n)])
    tree = w12.DeviceTree.from_arrays(i32([-1, 0, 1, 2, 3, -1, 5, 6, 7, 8]), i32([0, 1, 2, 3, 4] * 2, torch.uint8), i32([0] * 5 + [1] * 5),
                                      i32([0, 5, 10]))
    ws = w12.Workspace(1, 0, 0, 2)
    off, node = i32([0, P, 2 * P]), i32([4, 9])
    S0, state, final = c.S0.cuda(), torch.empty(2, H, D, D, device="cuda"), torch.empty(2, H, D, D, device="cuda")
    layer = w12.GdnLayer(state, *(t[idx].reshape(-1, H, D).contiguous() for t in (c.rows.q, c.rows.k, c.rows.v)),
                         c.rows.alpha[idx].contiguous(), c.rows.beta[idx].contiguous())
    outs = [torch.empty(2 * P, H, D, device="cuda")] + [torch.empty(2, H, D, device="cuda") for _ in range(3)]
    o_tree = torch.empty(10, H, D, device="cuda")

    def loop():
        w12.w12_gdn_prefill(prompt, off, ws, S0=S0, state=state, out=outs[0])
        for s, o in zip(steps, outs[1:]):
            w12.w12_gdn_step(s, S0=state, state=state, out=o)
        w12.w12_gdn_tree_verify(layer, tree, 2, ws, out=o_tree)
        w12.w12_gdn_commit(layer, tree, 2, node, ws, state=final)

    loop()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop()
    final.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert ws.status() == 0
    got = torch.empty(2 * n, H, D)
    for r in range(2):
        got[r * n:r * n + P] = outs[0][r * P:(r + 1) * P].cpu()
        for i in range(3):
            got[r * n + P + i] = outs[1 + i][r].cpu()
        got[r * n + P + 3:(r + 1) * n] = o_tree[r * 5:(r + 1) * 5].cpu()
    c.check(got, final)
