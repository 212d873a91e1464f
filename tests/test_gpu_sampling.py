"""GPU parity of the sampled verification through the C ABI (marked gpu).

Tokens are compared with the 64-bit form in oracle/attention.py; a decision
that lies within eps of its boundary may go either way there.  eps: the
kernel's weights are FP32 exponentials of FP32 z - max, |z - max| < 64 for any
weight that counts (2^-40 of the largest), so each is within 2^-23 (64 + 3) <
2^-16 of its value, and the sums add no error."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from oracle import attention as ref
from test_gpu_attention import dev_tree, make_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
EPS = 2.0 ** -16


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


def draw(g, rows, vocab, draft, chain=False, f32=True, hot=8.0):
    t = make_tree(g, rows, chain)
    R = len(t[0])
    z = g.standard_normal((R, vocab)).astype(np.float32) * 2
    for i in range(R):
        z[i, g.integers(0, vocab, 5)] += hot
    zt = torch.from_numpy(z).cuda()
    if not f32:
        zt = zt.bfloat16()
    z = zt.float().cpu().numpy()
    e = np.exp(z - z.max(1, keepdims=True) + 0.7 * g.standard_normal(z.shape))
    q = (e / e.sum(1, keepdims=True)).astype(np.float32)
    token = g.integers(0, vocab, R).astype(np.int32)
    for j in range(R):
        p = t[0][j]
        if p >= 0:
            token[j] = g.choice(vocab, p=q[p].astype(np.float64) / q[p].sum(dtype=np.float64)) if draft else \
                np.argsort(-z[p], kind="stable")[int(np.sum(t[0][:j] == p)) % vocab]
    u = g.random((2, R)).astype(np.float32)
    return t, z, zt, q, token, np.minimum(u, np.float32(1 - 2.0 ** -24))


def check(w12, t, z, zt, q, token, u, temp, p_max=40):
    R, n_req = len(t[0]), len(t[3]) - 1
    c = lambda a: None if a is None else torch.from_numpy(a).cuda()
    tree = dev_tree(w12, t, token)
    ws = w12.Workspace(1, 0, 0, n_req)
    dist = w12.SampleRows(zt, c(u[1]), c(temp), c(q), c(u[0]) if q is not None else None)
    row_tok = torch.empty(R, dtype=torch.int32, device="cuda")
    logp = torch.empty(R, dtype=torch.float32, device="cuda")
    tok, length, node = w12.w12_tree_verify_sampled(dist, tree, n_req, 33, ws, row_tok, logp)
    only = w12.w12_tree_sample(dist, tree, n_req, ws)
    torch.cuda.synchronize()
    assert ws.status() == 0
    got, lp = row_tok.cpu().numpy(), logp.cpu().numpy()
    assert np.array_equal(only.cpu().numpy(), got)
    undecided = 0
    for i in range(R):
        T = 1.0 if temp is None else float(temp[t[2][i]])
        p = ref.target(z[i], T)
        kids = [j for j in range(R) if t[0][j] == i]
        may = ref.sample_row(p, token[kids], None if q is None else q[i].astype(np.float64), u[0][kids], u[1][i], EPS)
        if may is None or len(may) > 1:
            undecided += 1
        assert may is None or int(got[i]) in may, i
        if T > 0:
            zi = z[i].astype(np.float64) / T
            want = zi[got[i]] - zi.max() - np.log(np.exp(zi - zi.max()).sum())
            assert abs(lp[i] - want) <= 2.0 ** -18 * (1 + abs(want) + np.abs(zi).max())
        else:
            assert lp[i] == 0
    want_tok, want_len, want_node = oracle.tree_accept(
        _as_tree(t, token), got, n_req, 33)
    assert np.array_equal(length.cpu().numpy(), want_len) and np.array_equal(node.cpu().numpy(), want_node)
    assert np.array_equal(tok.cpu().numpy(), want_tok)
    return undecided


def _as_tree(t, token):
    R = len(t[0])
    return oracle.Tree(R=R, parent=t[0], token=token, depth=t[1], req=t[2], score=np.zeros(R, np.float32),
                       rank=np.zeros(R, np.uint8), req_row_off=t[3])


CASES = [
    # rows per request, vocabulary, draft probabilities, chain, 32-bit logits, temperatures
    ([1], 1, False, True, True, None),
    ([1], 5, False, True, False, [0.7]),
    ([4], 33, False, False, True, [1.0]),
    ([6, 1, 3], 1000, False, False, False, [0.8, 0.0, 1.3]),
    ([5, 4], 2049, True, False, True, [0.9, 1.0]),
    ([12], 4096, True, False, True, None),
    ([20, 7], 10007, True, True, True, [0.6, 0.0]),
    ([3, 3], 65536, True, False, False, [1.0, 0.5]),
    ([2, 2], 151936, False, False, False, [0.7, 1.0]),
    ([3], 151937, True, False, True, [1.1]),
]


@pytest.mark.parametrize("rows,vocab,draft,chain,f32,temp", CASES)
def test_sampled_verification(w12, rows, vocab, draft, chain, f32, temp):
    g = np.random.default_rng(vocab)
    t, z, zt, q, token, u = draw(g, rows, vocab, draft, chain, f32)
    temp = None if temp is None else np.asarray(temp, np.float32)
    undecided = check(w12, t, z, zt, q if draft else None, token, u, temp)
    if 4 * EPS * vocab < 1:              # a token's mean share is over the boundaries' uncertainty: most rows are decided
        assert undecided <= 1 + len(t[0]) // 4


# rows and vocabularies that give a thread 2, 4, 8 and 16 pieces of a row
MANY = [([45], 60000, False, False, True, None), ([20] * 6, 70001, True, False, True, None),
        ([10] * 24, 151936, False, False, False, None), ([1] * 260, 151936, False, True, True, None),
        ([6] * 20, 140001, True, False, False, None)]


@pytest.mark.parametrize("rows,vocab,draft,chain,f32,temp", MANY)
def test_sampled_verification_of_many_rows(w12, rows, vocab, draft, chain, f32, temp):
    g = np.random.default_rng(vocab + 1)
    t, z, zt, q, token, u = draw(g, rows, vocab, draft, chain, f32)
    check(w12, t, z, zt, q if draft else None, token, u, temp)


def test_exact_boundaries(w12):
    """Equal logits: every weight is 2^40, so token floor(u V) is the answer without any rounding."""
    for V in (4, 1000, 4096, 150000):
        R = 64
        u = np.concatenate([np.arange(32) / 32.0, [0.0, 1 - 2.0 ** -24], np.random.default_rng(1).random(30)]).astype(np.float32)
        u = np.minimum(u, np.float32(1 - 2.0 ** -24))
        t = make_tree(np.random.default_rng(0), [1] * R)
        dist = w12.SampleRows(torch.zeros(R, V, device="cuda"), torch.from_numpy(u).cuda())
        tok = w12.w12_tree_sample(dist, dev_tree(w12, t), R, w12.Workspace(1, 0, 0, R))
        assert tok.cpu().tolist() == [int(x) for x in np.floor(u.astype(np.float64) * V)]


def test_a_row_does_not_depend_on_its_batch(w12):
    g = np.random.default_rng(5)
    t, z, zt, q, token, u = draw(g, [40], 30001, False, False, True)
    c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    ws = w12.Workspace(1, 0, 0, 1)
    full = w12.w12_tree_sample(w12.SampleRows(zt, c(u[1])), dev_tree(w12, t), 1, ws)
    one = make_tree(g, [1])
    for i in (0, 7, 39):
        wide = torch.empty(1, 30001 + 3, device="cuda")
        wide[:, 3:] = zt[i]                                  # another alignment and stride
        got = w12.w12_tree_sample(w12.SampleRows(wide[:, 3:], c(u[1][i:i + 1])), dev_tree(w12, one), 1, ws)
        assert int(got) == int(full[i])


def test_masked_logits(w12):
    """-inf, NaN and the type's lowest value never win; a row without anything gives -1; +inf takes all."""
    V = 3000
    z = torch.full((5, V), -float("inf"), device="cuda")
    z[0, 17] = 2.0
    z[1, 100:200] = float("nan")
    z[2, :] = torch.finfo(torch.float32).min
    z[2, 2999] = 1.0
    z[3, :] = 0.0
    z[3, 5] = float("inf")
    z[4, :] = torch.finfo(torch.float32).min                 # nothing but the lowest value: all equal
    t = make_tree(np.random.default_rng(0), [1] * 5)
    ws = w12.Workspace(1, 0, 0, 5)
    lp = torch.empty(5, device="cuda")
    for u in (0.0, 0.5, 1 - 2.0 ** -24):
        us = torch.full((5,), u, device="cuda")
        tok = w12.w12_tree_sample(w12.SampleRows(z, us), dev_tree(w12, t), 5, ws, row_logp=lp)
        assert tok.cpu().tolist() == [17, -1, 2999, 5, int(u * V)]
        assert lp.cpu().tolist()[1] == -float("inf") and lp.cpu().tolist()[0] == 0.0
    acc = w12.w12_tree_verify_sampled(w12.SampleRows(z, us), dev_tree(w12, t), 5, 2, ws)
    assert acc[1].cpu().tolist() == [1] * 5 and acc[0][:, 0].cpu().tolist() == tok.cpu().tolist()
    assert ws.status() == 0


def test_draft_equal_to_the_target_is_always_accepted(w12):
    g = np.random.default_rng(9)
    t, z, zt, q, token, u = draw(g, [17], 500, True, True)
    e = np.exp((z - z.max(1, keepdims=True)).astype(np.float64))
    q = (e / e.sum(1, keepdims=True) * (1 - 2.0 ** -12)).astype(np.float32)     # below p by more than the roundings
    for j in range(1, 17):
        token[j] = int(np.argmax(q[t[0][j]]))
    c = lambda a: torch.from_numpy(a).cuda()
    dist = w12.SampleRows(zt, c(u[1]), None, c(q), c(u[0]))
    tok, length, node = w12.w12_tree_verify_sampled(dist, dev_tree(w12, t, token), 1, 16, w12.Workspace(1, 0, 0, 1))
    assert int(length) == 17 and int(node) == 16 and tok[0, :16].cpu().tolist() == token[1:].tolist()


def test_rejected_everywhere_draws_from_the_residual(w12):
    """p and q have no token in common: every draft is rejected, and the token comes from p."""
    V, R = 640, 5
    t = make_tree(np.random.default_rng(0), [R])
    t[0][1:] = 0                                             # four children of the root
    t[1][1:] = 1
    z = torch.full((R, V), -30.0, device="cuda")
    z[:, 300:310] = 0.0
    q = torch.zeros(R, V, device="cuda")
    q[:, 5:9] = 0.25
    token = np.asarray([0, 5, 6, 5, 8], np.int32)
    us = torch.full((R,), 0.55, device="cuda")
    dist = w12.SampleRows(z, us, None, q, torch.full((R,), 0.01, device="cuda"))
    ws = w12.Workspace(1, 0, 0, 1)
    tok, length, node = w12.w12_tree_verify_sampled(dist, dev_tree(w12, t, token), 1, 4, ws)
    assert int(length) == 1 and int(node) == 0 and int(tok[0, 0]) == 305
