"""Sampled verification where its weights, rejections and searches can go wrong
(marked gpu), against the 64-bit form in oracle/attention.py."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import attention as ref
from test_gpu_attention import dev_tree, make_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
U_TOP = 1 - 2.0 ** -24
STALE = -77                      # what the outputs hold before the call


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def sample(w12, z, temp, u, t=None, token=None, q=None, ua=None, p_max=3):
    """row_tok, row_logp, acc_tok, acc_len of a verification whose outputs held something else before."""
    R = len(z)
    t = t or make_tree(np.random.default_rng(0), [1] * R)
    n = len(t[3]) - 1
    ws = w12.Workspace(1, 0, 0, n)
    dist = w12.SampleRows(z, cuda(np.float32(u)), cuda(np.float32(temp)), None if q is None else cuda(q),
                          None if ua is None else cuda(np.float32(ua)))
    dist.scratch.fill_(0x5A)
    new = lambda *s, dt=torch.int32: torch.full(s, STALE, dtype=dt, device="cuda")
    row, lp, tok, length, node = new(R), new(R, dt=torch.float32), new(n, p_max + 1), new(n), new(n)
    w12.w12_tree_verify_sampled(dist, dev_tree(w12, t, token), n, p_max, ws, row, lp, tok, length, node)
    torch.cuda.synchronize()
    assert ws.status() == 0
    return row.cpu().numpy(), lp.cpu().numpy(), tok.cpu().numpy(), length.cpu().numpy()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [40, 3000, 151936])
@pytest.mark.parametrize("T", [0.5, 0.1, 1e-3, 1e-30])
def test_scaled_logits_past_the_types_range(w12, f32, V, T):
    """Logits that are numbers, over a temperature that leaves none: the largest ones share the mass."""
    dt = torch.float32 if f32 else torch.bfloat16
    big = torch.finfo(dt).max
    z = torch.full((5, V), -big, dtype=dt, device="cuda")          # 0: all the lowest value
    z[1] = big                                                     # 1: all the highest
    z[2, 7::5] = -0.9 * big                                        # 2: some a little higher, yet past the range
    z[3] = 0.0
    z[3, [3, V - 1]] = big                                         # 3: two at the top
    z[4] = -float("inf")
    z[4, V // 2:] = -big                                           # 4: the lowest value among nothing
    alike = [list(range(V)), list(range(V)), list(range(7, V, 5)), [3, V - 1], list(range(V // 2, V))]
    for u in (0.0, 0.37, 0.5, U_TOP):
        row, lp, tok, length = sample(w12, z, [T] * 5, [u] * 5)
        want = [a[int(np.float32(u) * np.float64(len(a)))] for a in alike]
        assert row.tolist() == want and tok[:, 0].tolist() == want and (length == 1).all()
        # log of a count under 2^18 in FP32
        assert np.abs(lp + [np.log(len(a)) for a in alike]).max() <= 2.0 ** -18


@pytest.mark.parametrize("V", [40, 3000, 151936])
def test_the_least_temperatures(w12, V):
    """1 / T still a number, the scaled logits not: the largest logit takes all."""
    g = np.random.default_rng(V)
    z = np.stack([g.standard_normal(V) - 20, g.standard_normal(V) + 20, g.standard_normal(V)]).astype(np.float32)
    z[:, V // 3] = z.max(1) + 1
    for u in (0.0, 0.6, U_TOP):
        row, lp, _, _ = sample(w12, cuda(z), [1e-38, 1e-38, 1e-37], [u] * 3)
        assert row.tolist() == [V // 3] * 3 and (lp == 0).all()


def test_an_infinite_temperature(w12):
    """Every logit above -inf weighs the same; infinite ones take all."""
    V = 5000
    z = torch.randn(3, V, device="cuda") * 9
    z[1, ::2] = -float("inf")
    z[2, [11, 4000]] = float("inf")
    alike = [list(range(V)), list(range(1, V, 2)), [11, 4000]]
    for u in (0.0, 0.3, 0.5, U_TOP):
        row, lp, _, _ = sample(w12, z, [np.inf] * 3, [u] * 3)
        assert row.tolist() == [a[int(np.float32(u) * np.float64(len(a)))] for a in alike]
        assert np.abs(lp + [np.log(len(a)) for a in alike]).max() <= 2.0 ** -18


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("V", [64, 4096, 65536])
def test_rejections_past_the_types_range(w12, f32, V):
    """The same rows with a drafter's probabilities: accepted, rejected into a residual, and rejected with p = q.
    V is a power of two, so p, q and the residuals are exact."""
    dt = torch.float32 if f32 else torch.bfloat16
    R = 9
    parent = np.asarray([-1, 0, 0, -1, 3, -1, 5, -1, 7], np.int32)
    t = (parent, (parent >= 0).astype(np.uint8), np.asarray([0, 0, 0, 1, 1, 2, 2, 3, 3], np.int32), np.asarray([0, 3, 5, 7, 9], np.int32))
    z = torch.full((R, V), torch.finfo(dt).min, dtype=dt, device="cuda")        # p = 1 / V everywhere
    q = np.zeros((R, V), np.float32)
    q[0, :8] = 1 / 8                 # request 0: both children rejected, twice the residual over the tokens from 8 on
    q[3, :V // 2] = 2 / V            # request 1: rejected, the residual in the upper half
    q[5] = 1 / V                     # request 2: accepted
    q[7] = 1 / V                     # request 3: u q = p is a rejection, and p = q leaves p
    token = np.asarray([1, 2, 3, 4, 5, 6, 9, 10, 11], np.int32)
    ua = np.full(R, 0.9, np.float32)
    ua[1:3], ua[8] = 0.99, 1.0
    us = np.full(R, 0.25, np.float32)
    row, lp, tok, length = sample(w12, z, [0.5] * 4, us, t, token, q, ua)
    assert row[0] == 8 + (V - 8) // 4            # equal weights over V - 8 tokens
    assert row[3] == V // 2 + V // 8 and row[5] == 9 and row[7] == V // 4
    assert length.tolist() == [1, 1, 2, 1] and tok[:, 0].tolist() == [row[0], row[3], 9, row[7]]
    assert np.abs(lp + np.log(V)).max() <= 2.0 ** -18
    rest = [i for i in range(R) if i not in (0, 3, 5, 7)]
    assert (row[rest] == V // 4).all()


# ---------------------------------------------------------------------------
# rejections over large vocabularies
# ---------------------------------------------------------------------------

def decide(p, kids, q, ua, us):
    """The token that a row must emit and by how many rejections, or (None, ..) where a roundoff may turn a decision.

    A weight is within 2^-16 of its value (an FP32 exponential of an FP32 z - max, |z - max| < 64), and so is their
    sum, but for 2^-40 a token: err, the error of p, starts at 2^-14 of each.  A rejection keeps it and divides by
    what is left, whose own error is theirs together; its own products and differences round within 2^-22."""
    err, floor = p * 2.0 ** -14, len(p) * 2.0 ** -40
    for n, x in enumerate(kids):
        a, b = float(ua[n]) * q[x], p[x]
        if abs(a - b) <= err[x] + 2.0 ** -22 * a:
            return None, n
        if a < b:
            return int(x), n
        rest = np.maximum(p - q, 0.0)
        S = rest.sum()
        if S <= 64 * (err.sum() + floor):
            return None, n
        gone = err.sum() + 2.0 ** -22 + floor
        p, err = rest / S, np.where(p + err > q, err + 2.0 ** -22 * (p + q), 0.0) / S
        err = err + p * gone / S
    cum = np.cumsum(p)
    off = err.sum() + floor + 2.0 ** -22
    lo, hi = (int(np.searchsorted(cum, (float(us) + s) * cum[-1], side="right")) for s in (-off, off))
    return (lo, len(kids)) if lo == hi and lo < len(p) else (None, len(kids))


def likely_rejected(g, rows, vocab, f32, temps, chain):
    """Rows whose mass lies on a dozen tokens, and drafts of which the drafter is much too sure."""
    t = make_tree(g, rows, chain)
    R = len(t[0])
    T = np.asarray([temps[r % len(temps)] for r in range(len(rows))], np.float32)
    z = g.standard_normal((R, vocab)).astype(np.float32)
    hot = np.stack([g.choice(vocab, 12, replace=False) for _ in range(R)])
    rowT = T[t[2]][:, None].astype(np.float64)
    np.put_along_axis(z, hot, ((np.log(vocab) + 2 + 3 * g.random((R, 12))) * rowT).astype(np.float32), 1)
    zt = cuda(z) if f32 else cuda(z).bfloat16()
    z = zt.float().cpu().numpy()
    p = np.stack([ref.target(z[i], float(rowT[i, 0])) for i in range(R)])
    lift = np.zeros((R, vocab))
    np.put_along_axis(lift, hot, g.choice([-1.5, 0.0, 1.5], (R, 12)), 1)
    q = p * np.exp(lift)
    q = (q / q.sum(1, keepdims=True)).astype(np.float32)
    token = g.integers(0, vocab, R).astype(np.int32)
    for j in range(R):
        i = t[0][j]
        if i >= 0:
            over = hot[i][np.argsort(p[i][hot[i]] / q[i][hot[i]])]         # those that q overrates most come first
            token[j] = over[min(11, int(g.integers(0, 16)) // 2)]
    ua = np.float32(0.6 + 0.4 * g.random(R)) * np.float32(U_TOP)
    us = np.minimum(g.random(R).astype(np.float32), np.float32(U_TOP))
    return t, T, zt, z, p, q, token, ua, us


REJECTIONS = [
    # rows per request, vocabulary, 32-bit logits, temperatures, chain
    ([3] * 6, 151937, True, [1.1, 1.0], False),
    ([4] * 6, 65536, False, [1.0, 0.5], False),
    ([20] * 6, 70001, True, [0.8], False),
    ([6] * 20, 140001, False, [1.0, 0.7, 1.2], False),
    ([8] * 32, 40000, True, [0.9], True),
    ([30], 10007, False, [1.0], False),
    ([7, 1, 9, 4], 333, True, [0.6, 1.0], False),
    ([16] * 4, 2048, False, [1.0], False),
]


@pytest.mark.parametrize("rows,vocab,f32,temps,chain", REJECTIONS)
def test_rejections(w12, rows, vocab, f32, temps, chain):
    g = np.random.default_rng(vocab)
    t, T, zt, z, p, q, token, ua, us = likely_rejected(g, rows, vocab, f32, temps, chain)
    row, lp, tok, length = sample(w12, zt, T, us, t, token, q, ua, p_max=33)
    parents = decided = drawn = twice = 0
    for i in range(len(row)):
        kids = [j for j in range(len(row)) if t[0][j] == i]
        want, n = decide(p[i], token[kids], q[i].astype(np.float64), ua[kids], us[i])
        if kids:
            parents += 1
            decided += want is not None
            drawn += want is not None and n == len(kids)
            twice += want is not None and n > 1
        if want is not None:
            assert row[i] == want, (i, n)
        assert abs(lp[i] - np.log(p[i][row[i]])) <= 2.0 ** -16 * (1 + np.abs(z[i]).max() / T[t[2][i]])
    # the oracle alone: most rows are decided, many of them by a draw from what a rejection left
    assert decided >= 0.8 * parents and drawn >= max(2, parents // 8) and (chain or twice >= 1), (parents, decided, drawn, twice)


def test_rejections_of_one_row_by_the_dozen(w12):
    """Every one of 40 children is rejected; what is left are always the same ten tokens of equal weight."""
    V, R = 20011, 41
    t = (np.asarray([-1] + [0] * 40, np.int32), np.asarray([0] + [1] * 40, np.uint8), np.zeros(R, np.int32), np.asarray([0, R], np.int32))
    z = np.full((R, V), -200.0, np.float32)
    z[:, 5000:5010] = 6.0
    q = np.zeros((R, V), np.float32)
    q[0, 100:140] = 1 / 40
    token = np.concatenate([[0], 100 + np.random.default_rng(3).permutation(40)]).astype(np.int32)
    row, lp, tok, length = sample(w12, cuda(z), [1.0], np.full(R, 0.45), t, token, q, np.full(R, 0.99))
    assert (row == 5004).all() and length.tolist() == [1] and tok[0].tolist() == [5004, -1, -1, -1]
    assert np.abs(lp + np.log(10)).max() <= 2.0 ** -20
