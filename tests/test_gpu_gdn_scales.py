"""w12_gdn_prefill where a run of 64 rows holds values of very different sizes: gates above 1, values and states that a gate makes
the layer forget, single rows far larger than the ones in front of them.  Every row's output is held against what that row
can be made of, so a row's accuracy may not depend on larger ones behind it or on what has been forgotten.

Tolerances.  With S the state in front of a run, the rows' outputs are sums (in the notation of the layer's chunked form)
    x_i = b_i (v_i - G_i S k_i),   u = M x,   o_i = G_i S q_i + sum over j <= i of A_ij u_j,
and SIZE_i is the same sum with every summand's magnitude in its place (2-norms over a head's 128 values; M's own error goes by
|M| (1 + |L|) |M|).  A summand passes through at most the sums of S k or S q (24 products), of u (18) and of A u (18), each of
which rounds by 2^-23 of the sum at most, the products that are left out (2^-21 of a summand, twice) and the 30 or so
roundings that make L, M and the gates' products: fewer than 128 roundings of 2^-23, or 2^-16 of SIZE_i.  The state is one more
such sum.  The next run's SIZE starts from the larger of the state's norm and its SIZE.  Where a request is cut into parts, the state
in front of one comes by way of P and Q, which are runs themselves, and their join: twice that."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from test_gpu_gdn_rows import Case, D

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOL = 2.0 ** -16


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


def sizes(S0, q, k, v, a, b):
    """(SIZE of every row's output, of the state behind the last one) of one head, in 64 bits; runs of 64 rows."""
    state, out, S = np.linalg.norm(S0), [], S0.copy()
    for r in range(0, len(a), 64):
        q_, k_, v_, a_, b_ = (t[r:r + 64] for t in (q, k, v, a, b))
        n = len(a_)
        Dij = np.eye(n)
        for i in range(1, n):
            Dij[i, :i] = Dij[i - 1, :i] * abs(a_[i])
        G = np.cumprod(np.abs(a_))
        L = np.tril(np.abs(b_)[:, None] * Dij * np.abs(k_ @ k_.T), -1)
        # (signed: M's entries are products, not sums of magnitudes)
        sign = np.eye(n)
        for i in range(1, n):
            sign[i, :i] = sign[i - 1, :i] * a_[i]
        M = np.abs(np.linalg.inv(np.eye(n) + np.tril(b_[:, None] * sign * (k_ @ k_.T), -1)))
        kn, qn = np.linalg.norm(k_, axis=1), np.linalg.norm(q_, axis=1)
        x = np.abs(b_) * (np.linalg.norm(v_, axis=1) + G * state * kn)
        u = M @ (np.eye(n) + L) @ M @ x
        out.append(G * state * qn + np.tril(Dij * np.abs(q_ @ k_.T)) @ u)
        for i in range(n):
            w = b_[i] * (v_[i] - a_[i] * (S @ k_[i]))
            S = a_[i] * S + np.outer(w, k_[i])
        state = max(np.linalg.norm(S), G[-1] * state + (Dij[-1] * kn) @ u)
    return np.concatenate(out), state


def run(w12, c, tol):
    """The case's rows as they are now, and every row and state of every head within `tol` of its size."""
    c.rows = w12.GdnRows(*(t.reshape(c.T, -1).cuda() for t in (c.q, c.k, c.v)), c.alpha.cuda(), c.beta.cuda())
    out, state = (t.cpu().double().numpy() for t in c.run(w12))
    o, S, _ = c.exact()
    f = lambda t: t.double().numpy()
    worst = 0.0
    for h in range(c.H):
        kh = h // (c.H // c.Hk)
        size, last = sizes(f(c.S0)[0, h], f(c.q)[:, kh], f(c.k)[:, kh], f(c.v)[:, h], f(c.alpha)[:, h], f(c.beta)[:, h])
        # Gates of 2 over 150 rows reach sizes of 2^150, and FP32 ends at 2^128: from the run on in which a size passes 2^127 nothing
        # is asked (what overflows may reach every row of its run, as what is not finite may).
        past = np.flatnonzero(np.append(size, last) >= 2.0 ** 127)
        held = past[0] // 64 * 64 if past.size else c.T
        assert held >= 64 and np.isfinite(out[:held, h]).all()
        e = np.linalg.norm(out[:held, h] - o[:held, h], axis=1) / size[:held]
        worst = max(worst, e.max())
        assert e.max() <= tol, (h, int(e.argmax()), e.max())
        if not past.size:
            worst = max(worst, np.linalg.norm(state[0, h] - S[0, h]) / last)
            assert np.linalg.norm(state[0, h] - S[0, h]) <= tol * last
    return worst


def gate(x):
    def change(c):
        c.alpha[:] = x
    return change


def one_gate_of_2_30(c):
    c.alpha[:], c.alpha[60] = 0.9, 2.0 ** 30


def forgotten(size, at, gates):
    """A value of some size, and the gates of the rows from `at` on."""
    def change(c):
        c.v[20] = c.v[20] * size
        for i, a in enumerate(gates):
            c.alpha[at + i] = a
    return change


def forgotten_state(c):
    c.S0 *= 2e10
    c.alpha[3] = 0


def late(name, size, row=60):
    def change(c):
        t = getattr(c, name)
        t[row] = t[row] * size
        if name == "k":
            c.beta[row] = c.beta[row] / size ** 2
    return change


CASES = {"gates 1.1": gate(1.1), "gates 1.2": gate(1.2), "gates 1.3": gate(1.3), "gates 1.5": gate(1.5), "gates -1.5": gate(-1.5),
         "gates 2": gate(2.0), "one gate of 2^30": one_gate_of_2_30, "1e4 forgotten": forgotten(1e4, 25, [0.0]),
         "1e8 forgotten": forgotten(1e8, 25, [0.0]), "1e8 fading": forgotten(1e8, 21, [1e-4] * 40), "1e30 forgotten": forgotten(1e30, 25, [0.0]),
         "state forgotten": forgotten_state, "value 2^40": late("v", 2.0 ** 40), "query 2^40": late("q", 2.0 ** 40), "key 2^20": late("k", 2.0 ** 20),
         "strength 2^10": late("beta", 2.0 ** 10), "value 2^-100": late("v", 2.0 ** -100)}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("T", [64, 150])
def test_each_row_for_itself(w12, name, T):
    c = Case(w12, [T], 2, 1, seed=len(name))
    CASES[name](c)
    run(w12, c, TOL)


@pytest.mark.parametrize("name", ["1e8 forgotten", "1e8 fading", "state forgotten", "value 2^40", "query 2^40"])
def test_of_a_long_request(w12, name):
    """Cut into parts."""
    c = Case(w12, [1100], 2, 2, seed=7)
    CASES[name](c)
    run(w12, c, 2 * TOL)
    assert c.rows.scratch.numel() > 0


@pytest.mark.parametrize("name", ["gates 1.3", "value 2^40", "query 2^40", "one gate of 2^30"])
def test_rows_behind_change_nothing(w12, name):
    """What comes behind a row does not change its bits."""
    c = Case(w12, [64], 2, 2, seed=8)
    run(w12, c, TOL)
    before, _ = c.run(w12)
    alpha = c.alpha.clone()
    CASES[name](c)
    if name == "gates 1.3":
        c.alpha[:60] = alpha[:60]
    elif name == "one gate of 2^30":
        c.alpha[:60], c.alpha[61:] = alpha[:60], alpha[61:]
    run(w12, c, TOL)
    after, _ = c.run(w12)
    assert torch.equal(before[:60], after[:60]) and not torch.equal(before[60:], after[60:])
