"""Sampled verification where its weights can go wrong (marked gpu)."""
from __future__ import annotations

import numpy as np
import pytest

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
