"""w12_gdn_prefill on few long requests, whose parts run beside one another, against the token-by-token form in 64 bits.

Tolerances: those of the whole runs.  The state in front of a part is S P + Q, P and Q being runs of the kernel: one sum of 128
products more for each part, and P's roundings, which meet S as those of a state do.  Where every gate is 1 no run of
64 rows is forgotten, and their roundings (2.3e-6 of the 2-norm each) add up: independently, over n runs, to sqrt(n) times that,
and twice that with the parts' sums."""
from __future__ import annotations

import numpy as np
import pytest

from test_gpu_gdn_rows import Case, D, GATES, NORM, WORST

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


def slow(T, H, g):
    return 1 - torch.rand(T, H, generator=g) * 0.01


# requests x heads: one pair and 63 parts' worth of SMs, ..., 48 pairs with three SMs each
CASES = [([1024], 1, 1), ([1023], 2, 1), ([961], 1, 1), ([4000], 1, 1), ([1500, 10, 0, 2000], 2, 2), ([2100], 32, 16), ([1400] * 3, 16, 4),
         ([1000, 1030, 1500, 64], 6, 1), ([1200, 1, 960], 5, 5)]


@pytest.mark.parametrize("counts,H,Hk", CASES, ids=str)
@pytest.mark.parametrize("s0", [True, False])
def test_long_prompts(w12, counts, H, Hk, s0):
    c = Case(w12, counts, H, Hk, seed=sum(counts) + H, s0=s0, gap=5 if H == 2 else 0, fused=H != 5)
    c.check(*c.run(w12))
    assert c.rows.scratch.numel() > 0


@pytest.mark.parametrize("gate", ["slow", *GATES])
def test_gates(w12, gate):
    c = Case(w12, [1700, 1100], 3, 3, seed=2, alpha=slow if gate == "slow" else GATES[gate])
    runs = 1700 / 64 if gate in ("slow", "one") else 1
    c.check(*c.run(w12), worst=2 * runs ** 0.5 * WORST if runs > 1 else WORST, norm=2 * runs ** 0.5 * 2.3e-6 if runs > 1 else NORM)


def test_in_one_piece_without_scratch(w12):
    """Without scratch a request's head is one SM's: the same values up to rounding, and too little scratch is refused."""
    c = Case(w12, [1500], 2, 1, seed=3)
    out, state = c.run(w12)
    again, s2 = c.run(w12)
    assert torch.equal(out, again) and torch.equal(state, s2)
    nbytes, addr = c.rows.c.scratch_bytes, c.rows.c.scratch
    c.rows.c.scratch_bytes = nbytes - 1
    with pytest.raises(w12.W12Error):
        c.run(w12)
    c.rows.c.scratch, c.rows.c.scratch_bytes = addr + 4, nbytes
    with pytest.raises(w12.W12Error):
        c.run(w12)
    c.rows.c.scratch, c.rows.c.scratch_bytes = None, 0
    one, s1 = c.run(w12)
    c.check(one, s1)
    assert not torch.equal(out, one)
    c.rows.c.scratch, c.rows.c.scratch_bytes = addr, nbytes
    out2, s2 = c.run(w12)
    assert torch.equal(out, out2) and torch.equal(state, s2)


def test_in_place(w12):
    c = Case(w12, [1100, 1400], 3, 1, seed=4)
    state = c.S0.cuda()
    out = torch.full((c.T, 3, D), 7.0, device="cuda")
    w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=state, state=state, out=out)
    torch.cuda.synchronize()
    assert c.ws.status() == 0
    c.check(out, state)


def test_scratch_of_nan(w12):
    """Nothing of the scratch is read that the call has not written."""
    c = Case(w12, [1100, 300, 2400], 2, 2, seed=5)
    out, state = c.run(w12)
    c.rows.scratch.view(torch.float32).fill_(float("nan"))
    again, s2 = c.run(w12)
    assert torch.equal(out, again) and torch.equal(state, s2)


def test_nan_reaches_only_what_is_behind_it(w12):
    c = Case(w12, [1300, 1300], 2, 2, seed=6)
    clean, cs = c.run(w12)
    row = 1300 + 700                                  # request 1, head 1: its eleventh run of 64
    c.rows.k[row, D:2 * D] = float("nan")
    out, state = c.run(w12)
    bad = torch.zeros(c.T, 2, dtype=torch.bool, device="cuda")
    bad[1300 + 640:, 1] = True
    assert torch.equal(out[~bad], clean[~bad]) and out[row:, 1].isnan().all()
    keep = torch.ones(2, 2, dtype=torch.bool, device="cuda")
    keep[1, 1] = False
    assert torch.equal(state[keep], cs[keep]) and state[1, 1].isnan().all()


def test_offsets_that_make_no_sense(w12):
    c = Case(w12, [1100, 1200, 1300], 2, 2, seed=7)
    good, gs = c.run(w12)
    S0 = c.S0.cuda()
    out, state = torch.full_like(good, 7.0), torch.full_like(S0, 9.0)
    off = torch.tensor([0, 1100, 2300, 3601], dtype=torch.int32, device="cuda")
    w12.w12_gdn_prefill(c.rows, off, c.ws, S0=S0, state=state, out=out)
    torch.cuda.synchronize()
    assert c.ws.status() == w12.W12_E_INVAL
    assert torch.equal(state[:2], gs[:2]) and (state[2] == 9.0).all()
    assert torch.equal(out[:2300], good[:2300]) and (out[2300:] == 7.0).all()


def test_a_wait_that_runs_out(w12):
    """The first part of one head gives up (test hook): its state is left alone, the other head's is not."""
    c = Case(w12, [1500], 2, 2, seed=8)
    S0 = c.S0.cuda()
    w12.debug_set(1, 50_000_000)
    try:
        state, out = torch.full_like(S0, 9.0), torch.full((c.T, 2, D), 7.0, device="cuda")
        w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=S0, state=state, out=out)
        torch.cuda.synchronize()
        assert c.ws.status() == w12.W12_E_TIMEOUT
        assert (state[0, 0] == 9.0).all() and not (state[0, 1] == 9.0).any()
    finally:
        w12.debug_set(0, 0)
    c.check(*c.run(w12))


def test_captured(w12):
    """Captured before the first eager call, and replayed on a side stream."""
    c = Case(w12, [1700], 4, 2, seed=9)
    S0 = c.S0.cuda()
    out, state = torch.zeros(c.T, 4, D, device="cuda"), torch.zeros_like(S0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=S0, state=state, out=out)
    assert not out.any()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.replay()
        graph.replay()
    torch.cuda.synchronize()
    assert c.ws.status() == 0
    c.check(out, state)
    want, ws_ = c.run(w12)
    assert torch.equal(out, want) and torch.equal(state, ws_)
