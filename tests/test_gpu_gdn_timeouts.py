"""w12_gdn_prefill when one role of a CTA gives up while the others still wait: what that role has signalled since is part of no
state, and a state is written whole or not at all."""
from __future__ import annotations

import numpy as np
import pytest

from test_gpu_gdn_rows import Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ONE_ROLE = 32       # debug flag: see w12_debug.h


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


@pytest.fixture
def one_role(w12):
    w12.debug_set(ONE_ROLE, 0)
    yield
    w12.debug_set(0, 0)


def last_pair_of_the_first_cta(w12, counts, H):
    """(request, head): requests by their rows, their heads beside one another, dealt to the CTAs forth and back."""
    order = sorted(range(len(counts)), key=lambda r: (-counts[r], r))
    pairs = [(r, h) for r in order for h in range(H) if counts[r]]
    grid = min(len(counts) * H, w12.lib().w12_debug_num_sms())
    own = [i * grid + (grid - 1 if i & 1 else 0) for i in range(-(-len(pairs) // grid))]
    return pairs[[i for i in own if i < len(pairs)][-1]]


@pytest.mark.parametrize("counts,H,cut", [([150, 40], 2, False), ([64], 1, False), ([70] * 100, 4, False), ([1500], 2, True),
                                          ([1100, 1400], 3, True)], ids=["150+40", "64", "100x70", "1500", "1100+1400"])
@pytest.mark.parametrize("in_place", [False, True])
def test_one_role_gives_up(w12, one_role, counts, H, cut, in_place):
    c = Case(w12, counts, H, 1, seed=len(counts))
    w12.debug_set(0, 0)
    good, want = c.run(w12)
    w12.debug_set(ONE_ROLE, 0)
    S0 = c.S0.cuda()
    state = S0.clone() if in_place else torch.full_like(S0, 9.0)
    before = state.clone()
    w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=state if in_place else S0, state=state, out=torch.empty_like(good))
    torch.cuda.synchronize()
    assert c.ws.status() == w12.W12_E_TIMEOUT
    # (where requests are cut into parts the first CTA has the first part of the longest one's first head)
    r, h = (int(np.argmax(counts)), 0) if cut else last_pair_of_the_first_cta(w12, counts, H)
    assert torch.equal(state[r, h], before[r, h])
    want[r, h] = before[r, h]
    assert torch.equal(state, want)
    # and without the hook the call is right again
    w12.debug_set(0, 0)
    out, again = c.run(w12)
    assert torch.equal(out, good)
    c.check(out, again)
