"""w12_gdn_prefill again and again on the same inputs, right behind one another: every call gives the first one's bits, whatever its
launches meet on the machine."""
from __future__ import annotations

import pytest

from test_gpu_gdn_rows import Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


# cut into parts whose launches overlap (three SMs a pair, one wave and several of the join), many pairs a CTA
@pytest.mark.parametrize("counts,H,Hk", [([1400] * 3, 16, 4), ([2100], 32, 16), ([1500, 10, 0, 2000], 2, 2), ([200, 150, 64, 300] * 20, 4, 2)],
                         ids=["3x1400", "2100", "1500+10+0+2000", "80 requests"])
def test_every_call_gives_the_same(w12, counts, H, Hk):
    c = Case(w12, counts, H, Hk, seed=sum(counts) + H)
    S0 = c.S0.cuda()
    out, state = c.run(w12)
    c.check(out, state)
    again, s2 = torch.empty_like(out), torch.empty_like(state)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    inside = c.inside.cuda()
    for i in range(600):
        if i % 3 == 1:
            again.zero_()
        w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=S0, state=s2, out=again)
        differ += (again[inside] != out[inside]).any() | (s2 != state).any()
    assert int(differ) == 0 and c.ws.status() == 0
