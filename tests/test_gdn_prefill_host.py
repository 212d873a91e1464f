"""Host tests of w12_gdn_prefill: what of the kernel can be looked at without running it."""
from __future__ import annotations

import pytest


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


def test_the_inverse_of_a_chunk_waits_for_the_one_before(w12):
    """No word of shared memory is written by one of the inverse's warps while another may still use it, the next chunk's
    steps right behind a chunk's included (counted from the places and barriers that the kernel runs by)."""
    assert w12.lib().w12_debug_gdn_inverse_conflicts() == 0


def test_scratch_of_several_layers(w12):
    """A scratch is taken by any rows that it is large enough for, and by no others."""
    torch = pytest.importorskip("torch")
    b = lambda T, n: torch.zeros(T, n, dtype=torch.bfloat16)
    rows = lambda T, s, H=4: w12.GdnRows(b(T, 256), b(T, 256), b(T, 128 * H), torch.zeros(T, H), torch.zeros(T, H), scratch=s)
    large, none = w12.GdnScratch(4, 5000, device="cpu"), w12.GdnScratch(4, 100, device="cpu")
    assert large.nbytes == w12.lib().w12_gdn_scratch_bytes(4, 5000) > 0 and none.nbytes == 0
    for T, s in ((5000, large), (100, large), (2000, large), (100, none)):
        r = rows(T, s)
        assert r.scratch is s.buf and (r.c.scratch or 0) == (s.buf.data_ptr() if s.nbytes else 0) and r.c.scratch_bytes == s.nbytes
    with pytest.raises(ValueError):
        rows(5000, none)
