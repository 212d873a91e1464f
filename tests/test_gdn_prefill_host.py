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
