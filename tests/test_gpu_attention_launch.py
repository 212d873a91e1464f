"""What the attention's launches rely on (marked gpu)."""
from __future__ import annotations

import ctypes as C

import pytest

from test_gpu_attention import World, attend, inputs, make_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


def test_every_shape_has_the_registers_its_shares_need(w12):
    """Each of the three kernels is looked at for itself, whichever ran first."""
    s = World(w12, [300], 1, 64, seed=40)
    for G in (64, 40, 1):                                   # segments of 80, 48 and 16 columns
        t = make_tree(s.g, [1])
        attend(w12, s, t, inputs(s.g, 1, 1, G, s)[3], 1, G, 1)
    wanted = C.c_int32(0)
    for cols in (16, 48, 80):
        assert w12.lib().w12_debug_attn_registers(cols, C.byref(wanted)) >= wanted.value > 0
    assert w12.lib().w12_debug_attn_registers(32, None) == 0
    assert s.ws.status() == 0
