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


def test_a_call_of_malformed_rows_ends_with_its_context(w12):
    """A tree in which no row is well formed, over a long context, and at once another call on the same scratch."""
    s = World(w12, [300, 200], 1, 64, seed=41)
    t = make_tree(s.g, [3, 2])
    dev = inputs(s.g, 5, 1, 4, s)[3]
    want = attend(w12, s, t, dev, 1, 4, 2)
    n, per = 4, 1024                                         # 4 requests of 131072 tokens, all of the same blocks
    z = lambda *a, dt=torch.uint8: torch.zeros(a, dtype=dt, device="cuda")
    long = w12.KvCache(z(per, 4, 128, 128), z(per, 4, 128, 128), z(per, 4, dt=torch.float32) + 1, z(per, 4, dt=torch.float32) + 1,
                       torch.arange(per, dtype=torch.int32, device="cuda").repeat(n, 1), z(n, dt=torch.int32) + per * 128)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    bad = w12.DeviceTree.from_arrays(i32([3, 3, 3, 3]), z(4), i32([0, 1, 2, 3]), i32([0, 1, 2, 3, 4]))   # parents outside or behind
    rows = torch.randn(4, 4 * 128, device="cuda").bfloat16()
    good = w12.DeviceTree.from_arrays(*(torch.from_numpy(x).cuda() for x in t))
    aws = w12.AttentionWorkspace(5, 16, 4, 4)
    ws = w12.Workspace(1, 0, 0, 4)
    out, got = z(4, 4, 128, dt=torch.bfloat16) + 1, torch.empty_like(want)
    torch.cuda.synchronize()
    for _ in range(20):
        w12.w12_tree_attention(long, None, bad, n, rows, rows, rows, ws, aws, out=out)
        w12.w12_tree_attention(s.cache, s.rope, good, 2, *dev, ws, aws, out=got)
        assert torch.equal(got, want) and (out == 0).all()
    assert ws.status() == w12.W12_E_INVAL
