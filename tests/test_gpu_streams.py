"""Memory that a call makes for itself, where it runs on another stream than the current one: neither memory that the current
stream may still use, nor memory that the current stream gets back while the call still uses it.  (What a torch allocation
returns is what the stream under which it is made last freed: so a block that has just been freed shows whose memory it was.)"""
from __future__ import annotations

import numpy as np
import pytest

from test_gpu_gdn_rows import Case, D

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


def busy(stream):
    """A tenth of a second's work in front of what comes next there."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(200_000_000)


def freed(nbytes):
    """The address of a block of the current stream's that has just become free."""
    t = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    at = t.data_ptr()
    del t
    again = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() == at          # (the next one would get it)
    del again
    return at


def overlap(t, at, nbytes):
    return t.data_ptr() < at + nbytes and at < t.data_ptr() + t.numel() * t.element_size()


@pytest.fixture
def side():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    yield s
    torch.cuda.synchronize()


def case(w12):
    c = Case(w12, [1500], 4, 4, seed=1)
    need = int(w12.lib().w12_gdn_scratch_bytes(4, c.T))
    assert need > 1 << 20
    return c, need


def test_scratch_is_not_the_current_streams(w12, side):
    c, need = case(w12)
    want, state = c.run(w12)
    c.rows = w12.GdnRows(c.rows.q, c.rows.k, c.rows.v, c.rows.alpha, c.rows.beta)
    S0, out, mine = c.S0.cuda(), torch.empty_like(want), torch.empty_like(state)
    side.wait_stream(torch.cuda.current_stream())
    at = freed(need)
    w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=S0, state=mine, out=out, stream=side)
    assert not overlap(c.rows.scratch, at, need)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(mine, state)


@pytest.mark.parametrize("first_on_current", [False, True])
def test_scratch_outlives_its_rows(w12, side, first_on_current):
    c, need = case(w12)
    want, state = c.run(w12)
    S0, out, mine = c.S0.cuda(), torch.empty_like(want), torch.empty_like(state)
    if not first_on_current:
        c.rows = w12.GdnRows(c.rows.q, c.rows.k, c.rows.v, c.rows.alpha, c.rows.beta)
    side.wait_stream(torch.cuda.current_stream())
    busy(side)
    rows, kept = c.rows, (c.rows.q, c.rows.k, c.rows.v, c.rows.alpha, c.rows.beta)
    c.rows = None
    w12.w12_gdn_prefill(rows, c.row_off, c.ws, S0=S0, state=mine, out=out, stream=side)
    at = rows.scratch.data_ptr()
    del rows
    other = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not any(overlap(t, at, need) for t in other)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(mine, state) and c.ws.status() == 0
    del kept


def norms(w12, stream):
    g = torch.Generator().manual_seed(2)
    new = lambda *s: torch.randn(s, generator=g)
    o, w, h, y = new(300, 4, D).cuda(), new(D).bfloat16().cuda(), new(300, 512).cuda(), new(300, 512).bfloat16().cuda()
    pre = new(512).bfloat16().cuda()
    torch.cuda.synchronize()
    return o, w, h, y, pre


def test_outputs_are_not_the_current_streams(w12, side):
    """What the calls make where the caller passes no output, while blocks of the same sizes have just been freed on the current
    stream; and it is not the current stream's again while the call still runs."""
    c, _ = case(w12)
    o, w, h, y, pre = norms(w12, side)
    step = Case(w12, [1] * 40, 4, 4, seed=3)
    S0, S1 = c.S0.cuda(), step.S0.cuda()
    torch.cuda.synchronize()
    calls = [lambda **k: w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=S0, **k), lambda **k: w12.w12_gdn_step(step.rows, S0=S1, **k),
             lambda **k: (w12.w12_gdn_norm(o, w, **k),), lambda **k: w12.w12_block_norm(h, y, pre=pre, **k)]
    for call in calls:
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        sizes = [t.numel() * t.element_size() for t in want]
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        at = [b.data_ptr() for b in blocks]
        del blocks
        busy(side)
        got = call(stream=side)
        for t in got:
            assert not any(overlap(t, a, n) for a, n in zip(at, sizes))
        for t, ref in zip(got, want):
            torch.cuda.current_stream().wait_stream(side)
            assert torch.equal(t, ref)
        busy(side)
        got = call(stream=side)
        where = [(t.data_ptr(), n) for t, n in zip(got, sizes)]
        del got, t
        other = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        assert not any(overlap(t, *w_) for t in other for w_ in where)
        del other
        torch.cuda.synchronize()


def test_the_current_stream_named(w12, side):
    """stream= the current one is as no stream."""
    c, _ = case(w12)
    want, state = c.run(w12)
    with torch.cuda.stream(side):
        out, mine = w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=c.S0.cuda(), stream=torch.cuda.current_stream())
        assert torch.equal(out, want) and torch.equal(mine, state)


def test_layers_share_a_scratch(w12, side):
    """Two layers' calls in a row, several times over, with one scratch between them."""
    cases = [case(w12)[0], Case(w12, [1100, 1300], 2, 1, seed=5)]
    want = [c.run(w12) for c in cases]
    scratch = w12.GdnScratch(4, 2400)
    for c in cases:
        c.rows = w12.GdnRows(c.rows.q, c.rows.k, c.rows.v, c.rows.alpha, c.rows.beta, scratch=scratch)
    S0 = [c.S0.cuda() for c in cases]
    torch.cuda.synchronize()
    got = [[w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=s, stream=side) for c, s in zip(cases, S0)] for _ in range(3)]
    side.synchronize()
    for pair in got:
        for (o, s), (o_ref, s_ref), c in zip(pair, want, cases):
            assert c.ws.status() == 0 and c.rows.scratch is scratch.buf
            assert torch.equal(o[c.off[0]:c.off[-1]], o_ref[c.off[0]:c.off[-1]]) and torch.equal(s, s_ref)


def older_calls(w12):
    """The other calls that make their outputs, on small inputs: name -> (call, its outputs' tensors)."""
    from speculative_decoding_tree_w12_gb300 import synth
    from test_binding_devices import parts

    w = synth.scaled(synth.WORKLOADS["tiny"], n_req=3, positions=(2, 4, 6), budget=12, n_cand=16, hit_rate=0.9)
    lat = w12.DeviceLattice(synth.lattice(w, 3))
    ws = w12.Workspace(12, 1024, 1024, 3)
    tree = w12.w12_tree_build(lat, w.budget, ws)
    R = tree.R
    g = torch.Generator().manual_seed(4)
    bits = lambda *s: torch.randn(s, generator=g).bfloat16().view(torch.int16).numpy().view(np.uint16)
    lin, head = (w12.DeviceWeight(w12.w12_pack(bits(1024, 512))) for _ in range(2))
    x = torch.randn(R, 512, generator=g).bfloat16().cuda()
    argmax = torch.randint(0, 16, (R,), generator=g, dtype=torch.int32).cuda()
    norms = w12.w12_head_cert_norms(head)
    cws = w12.CertWorkspace(R, 1024)
    xg = synth.gdn_inputs(R, 3, 2, 128, seed=4)
    dev = lambda a: torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()
    layer = w12.GdnLayer(torch.from_numpy(xg.S0).cuda(), dev(xg.q), dev(xg.k), dev(xg.v), torch.from_numpy(xg.alpha).cuda(),
                         torch.from_numpy(xg.beta).cuda())
    node = (tree.req_row_off[1:] - 1).contiguous()
    _, u = w12.w12_gdn_wy_verify(layer, tree, 3, ws)
    a = parts(w12, "cuda")
    fields = lambda t: (t.parent[:R], t.token[:R], t.depth[:R], t.req[:R], t.score[:R], t.rank[:R], t.req_row_off)
    torch.cuda.synchronize()
    return {
        "unpack": lambda **k: (w12.w12_unpack(lin, **k),),
        "gemm": lambda **k: (w12.w12_gemm(lin, x, ws, **k),),
        "argmax": lambda **k: (w12.w12_lmhead_argmax(head, x, ws, **k),),
        "norms": lambda **k: (w12.w12_head_cert_norms(head, **k),),
        "certified": lambda **k: (w12.w12_lmhead_argmax_certified(head, norms, x, ws, cws, **k),),
        "tree": lambda **k: fields(w12.w12_tree_build(lat, w.budget, ws, **k)),
        "accept": lambda **k: w12.w12_tree_accept(tree, 3, w.p_max, argmax, **k)[1:],
        "gdn verify": lambda **k: (w12.w12_gdn_tree_verify(layer, tree, 3, ws, **k),),
        "gdn commit": lambda **k: (w12.w12_gdn_commit(layer, tree, 3, node, ws, **k),),
        "wy verify": lambda **k: w12.w12_gdn_wy_verify(layer, tree, 3, ws, **k),
        "wy commit": lambda **k: (w12.w12_gdn_wy_commit(layer, tree, 3, node, u, ws, **k),),
        "attention": lambda **k: (w12.w12_tree_attention(a["cache"], a["rope"], a["tree"], 2, a["q"], a["k"], a["v"], a["ws"], a["aws"], **k),),
        "sample": lambda **k: (w12.w12_tree_sample(a["dist"], a["tree"], 2, a["ws"], **k),),
        "verify sampled": lambda **k: w12.w12_tree_verify_sampled(a["dist"], a["tree"], 2, 2, a["ws"], **k)[1:],
    }


def test_outputs_of_the_other_calls(w12, side):
    for name, call in older_calls(w12).items():
        want = [t.clone() for t in call()]
        torch.cuda.synchronize()
        sizes = [t.untyped_storage().nbytes() for t in want]
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
        at = [(b.data_ptr(), b.numel()) for b in blocks]
        del blocks
        # the current stream is behind: what it does to memory of its own comes after the call
        busy(torch.cuda.current_stream())
        got = call(stream=side)
        for t in got:
            assert not any(overlap(t, *b) for b in at), name
        torch.cuda.synchronize()
        for t, ref in zip(got, want):
            assert torch.equal(t, ref), name


def test_sampling_scratch_outlives_its_rows(w12, side):
    from test_binding_devices import parts
    a = parts(w12, "cuda")
    logits, u = torch.randn(4, 70000, device="cuda"), torch.rand(4, device="cuda")
    make = lambda: w12.SampleRows(logits, u)
    want = w12.w12_tree_sample(make(), a["tree"], 2, a["ws"]).clone()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    dist = make()
    at, n = dist.scratch.data_ptr(), dist.scratch.numel()
    busy(side)
    tok = w12.w12_tree_sample(dist, a["tree"], 2, a["ws"], stream=side)
    del dist
    other = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert not any(overlap(t, at, n) for t in other)
    side.synchronize()
    assert torch.equal(tok, want)
