"""The recurrent layer over rows where its calls are larger, stranger or nearer one another than elsewhere: many requests a
CTA, gates and strengths outside [0, 1], two calls at once, and a whole layer's calls in a row.

Tolerances.  Strengths up to 2 make u = b (v - a S k) up to twice the bound B of the other tests, and so its roundings: twice their
tolerances.  B takes the states' growth in, where gates above 1 make them grow.  In the run of a layer each call is held
against its formula in 64 bits on the rows that it was given: the norms to BF16's half step of a value and 2^-18 (their FP32
part), which for h + scale t is 2^-18 of |h| + |scale t|: t's own error and the sum's rounding are relative to those, however
near zero the sum comes.  The linears to half a step of a value and 2^-16 of its row's |x| |w| (sums of 512 and 256 FP32 products)."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from test_gpu_gdn_rows import Case, D, NORM, WORST
from test_gpu_norms import BF16, F32, near, rms, silu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


@pytest.mark.parametrize("n,H,Hk,longest,in_place", [(40, 6, 3, 200, False), (100, 4, 4, 130, True), (512, 1, 1, 3, False), (31, 9, 1, 260, True)])
def test_several_pairs_to_a_cta(w12, n, H, Hk, longest, in_place):
    """More requests and heads than SMs, of all lengths, empty ones among them."""
    r = np.random.default_rng(n)
    counts = [int(x) for x in r.integers(0, longest + 1, n)]
    counts[n // 2] = counts[-1] = 0
    c = Case(w12, counts, H, Hk, seed=n)
    if in_place:
        state = c.S0.cuda()
        out = torch.full((c.T, H, D), 7.0, device="cuda")
        w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=state, state=state, out=out)
        torch.cuda.synchronize()
        assert c.ws.status() == 0
        c.check(out, state)
    else:
        c.check(*c.run(w12))


def test_many_with_offsets_that_make_no_sense(w12):
    """Two of sixty requests cannot be: they are left as they were, the others served."""
    c = Case(w12, [50 + i for i in range(60)], 5, 5, seed=1)
    good, gs = c.run(w12)
    S0, off = c.S0.cuda(), c.off.copy()
    off[20], off[60] = off[21] + 1, c.T + 1           # request 19 takes 20's rows in and one more, 20 descends; 59 leaves the rows
    out, state = torch.full_like(good, 7.0), torch.full_like(S0, 9.0)
    w12.w12_gdn_prefill(c.rows, torch.from_numpy(off).cuda(), c.ws, S0=S0, state=state, out=out)
    torch.cuda.synchronize()
    assert c.ws.status() == w12.W12_E_INVAL
    keep = [r for r in range(60) if r not in (19, 20, 59)]
    assert torch.equal(state[keep], gs[keep]) and (state[[20, 59]] == 9.0).all()
    a, b, e = int(c.off[19]), int(c.off[22]), int(c.off[59])
    assert torch.equal(out[:a], good[:a]) and torch.equal(out[b:e], good[b:e]) and (out[e:] == 7.0).all()


@pytest.mark.parametrize("gate", ["negative", "above one", "growing"])
@pytest.mark.parametrize("counts", [[150, 70], [1500]], ids=str)
def test_gates_and_strengths_outside_the_unit_range(w12, gate, counts):
    span = {"negative": (-1.0, 1.0), "above one": (0.8, 1.1), "growing": (1.0, 1.02)}[gate]
    alpha = lambda T, H, g: torch.rand(T, H, generator=g) * (span[1] - span[0]) + span[0]
    beta = lambda T, H, g: torch.rand(T, H, generator=g) * 2
    c = Case(w12, counts, 3, 3, seed=2, alpha=alpha, beta=beta)
    runs = max(counts) / 64 if gate == "growing" else 4      # that a state remembers
    c.check(*c.run(w12), worst=2 * WORST * runs ** 0.5, norm=2 * NORM * runs ** 0.5)


def test_two_calls_at_once(w12):
    """Two calls on two streams, one of few long requests and one of many short ones, each with its own rows and workspace."""
    a, b = Case(w12, [1800], 4, 4, seed=3), Case(w12, [90] * 30, 4, 2, seed=4)
    want = [c.run(w12) for c in (a, b)]
    S0 = [c.S0.cuda() for c in (a, b)]
    outs = [[torch.full_like(o, 7.0) for _ in range(6)] for o, _ in want]
    states = [[torch.empty_like(s) for _ in range(6)] for _, s in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(6):
        for k, c in enumerate((a, b)):
            w12.w12_gdn_prefill(c.rows, c.row_off, c.ws, S0=S0[k], state=states[k][i], out=outs[k][i], stream=streams[k])
    torch.cuda.synchronize()
    for k, c in enumerate((a, b)):
        assert c.ws.status() == 0
        for i in range(6):
            assert torch.equal(outs[k][i], want[k][0]) and torch.equal(states[k][i], want[k][1])


def test_on_another_device_than_the_current_one(w12, monkeypatch):
    """The library launches on the current device: with tensors elsewhere the calls are refused (the current device here
    is made another one by its name only)."""
    c = Case(w12, [10], 2, 2, seed=6)
    o, w = torch.zeros(10, 2, D, device="cuda"), torch.ones(D, dtype=torch.bfloat16, device="cuda")
    h = torch.zeros(10, 64, dtype=torch.bfloat16, device="cuda")
    calls = [lambda: w12.w12_gdn_prefill(c.rows, c.row_off, c.ws), lambda: w12.w12_gdn_step(c.rows), lambda: w12.w12_gdn_norm(o, w),
             lambda: w12.w12_block_norm(h, h)]
    for call in calls:
        call()
    monkeypatch.setattr(w12, "_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError):
            call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("post,f32", [(False, False), (True, True)])
def test_a_layer_of_prompts_and_tokens(w12, post, f32):
    """norm - linear - recurrent layer - norm with gate - linear - residual and norm, over a prompt and over two tokens behind it,
    captured as one graph; every call against its formula on what it was given."""
    n, H, counts, two = 256, 2, [90, 0, 33], 2
    g = torch.Generator().manual_seed(5)
    wide = 4 * H * D                                         # q, k, v, z of a row
    bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    Wi = (torch.randn(wide, n, generator=g) / n ** 0.5).bfloat16()
    Wo = (torch.randn(n, H * D, generator=g) / (H * D) ** 0.5).bfloat16()
    wi, wo = (w12.DeviceWeight(w12.w12_pack(bits(w))) for w in (Wi, Wo))
    vec = lambda m: torch.randn(m, generator=g).bfloat16().cuda()
    pre, after, weight, behind = vec(n), vec(n), vec(D), vec(n) if post else None
    off = torch.from_numpy(np.cumsum([0] + counts).astype(np.int32)).cuda()
    S0 = (torch.randn(3, H, D, D, generator=g) * 0.05).cuda()
    state = torch.empty_like(S0)

    class Rows:
        def __init__(self, R):
            new = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")
            stream = torch.float32 if f32 else torch.bfloat16
            self.h = torch.randn(R, n, generator=g).to(stream).cuda()
            self.x, self.r, self.a, self.y, self.h2, self.x2 = new(R, n), new(R, wide), new(R, H * D), new(R, n), new(R, n, t=stream), new(R, n)
            self.o = new(R, H, D, t=torch.float32)
            self.alpha, self.beta = (torch.rand(R, H, generator=g).cuda() for _ in range(2))
            self.alpha = self.alpha * 0.3 + 0.7
            # keys and queries of some unit length: the linear's outputs over 16
            self.qk = new(R, 2 * H * D)
            self.ws = w12.Workspace(R, wide, 0, 3)
            self.rows = w12.GdnRows(self.qk[:, :H * D], self.qk[:, H * D:], self.r[:, 2 * H * D:3 * H * D], self.alpha, self.beta)

        def forward(self, layer):
            w12.w12_block_norm(self.h, pre=pre, out=self.x)
            w12.w12_gemm(wi, self.x, self.ws, y=self.r)
            self.qk.copy_(self.r[:, :2 * H * D] / 16)
            layer(self)
            w12.w12_gdn_norm(self.o, weight, z=self.r[:, 3 * H * D:], out=self.a)
            w12.w12_gemm(wo, self.a, self.ws, y=self.y)
            w12.w12_block_norm(self.h, self.y, pre=after, post=behind, scale=0.5, h_out=self.h2, out=self.x2)

        def check(self, S0, counts, state):
            d = lambda t: t.double()
            near(d(self.x), rms(d(self.h)) * d(pre), BF16)
            for y, x, W in ((self.r, self.x, Wi), (self.y, self.a, Wo)):
                W = d(W.cuda())
                floor = d(x).norm(dim=1)[:, None] * W.norm(dim=1)[None] * 2.0 ** -16
                assert ((d(y) - d(x) @ W.T).abs() <= BF16 * (d(x) @ W.T).abs() + floor).all()
            heads = lambda t: bits(t).reshape(-1, H, D)
            o, S, top = oracle.gdn_sequence(S0.cpu().numpy(), heads(self.qk[:, :H * D]), heads(self.qk[:, H * D:]),
                                            heads(self.r[:, 2 * H * D:3 * H * D]), self.alpha.cpu().numpy(), self.beta.cpu().numpy(),
                                            np.cumsum([0] + counts))
            # (keys of up to some 1.3: the bound on what lies in between with their squares)
            far = 4 * WORST * top.max()
            assert np.abs(self.o.cpu().double().numpy() - o).max() <= far and np.abs(state.cpu().double().numpy() - S).max() <= far
            R = self.o.shape[0]
            near(d(self.a), (rms(d(self.o)) * d(weight) * silu(d(self.r[:, 3 * H * D:]).reshape(R, H, D))).reshape(R, -1), BF16, 2.0 ** -18)
            t = d(self.y)
            if post:
                t = rms(t) * d(behind)
            h = d(self.h) + 0.5 * t
            summands, size = d(self.h).abs() + 0.5 * t.abs(), (h.square().mean(-1, keepdim=True) + 1e-6).sqrt()
            near(d(self.h2), h, *((F32, summands) if f32 else (BF16, summands * (F32 / BF16))))
            near(d(self.x2), rms(h) * d(after), BF16, d(after).abs() * summands / size * (F32 / BF16))

    prompt, token = Rows(sum(counts)), Rows(3)
    last = [state.clone() for _ in range(3)]

    def run():
        prompt.forward(lambda s: w12.w12_gdn_prefill(s.rows, off, s.ws, S0=S0, state=state, out=s.o))
        last[0].copy_(state)
        for i in range(two):
            token.forward(lambda s: w12.w12_gdn_step(s.rows, S0=state, state=state, out=s.o))
            last[i + 1].copy_(state)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for t in (prompt.x2, prompt.o, token.x2, token.o, state):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert prompt.ws.status() == 0 and token.ws.status() == 0
    prompt.check(S0, counts, last[0])
    token.check(last[1], [1, 1, 1], last[2])                 # (its buffers hold the second token's)


@pytest.mark.parametrize("long", [False, True])
def test_replayed_with_other_offsets(w12, long):
    """A graph's call reads its offsets when it is replayed: where requests are cut follows them."""
    T, H = (2600, 2) if long else (300, 3)
    c = Case(w12, [T // 2, T - T // 2], H, 1, seed=7)
    S0, off = c.S0.cuda(), c.row_off.clone()
    out, state = torch.empty(T, H, D, device="cuda"), torch.empty_like(S0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w12.w12_gdn_prefill(c.rows, off, c.ws, S0=S0, state=state, out=out)
    for cut in (T // 2, 1, T, 0, 65, T - 700 if long else 64):
        off.copy_(torch.tensor([0, cut, T], dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        want, ws_ = w12.w12_gdn_prefill(c.rows, off, c.ws, S0=S0)
        torch.cuda.synchronize()
        assert c.ws.status() == 0 and torch.equal(out, want) and torch.equal(state, ws_)
        c.counts, c.off = [cut, T - cut], np.asarray([0, cut, T], np.int32)
        if not long or cut in (1, T - 700):
            c.check(out, state)


def test_calls_overlap_only_where_nothing_depends(w12):
    """Kernels begin while the ones before them end.  Forty tokens through a layer whose rows are small and whose calls
    feed one another, in one go, give what they give with a pause behind every call."""
    n, H, R = 256, 4, 5
    g = torch.Generator().manual_seed(8)
    bits = lambda t: t.contiguous().view(torch.int16).numpy().view(np.uint16)
    weight = lambda a, b: w12.DeviceWeight(w12.w12_pack(bits((torch.randn(a, b, generator=g) / b ** 0.5).bfloat16())))
    wi, wo = weight(3 * H * D, n), weight(n, H * D)
    one = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    head = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    h0 = torch.randn(R, n, generator=g).cuda()
    S0 = (torch.randn(R, H, D, D, generator=g) * 0.05).cuda()
    alpha, beta = (torch.rand(R, H, generator=g).cuda() for _ in range(2))
    ws = w12.Workspace(R, 3 * H * D, 0, R)
    off = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    new = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")

    def run(pause):
        h, state, x, r, a, y = h0.clone(), S0.clone(), new(R, n), new(R, 3 * H * D), new(R, H * D), new(R, n)
        o = new(R, H, D, t=torch.float32)
        rows = w12.GdnRows(r[:, :H * D], r[:, H * D:2 * H * D], r[:, 2 * H * D:], alpha, beta)
        w12.w12_block_norm(h, pre=one, out=x)
        for i in range(40):
            calls = [lambda: w12.w12_gemm(wi, x, ws, y=r),
                     # unit keys and queries
                     lambda: w12.w12_gdn_norm(r[:, :2 * H * D].float().view(R, 2 * H, D), head, out=r[:, :2 * H * D]),
                     lambda: r[:, :2 * H * D].mul_(D ** -0.5),
                     (lambda: w12.w12_gdn_step(rows, S0=state, state=state, out=o)) if i % 3 else
                     (lambda: w12.w12_gdn_prefill(rows, off, ws, S0=state, state=state, out=o)),
                     lambda: w12.w12_gdn_norm(o, head, out=a),
                     lambda: w12.w12_gemm(wo, a, ws, y=y),
                     lambda: w12.w12_block_norm(h, y, pre=one, scale=0.5, h_out=h, out=x)]
            for call in calls:
                call()
                if pause:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert ws.status() == 0
        return h, state, x

    want = run(True)
    assert all(torch.isfinite(t.float()).all() for t in want)
    for _ in range(3):
        for got, ref in zip(run(False), want):
            assert torch.equal(got, ref)
