"""The norms around a block (w12_gdn_norm, w12_block_norm) against their formulas in 64 bits.

Tolerances.  A sum of n FP32 squares has no terms of opposite sign, so it is off by (n / threads + 20) * 2^-24 of itself at
most, some 40 * 2^-24 here; its inverse root, the products and the gate's 2^x and reciprocal add less than 2^-19 together.  So
an FP32 result is within 2^-18 of its value (where two summands cancel: of the larger one).  BF16 has eight significant bits,
so its steps are at most 2^-7 of a value (torch.finfo's eps) and rounding to it is off by half of that, 2^-8."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

D = 128
F32 = 2.0 ** -18
BF16 = torch.finfo(torch.bfloat16).eps / 2 + F32
EPS = 1e-6


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


def rms(x, eps=EPS):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def near(got, ref, tol, floor=0.0):
    e = (got.double() - ref).abs()
    assert torch.isfinite(got).all()
    assert (e <= tol * (ref.abs() + floor) + 1e-37).all(), (e / (ref.abs() + floor + 1e-300)).max().item()


def silu(z):
    return z * torch.sigmoid(z)


@pytest.mark.parametrize("R,H", [(1, 1), (1, 3), (2, 32), (33, 5), (700, 7)])
@pytest.mark.parametrize("mode", ["plain", "gate", "first"])
@pytest.mark.parametrize("fused", [False, True])
def test_outputs_of_the_recurrent_layer(w12, R, H, mode, fused):
    g = torch.Generator().manual_seed(R * 100 + H)
    o = (torch.randn(R, H, D, generator=g) * torch.randn(R, H, 1, generator=g).exp()).cuda()
    o[R // 2, H - 1] = 0
    pad = 24 if fused else 0
    z = (torch.randn(R, H * D + pad, generator=g) * 3).bfloat16().cuda()[:, pad:]
    z[0, :6] = torch.tensor([0.0, -0.0, 80.0, -80.0, 200.0, -300.0])
    w = torch.randn(D, generator=g).bfloat16().cuda()
    back = torch.full((R + 2, H * D + pad), 3.0, dtype=torch.bfloat16, device="cuda")
    out = back[1:R + 1, pad:]
    got = w12.w12_gdn_norm(o, w, z=None if mode == "plain" else z, eps=EPS, gate_first=mode == "first", out=out)
    torch.cuda.synchronize()
    assert got is out
    od, zd, wd = o.double(), z.double().reshape(R, H, D), w.double()
    ref = rms(od) * wd if mode == "plain" else rms(od * silu(zd)) * wd if mode == "first" else rms(od) * wd * silu(zd)
    near(out, ref.reshape(R, H * D), BF16)
    assert (back[0] == 3).all() and (back[R + 1] == 3).all() and (back[:, :pad] == 3).all()
    if mode != "plain":
        w12.w12_gdn_norm(o, w, z=z, eps=EPS, gate_first=mode == "first", out=z)      # in place
        assert torch.equal(z, out)


def test_sizes_of_outputs(w12):
    """Heads of very large and very small outputs: eps decides below 1e-3, squares reach 1e36."""
    for scale in (1e18, 1e3, 1e-3, 1e-6, 1e-18):
        o = torch.randn(4, 2, D, device="cuda") * scale
        w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
        near(w12.w12_gdn_norm(o, w), rms(o.double()).reshape(4, -1), BF16)


def test_a_head_that_is_not_finite(w12):
    o = torch.randn(3, 2, D, device="cuda")
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    z = torch.randn(3, 2 * D, device="cuda").bfloat16()
    clean = w12.w12_gdn_norm(o, w, z=z)
    o[1, 1, 5] = float("nan")
    got = w12.w12_gdn_norm(o, w, z=z)
    assert got[1, D:].isnan().all()
    got[1, D:] = clean[1, D:]
    assert torch.equal(got, clean)


SIZES = [(1, 8), (3, 16), (2, 256), (5, 264), (1, 5120), (192, 5120), (4, 8192), (3, 8200), (2, 16384)]


@pytest.mark.parametrize("R,n", SIZES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("parts", ["y+pre", "y+post+pre", "pre", "y", "y+post"])
def test_between_blocks(w12, R, n, f32, parts):
    parts = parts.split("+")
    g = torch.Generator().manual_seed(n + R)
    new = lambda *s: torch.randn(s, generator=g)
    dt = torch.float32 if f32 else torch.bfloat16
    h = (new(R, n + 8) * 3).to(dt).cuda()[:, 8:]
    y = new(R, n + 16).bfloat16().cuda()[:, 16:] if "y" in parts else None
    if y is not None and R > 1:
        y[1] = 0
    post = (1 + 0.3 * new(n)).bfloat16().cuda() if "post" in parts else None
    pre = (1 + 0.3 * new(n)).bfloat16().cuda() if "pre" in parts else None
    back = torch.full((R + 2, n + 8), 5.0, dtype=dt, device="cuda")
    h_out = back[1:R + 1, :n] if y is not None else None
    scale = -0.375
    before = h.clone()
    got_h, x = w12.w12_block_norm(h, y, pre=pre, post=post, scale=scale, eps=EPS, h_out=h_out)
    torch.cuda.synchronize()
    assert torch.equal(h, before)
    hd = h.double()
    big = hd.abs()
    if y is not None:
        t = y.double() if post is None else rms(y.double()) * post.double()
        big = torch.maximum(big, (scale * t).abs())
        hd = hd + scale * t
        e = (got_h.double() - hd).abs()
        assert (e <= F32 * big + (0 if f32 else BF16) * hd.abs() + F32 * hd.abs()).all()
        assert (back[0] == 5).all() and (back[R + 1] == 5).all() and (back[:, n:] == 5).all()
    else:
        assert got_h is h
    if pre is None:
        assert x is None
        return
    r = 1 / (hd.square().mean(-1, keepdim=True) + EPS).sqrt()
    e = (x.double() - hd * r * pre.double()).abs()
    assert (e <= F32 * big * r * pre.double().abs() + BF16 * (hd * r * pre.double()).abs()).all()
    if y is not None:                                     # in place: h' over h, x over y
        h2, x2 = w12.w12_block_norm(h, y, pre=pre, post=post, scale=scale, eps=EPS, h_out=h, out=y)
        assert h2 is h and x2 is y and torch.equal(h, got_h) and torch.equal(y, x)


def test_x_comes_from_the_sum_before_it_is_rounded(w12):
    """h = 256 and y = 1/2 add up to what BF16 does not hold (its step there is 2)."""
    n = 64
    h = torch.full((1, n), 256.0, dtype=torch.bfloat16, device="cuda")
    h[0, 0] = 0
    y = torch.full((1, n), 0.5, dtype=torch.bfloat16, device="cuda")
    pre = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    got, x = w12.w12_block_norm(h, y, pre=pre)
    assert (got[0, 1:] == 256).all() and got[0, 0] == 0.5
    ref = torch.full((1, n), 256.5, dtype=torch.float64, device="cuda")
    ref[0, 0] = 0.5
    near(x, rms(ref), BF16)


def test_no_rows(w12):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
    assert w12.w12_gdn_norm(z(0, 4, D, dt=torch.float32), z(D)).shape == (0, 4 * D)
    h, x = w12.w12_block_norm(z(0, 64), z(0, 64), pre=z(64))
    assert h.shape == x.shape == (0, 64)


def test_many_rows_captured_on_another_stream(w12):
    R, n = 70000, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(R, n, generator=g, device="cuda").bfloat16()
    y = torch.randn(R, n, generator=g, device="cuda").bfloat16()
    pre = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    want_h, want = w12.w12_block_norm(h, y, pre=pre)
    torch.cuda.synchronize()
    near(want, rms(h.double() + y.double()), BF16, floor=1e-3)
    out, h_out = torch.zeros_like(y), torch.zeros_like(h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w12.w12_block_norm(h, y, pre=pre, h_out=h_out, out=out)
    assert not out.any()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(h_out, want_h)
    side = torch.cuda.Stream()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    w12.w12_block_norm(h, y, pre=pre, h_out=h_out, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
