"""w12_gdn_norm's gate over its whole range, against the formula in 64 bits.

Tolerances: those of the norms (half a BF16 step and 2^-18 of a value), the gate's own (8 + 0.45 |z|) 2^-23 (its 2^x is off by 2
units of 2^-23, its reciprocal by 1, log2(e) by 0.12 |z|, the exponent by half its last place, four products by 4 halves), and where
results are not normal numbers half of BF16's smallest step, 2^-134; with the gate in front, o silu(z) is then rounded by FP32's
smallest half steps, 2^-150 (|o| + 1), before it is multiplied by 1 / sqrt(eps) = 1000 and a weight, |o| + 1 <= 5.5 and |w| <= 4 here:
2^-135.5 more, so 2^-133 in all."""
from __future__ import annotations

import pytest

from test_gpu_norms import BF16, D, EPS, rms

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


SPANS = {"far below": (-89.5, -87.0), "down to nothing": (-110.0, -85.0), "below": (-87.0, -20.0), "around zero": (-20.0, 20.0),
         "above": (20.0, 110.0), "very far": (-3e38, 3e38)}


@pytest.mark.parametrize("first", [False, True])
@pytest.mark.parametrize("span", SPANS)
def test_gates_of_any_size(w12, span, first):
    lo, hi = SPANS[span]
    R, H = 33, 3
    g = torch.Generator().manual_seed(1)
    z = (torch.rand(R, H * D, generator=g, dtype=torch.float64) * (hi - lo) + lo).bfloat16().cuda()
    o = torch.randn(R, H, D, generator=g).cuda()
    if first and span == "very far":
        o *= 1e-30                       # (o silu(z) is squared)
    w = torch.randn(D, generator=g).bfloat16().cuda()
    got = w12.w12_gdn_norm(o, w, z=z, eps=EPS, gate_first=first).double()
    od, zd, wd = o.double(), z.double().reshape(R, H, D), w.double()
    silu = zd * torch.sigmoid(zd)
    ref = (rms(od * silu) * wd if first else rms(od) * wd * silu).reshape(R, H * D)
    held = ref.abs() < torch.finfo(torch.bfloat16).max          # (times w, the largest gates leave BF16's range)
    e = (got - ref).abs()[held]
    assert held.float().mean() > 0.2
    own = (8 + 0.45 * z.double().abs().clamp(max=110)) * 2.0 ** -23
    assert o.abs().max() <= 4.5 and w.abs().max() <= 4
    assert (e <= (BF16 + own)[held] * ref.abs()[held] + 2.0 ** -133).all(), (e / ref.abs()[held]).max()
    assert torch.isfinite(got[held]).all() and (got[~held].isinf() | (ref[~held].abs() < 1.01 * torch.finfo(torch.bfloat16).max)).all()
