"""Tree attention over contexts whose scores span a wide range (marked gpu):
dominating keys, scores that rise or fall along the context, values that are
not numbers.  Compared with the softmax in 64 bits, within bounds derived from
the roundings that include/w12.h states."""
from __future__ import annotations

import math

import numpy as np
import pytest

from oracle import attention as ref
from test_gpu_attention import D, World, attend, close, inputs, make_tree

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
BT = 128


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


class Shared:
    """n requests of one row each that read one cached context of `tokens` tokens (one head, no rotation): as many
    segments as that are not split over CTAs.  Keys: dimension 0 as given, small random codes in eight others; the rows'
    own keys: own_k0 in dimension 0."""

    def __init__(self, w12, n, G, k0, seed, v=None, own_k0=0.0):
        g = np.random.default_rng(seed)
        tokens = len(k0)
        blocks = -(-tokens // BT)
        k = np.zeros((blocks * BT, D))
        k[:tokens, 0] = k0
        k[:, 1:9] = g.standard_normal((blocks * BT, 8))
        v = 8 + 16 * g.standard_normal((blocks * BT, D)) if v is None else v
        self.kc, self.vc = ref.e4m3_encode(k), ref.e4m3_encode(np.clip(v, -448, 448))
        self.n, self.G, self.tokens = n, G, tokens
        self.heads = list(range(0, G, 9)) + [G - 1]                # those that are compared
        c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        ones = torch.ones(blocks, 1, device="cuda")
        table = torch.arange(blocks, dtype=torch.int32, device="cuda").repeat(n, 1)
        self.cache = w12.KvCache(c(self.kc.reshape(blocks, 1, BT, D)), c(self.vc.reshape(blocks, 1, BT, D).transpose(0, 1, 3, 2)),
                                 ones, ones / 16, table, torch.full((n,), tokens, dtype=torch.int32, device="cuda"))
        j = np.arange(n)
        i32 = lambda a: c(np.asarray(a, np.int32))
        self.tree = w12.DeviceTree.from_arrays(i32(np.full(n, -1)), torch.zeros(n, dtype=torch.uint8, device="cuda"), i32(j),
                                               i32(np.arange(n + 1)))
        q = np.zeros((n, G, D))
        q[:, :, 0] = 1.0
        q[:, :, 1:9] = np.round(g.standard_normal((n, G, 8)) * 16) / 64
        self.own_k0, own_k = own_k0, np.zeros((n, D))
        own_k[:, 0] = own_k0
        x = np.concatenate([q.reshape(n, -1), own_k, np.round(g.standard_normal((n, D)) * 16) / 16], 1)
        self.rows = c(x.astype(np.float32)).bfloat16()
        assert torch.equal(self.rows.double().cpu(), torch.from_numpy(x))
        self.ws = w12.Workspace(1, 0, 0, n)
        self.aws = w12.AttentionWorkspace(n, G, 1, n)

    def run(self, w12, scale):
        a, b = self.G * D, self.G * D + D
        out = w12.w12_tree_attention(self.cache, None, self.tree, self.n, self.rows[:, :a], self.rows[:, a:b], self.rows[:, b:],
                                     self.ws, self.aws, scale=scale)
        torch.cuda.synchronize()
        assert self.ws.status() == 0
        return out[:, self.heads].double()

    def exact(self, scale):
        """Of some of the heads: outputs, sum p |v|, sum |v|, the largest p and the largest score error ds, in 64 bits."""
        c = lambda a: torch.from_numpy(a).cuda()
        K, V = c(ref.E4M3[self.kc[:self.tokens]]), c(ref.E4M3[self.vc[:self.tokens]] / 16)
        G, x = self.G, self.rows.double()
        q, own = x[:, :G * D].reshape(-1, G, D)[:, self.heads].reshape(-1, D), x[:, G * D + D:].repeat_interleave(len(self.heads), 0)
        outs = []
        for at in range(0, len(q), 1024):
            Q, o = q[at:at + 1024], own[at:at + 1024]
            s = torch.cat([Q @ K.T * scale, Q[:, :1] * self.own_k0 * scale], 1)
            p = torch.softmax(s, 1)
            last = p[:, -1:]
            ds = scale * (Q.abs() @ K.abs().T * 2.0 ** -12 + 2.0 ** -17 * Q.abs().amax(1, keepdim=True) * K.abs().sum(1)).amax(1)
            outs.append((p[:, :-1] @ V + last * o, p[:, :-1] @ V.abs() + last * o.abs(), p.amax(1), ds))
        out, pv, top, ds = (torch.cat(t) for t in zip(*outs))
        return out, pv, V.abs().sum(0), top, ds


def compare(w12, s, scale, coarse):
    """coarse: tokens whose weights may be rounded to the multiples of 2^-26 of the largest."""
    got = s.run(w12, scale)
    out, pv, v_sum, top, ds = s.exact(scale)
    # scores within ds (of the token and of the sum); weights and sums within 2^-10; the output's rounding; and the
    # coarse weights within 2^-27 of the largest, each times |v|
    slack = (2 * ds[:, None] + 2.0 ** -10) * pv + 2.0 ** -8 * out.abs() + coarse * 2.0 ** -27 * top[:, None] * v_sum / s.tokens
    worst = ((got.reshape(out.shape) - out).abs() / slack.clamp(min=1e-30)).max().item()
    assert worst <= 1, worst
    return got


# one row of 1, 40 and 64 heads to a request: segments of 16, 48 and 80 columns
@pytest.mark.parametrize("G", [1, 40, 64])
@pytest.mark.parametrize("gap", [14.0, 20.0, 23.1, 26.5, 35.0])
@pytest.mark.parametrize("at", [0, 40000])
def test_a_dominating_key_without_a_value(w12, G, gap, at):
    """65536 all but flat keys behind (and before) one that outweighs each by 2^gap and whose value is zero: the output is
    what the flat ones hold.  Each of a segment's two groups comes back to the flat keys' range after 128 tiles of 128."""
    k0 = np.zeros(65536)
    k0[at] = 16.0
    v = 8 + 16 * np.random.default_rng(1).standard_normal((65536, D))
    v[at] = 0
    compare(w12, Shared(w12, 160, G, k0, 5, v), gap * math.log(2) / 16, 128 * 128)


@pytest.mark.parametrize("G", [1, 64])
@pytest.mark.parametrize("rise", [30.0, -30.0, 300.0, -300.0])
def test_scores_that_rise_or_fall(w12, G, rise):
    """Along 40000 tokens by 2^rise in all, which passes or leaves every reference there was."""
    k0 = np.linspace(0, 448, 40000) if rise > 0 else np.linspace(448, 0, 40000)
    compare(w12, Shared(w12, 170, G, k0, 6), abs(rise) * math.log(2) / 448, 128 * 128)


@pytest.mark.parametrize("G", [1, 40, 64])
def test_scores_in_steps(w12, G):
    """Plateaus up and down by 2^20 to 2^60, of lengths about the 128 tiles after which references come down."""
    g = np.random.default_rng(7)
    levels, lengths = [256, 0, 128, 448, 16, 0, 320, 64], [300, 33000, 700, 1, 17000, 16500, 2, 9000]
    k0 = np.concatenate([np.full(n, x) + 0.0 for x, n in zip(levels, lengths)])
    k0[g.choice(len(k0), 20, replace=False)] = 224
    compare(w12, Shared(w12, 160, G, k0, 8), 60 * math.log(2) / 448, 128 * 128 * 20)


@pytest.mark.parametrize("G", [1, 40, 64])
@pytest.mark.parametrize("tokens", [1, 100, 300, 5000])
@pytest.mark.parametrize("size", [100.0, 130.0, 1000.0, 20000.0])
def test_scores_far_from_zero(w12, G, tokens, size):
    """Every score is +- size (of log 2) and a little; the row's own key weighs as much as the cached ones, or all or
    nothing next to them."""
    for sign in (1, -1):
        for own in (16.0 * sign, 0.0, -16.0 * sign):
            s = Shared(w12, 3, G, np.full(tokens, 16.0 * sign), 9, own_k0=own)
            compare(w12, s, size * math.log(2) / 16, tokens)


@pytest.mark.parametrize("G", [2, 5, 16])
def test_rising_scores_split_over_ctas(w12, G):
    """A single request, so that a segment's shares meet different parts of the rise, behind the 64-bit form."""
    s = World(w12, [9000, 1], 1, 64, rot=0, seed=31)
    b = s.host["table"][0]
    for i in range(-(-9000 // 64)):
        s.host["k_scale"][b[i]] *= 2.0 ** (i // 40)             # scores grow by 2 every 40 blocks, in both directions
    s.upload()
    t = make_tree(s.g, [3, 2])
    q, k, v, dev = inputs(s.g, 5, 1, G, s)
    close(attend(w12, s, t, dev, 1, G, 2), *ref.tree_attention(s.host, t[0], t[1], t[2], q, k, v, None, None, False, D ** -0.5))
    assert s.ws.status() == 0


# ---------------------------------------------------------------------------
# not numbers
# ---------------------------------------------------------------------------

def world(w12, G, seed):
    s = World(w12, [700, 300], 2, 32, seed=seed)
    t = make_tree(s.g, [4, 3])
    return s, t, inputs(s.g, 7, 2, G, s)


@pytest.mark.parametrize("G", [1, 5, 16])
@pytest.mark.parametrize("token", [0, 150, 699])
def test_a_nan_key(w12, G, token):
    """A NaN among a live token's key codes makes that head of its request NaN, and nothing else."""
    s, t, (q, k, v, dev) = world(w12, G, 32)
    want, slack = ref.tree_attention(s.host, t[0], t[1], t[2], q, k, v, s.cos, s.sin, False, D ** -0.5)
    s.host["k"][s.host["table"][0, token // 32], 1, token % 32, 9] = 0x7F
    s.upload()
    out = attend(w12, s, t, dev, 2, G, 2)
    assert torch.isnan(out[:4, G:]).all()
    close(out[:4, :G], want[:4, :G], slack[:4, :G])
    close(out[4:], want[4:], slack[4:])
    assert s.ws.status() == 0


@pytest.mark.parametrize("G", [1, 5, 16])
@pytest.mark.parametrize("token", [0, 150, 299])
def test_a_nan_value(w12, G, token):
    """A NaN value code reaches its own dimension of its head's outputs."""
    s, t, (q, k, v, dev) = world(w12, G, 33)
    want, slack = ref.tree_attention(s.host, t[0], t[1], t[2], q, k, v, s.cos, s.sin, False, D ** -0.5)
    s.host["v"][s.host["table"][1, token // 32], 0, 77, token % 32] = 0xFF
    s.upload()
    out = attend(w12, s, t, dev, 2, G, 2)
    assert torch.isnan(out[4:, :G, 77]).all()
    out[4:, :G, 77] = 0
    want[4:, :G, 77] = 0
    close(out, want, slack)
    assert s.ws.status() == 0


@pytest.mark.parametrize("G", [1, 5, 16])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_query_that_is_no_number(w12, G, bad):
    """An infinite or NaN query makes its own row's head NaN."""
    s, t, (q, k, v, dev) = world(w12, G, 34)
    want, slack = ref.tree_attention(s.host, t[0], t[1], t[2], q, k, v, s.cos, s.sin, False, D ** -0.5)
    dev[0][2, (G + 0) * D + 5] = bad                             # row 2, the second head's first query
    out = attend(w12, s, t, dev, 2, G, 2)
    assert torch.isnan(out[2, G]).all()
    out[2, G] = 0
    want[2, G] = 0
    close(out, want, slack)
    assert s.ws.status() == 0
