"""The recurrent layer's prompts and single tokens, and the norms around a block: cases and plain forms.

Four entry points, as a serving loop over gated delta rule layers calls them:

* ``w12_gdn_prefill``  the outputs and the state behind whole prompts (or their continuations), many requests at once;
* ``w12_gdn_step``     one new token of every request: its output and the state behind it;
* ``w12_gdn_norm``     the RMS norm of a layer's outputs head by head with its SiLU gate, as the next linear reads it;
* ``w12_block_norm``   a block's output into the residual stream (norm behind the block, residual scale), and the norm
  in front of the next block.

A head's state S [d_v][d_k] follows S <- a S (I - b k k^T) + b v k^T, and a token's output is S q of the new state.
"""
import math
import random

import torch

own = False
DEVICE = "cuda"

D = 128      # head dimension
C = 64       # tokens the plain form takes at once
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _prefill(name, n_req, tok, heads, qk, s0, fused=True, shape=0):
    return dict(name=name, op="prefill", n_req=n_req, tok=tok, heads=heads, qk=qk, s0=s0, fused=fused, shape=shape)


def _step(name, n_req, heads, qk, fused=True, shape=0):
    return dict(name=name, op="step", n_req=n_req, heads=heads, qk=qk, s0=True, fused=fused, shape=shape)


def _gate(name, rows, heads, first=False, shape=0):
    return dict(name=name, op="gate", rows=rows, heads=heads, first=first, shape=shape)


def _block(name, rows, n, f32, post, shape=0):
    return dict(name=name, op="block", rows=rows, n=n, f32=f32, post=post, shape=shape)


def listed():
    return [
        # a short prompt through a small layer: where latency counts
        _prefill("prefill_short", 1, 100, 4, 4, False),
        # one prompt of 2048 tokens, the recurrent layer of the benchmark (32 heads)
        _prefill("prefill_2048", 1, 2048, 32, 32, False),
        # 24 ragged continuations of chunked admission, query and key heads shared by two value heads
        _prefill("prefill_ragged_24", 24, 701, 32, 16, True, shape=1),
        # one very long prompt: a single sequence's latency
        _prefill("prefill_long", 1, 32768, 32, 16, False, fused=False),
        # sixteen prompts of up to 8192 tokens at once: the largest admission
        _prefill("prefill_large", 16, 8192, 32, 32, True, shape=2),
        # plain decoding of one request
        _step("step_single", 1, 32, 32),
        # the 24 requests of the benchmark's batch, shared query and key heads
        _step("step_batch_24", 24, 32, 16, shape=3),
        # a large decode batch
        _step("step_large", 256, 32, 32, fused=False, shape=4),
        # the 192 tree rows of the benchmark's batch
        _gate("gate_tree_192", 192, 32),
        # the rows of a long prompt
        _gate("gate_prompt", 16384, 32, shape=5),
        # the 192 tree rows between two linears of the 27B-like layer
        _block("block_tree_192", 192, 5120, False, False),
        # the rows of a long prompt, a 32-bit residual stream and a norm behind the block as well
        _block("block_prompt", 16384, 5120, True, True, shape=6),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "gate", "block"])
    shape = rng.randrange(1, 1 << 20)
    heads = rng.choice([1, 2, 3, 4, 8, 16, 24, 32])
    qk = rng.choice([g for g in (1, 2, 3, 4, 8, 16, 24, 32) if heads % g == 0 and heads // g <= 8])
    if op == "prefill":
        n_req = _spread(rng, 1, 32)
        tok = min(_spread(rng, 1, 32768), 16 * 8192 // n_req)
        c = _prefill("", n_req, tok, heads, qk, rng.random() < 0.5, rng.random() < 0.5, shape)
    elif op == "step":
        c = _step("", _spread(rng, 1, 256), heads, qk, rng.random() < 0.5, shape)
    elif op == "gate":
        c = _gate("", _spread(rng, 1, 16384), heads, rng.random() < 0.3, shape)
    else:
        c = _block("", _spread(rng, 1, 16384), 8 * _spread(rng, 16, 1024), rng.random() < 0.5, rng.random() < 0.5, shape)
        c["rows"] = min(c["rows"], 16384 * 5120 // c["n"])
    del c["name"]
    return c


def _counts(case):
    """Tokens of the requests: the first has `tok`, the others between a quarter of it and all of it; a step has one each."""
    if case["op"] == "step":
        return [1] * case["n_req"]
    r = random.Random(case["shape"] * 7919 + case["tok"])
    return [case["tok"]] + [max(1, int(case["tok"] * r.uniform(0.25, 1.0))) for _ in range(case["n_req"] - 1)]


def work(case):
    if case["op"] in ("prefill", "step"):
        t, H = sum(_counts(case)), case["heads"]
        state = case["n_req"] * H * D * D * 4 * (2 if case["s0"] else 1)
        rows = t * (2 * case["qk"] * D * 2 + H * (D * 2 + D * 4 + 8))
        return {"bytes": state + rows, "flops": 6 * D * D * t * H}
    if case["op"] == "gate":
        n = case["rows"] * case["heads"] * D
        return {"bytes": n * (4 + 2 + 2), "flops": 8 * n}
    n = case["rows"] * case["n"]
    return {"bytes": n * (2 * (4 if case["f32"] else 2) + 2 + 2), "flops": (12 if case["post"] else 6) * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _unit(x):
    return x / x.square().sum(-1, keepdim=True).sqrt()


def _rows_of(case, g):
    """A recurrent layer's rows: keys and queries of unit norm, keys of one head with a common part as neighbouring
    tokens have, values N(0, 1), gates of every rate from a long memory to a short one, strengths over (0, 1)."""
    H, K, T = case["heads"], case["qk"], sum(_counts(case))
    new = lambda *s: torch.randn(s, generator=g, device=DEVICE)  # noqa: E731
    widths = [K * D, K * D, H * D]
    if case["fused"]:      # slices of one fused linear's rows
        parts = torch.empty(T, sum(widths), dtype=torch.bfloat16, device=DEVICE).split(widths, 1)
    else:
        parts = [torch.empty(T, w, dtype=torch.bfloat16, device=DEVICE) for w in widths]
    common = new(2, K, D) * 0.5
    rate = torch.exp(torch.rand(H, generator=g, device=DEVICE) * 7 - 7)
    alpha = torch.exp(-rate * torch.nn.functional.softplus(new(T, H) + 1))
    beta = torch.sigmoid(new(T, H))
    step = max(1, (1 << 26) // (H * D))
    for i in range(0, T, step):
        m = min(step, T - i)
        for j in range(2):
            parts[j][i:i + m] = _unit(new(m, K, D) + common[j]).reshape(m, K * D).bfloat16()
        parts[2][i:i + m] = new(m, H * D).bfloat16()
    return dict(q=parts[0], k=parts[1], v=parts[2], alpha=alpha, beta=beta)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed * 1000003 + case["shape"])
    s = dict(case=case)
    new = lambda *a: torch.randn(a, generator=g, device=DEVICE)  # noqa: E731
    if case["op"] in ("prefill", "step"):
        cnt, H = _counts(case), case["heads"]
        off = [0]
        for c in cnt:
            off.append(off[-1] + c)
        s.update(_rows_of(case, g), row_off=torch.tensor(off, dtype=torch.int32, device=DEVICE), most=max(cnt))
        s["S0"] = new(case["n_req"], H, D, D) * 0.05 if case["s0"] else None
        if case["op"] == "prefill":   # where each token stands in its request, as a batch's metadata has it
            s["req"] = torch.repeat_interleave(torch.arange(len(cnt), device=DEVICE), torch.tensor(cnt, device=DEVICE))
            s["pos"] = torch.arange(off[-1], device=DEVICE) - s["row_off"].long()[s["req"]]
    elif case["op"] == "gate":
        R, H = case["rows"], case["heads"]
        scale = torch.exp(torch.randn(R, H, 1, generator=g, device=DEVICE) - 1)    # outputs of small and large states
        s.update(o=new(R, H, D) * scale, z=(new(R, H * D) * 2).bfloat16(), weight=(1 + 0.2 * new(D)).bfloat16())
    else:
        R, n = case["rows"], case["n"]
        h = new(R, n) * 3
        s.update(h=h if case["f32"] else h.bfloat16(), y=new(R, n).bfloat16(), pre=(1 + 0.2 * new(n)).bfloat16(),
                 post=(1 + 0.2 * new(n)).bfloat16() if case["post"] else None, scale=0.25 if case["post"] else 1.0)
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a serving loop keeps between calls: the layer's rows, the workspace and the output buffers."""
    import speculative_decoding_tree_w12_gb300 as w12
    case = s["case"]
    new = lambda *a, dtype=torch.float32: torch.empty(a, dtype=dtype, device=DEVICE)  # noqa: E731
    if case["op"] in ("prefill", "step"):
        s["rows"] = w12.GdnRows(s["q"], s["k"], s["v"], s["alpha"], s["beta"])
        s["out"] = new(s["alpha"].shape[0], case["heads"], D)
        s["state"] = new(case["n_req"], case["heads"], D, D)
        s["ws"] = w12.Workspace(1, 0, 0, case["n_req"])
    elif case["op"] == "gate":
        s["x"] = new(case["rows"], case["heads"] * D, dtype=torch.bfloat16)
    else:
        s["x"], s["h_out"] = new(case["rows"], case["n"], dtype=torch.bfloat16), torch.empty_like(s["h"])


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _heads32(s):
    """q, k, v [T][H][D] in 32 bits, shared query and key heads repeated."""
    H, K = s["case"]["heads"], s["case"]["qk"]
    of = torch.arange(H, device=DEVICE) // (H // K)
    q, k = (s[x].reshape(-1, K, D)[:, of].float() for x in "qk")
    return q, k, s["v"].reshape(-1, H, D).float()


def _plain_prefill(s):
    """C tokens at once: with the gates' products G_i from the chunk's start and D_ij from token j to i,
    (1 + L) U = b (V - G K S^T), L_ij = b_i D_ij k_i.k_j (j < i);  O = G Q S^T + (D_ij q_i.k_j) U (j <= i);
    S' = G_C S + sum D_Cj u_j k_j^T.  Tokens past a request's end have b = 0 and a = 1."""
    case, n, H = s["case"], s["case"]["n_req"], s["case"]["heads"]
    nc = -(-s["most"] // C)
    at = s["req"] * (nc * C) + s["pos"]

    def padded(x, fill=0.0):
        y = torch.full((n * nc * C,) + x.shape[1:], fill, device=DEVICE)
        y[at] = x
        return y.reshape((n, nc, C) + x.shape[1:]).transpose(2, 3)     # [n][chunk][H][token]...

    q, k, v = _heads32(s)
    q, k, v = padded(q), padded(k), padded(v)
    a, b = padded(s["alpha"][..., None], 1.0)[..., 0], padded(s["beta"][..., None])
    g = a.double().log().cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device=DEVICE).tril()
    d = torch.where(low, g[..., :, None] - g[..., None, :], -math.inf).exp().float()
    kt = k.transpose(-1, -2)
    m = -(b * d * torch.matmul(k, kt)).tril(-1)                        # (1 + L)^-1 = (1 - L)(1 + L^2)(1 + L^4)...
    inv = torch.eye(C, device=DEVICE) + m
    for _ in range(5):
        m = torch.matmul(m, m)
        inv = inv + torch.matmul(inv, m)
    att = d * torch.matmul(q, kt)
    gate, tail, last = g.exp().float()[..., None], d[..., -1, :, None], g[..., -1].exp().float()[..., None, None]
    S = s["S0"].clone() if s["S0"] is not None else torch.zeros(n, H, D, D, device=DEVICE)
    out = torch.empty_like(v)
    for c in range(nc):        # each chunk starts from the state behind the one before it
        St = S.transpose(-1, -2)
        u = torch.matmul(inv[:, c], b[:, c] * (v[:, c] - gate[:, c] * torch.matmul(k[:, c], St)))
        out[:, c] = gate[:, c] * torch.matmul(q[:, c], St) + torch.matmul(att[:, c], u)
        S = last[:, c] * S + torch.matmul((tail[:, c] * u).transpose(-1, -2), k[:, c])
    return dict(o=out.transpose(2, 3).reshape(n * nc * C, H, D)[at], state=S)


def _plain_step(s):
    q, k, v = _heads32(s)
    a, b = s["alpha"][..., None], s["beta"][..., None]
    u = b * (v - a * (s["S0"] * k[:, :, None, :]).sum(-1))
    S = a[..., None] * s["S0"] + u[..., None] * k[:, :, None, :]
    return dict(o=(S * q[:, :, None, :]).sum(-1), state=S)


def _rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain_gate(s):
    z = s["z"].float().reshape(s["o"].shape)
    gate = z / (1 + (-z).exp())
    y = _rms(s["o"] * gate) * s["weight"].float() if s["case"]["first"] else _rms(s["o"]) * s["weight"].float() * gate
    return dict(x=y.reshape(s["z"].shape).bfloat16())


def _plain_block(s):
    y = s["y"].float()
    if s["post"] is not None:
        y = _rms(y) * s["post"].float()
    h = s["h"].float() + s["scale"] * y
    return dict(h=h.to(s["h"].dtype), x=(_rms(h) * s["pre"].float()).bfloat16())


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return dict(prefill=_plain_prefill, step=_plain_step, gate=_plain_gate, block=_plain_block)[op](s)
    import speculative_decoding_tree_w12_gb300 as w12
    if op == "prefill":
        w12.w12_gdn_prefill(s["rows"], s["row_off"], s["ws"], S0=s["S0"], state=s["state"], out=s["out"])
        return dict(o=s["out"], state=s["state"])
    if op == "step":
        w12.w12_gdn_step(s["rows"], S0=s["S0"], state=s["state"], out=s["out"])
        return dict(o=s["out"], state=s["state"])
    if op == "gate":
        return dict(x=w12.w12_gdn_norm(s["o"], s["weight"], z=s["z"], eps=EPS, gate_first=s["case"]["first"], out=s["x"]))
    h, x = w12.w12_block_norm(s["h"], s["y"], pre=s["pre"], post=s["post"], scale=s["scale"], eps=EPS, h_out=s["h_out"],
                              out=s["x"])
    return dict(h=h, x=x)


# ---------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------

def _exact_tokens(s):
    """Token by token, all requests that still have one at once."""
    case, n, H = s["case"], s["case"]["n_req"], s["case"]["heads"]
    group, off, cnt = H // case["qk"], s["row_off"].tolist(), _counts(case)
    S = s["S0"].double() if s["S0"] is not None else torch.zeros(n, H, D, D, dtype=torch.float64, device=DEVICE)
    o = torch.empty(off[-1], H, D, dtype=torch.float64, device=DEVICE)
    order = sorted(range(n), key=lambda r: -cnt[r])
    first = torch.tensor([off[r] for r in order], device=DEVICE)
    S = S[torch.tensor(order, device=DEVICE)].clone()
    live = n
    for t in range(cnt[order[0]]):
        while cnt[order[live - 1]] <= t:
            live -= 1
        rows = first[:live] + t
        q, k = (s[x][rows].double().reshape(live, -1, D).repeat_interleave(group, 1)[..., None] for x in "qk")
        v = s["v"][rows].double().reshape(live, H, D, 1)
        a, b = (s[x][rows].double()[..., None, None] for x in ("alpha", "beta"))
        T = S[:live]
        T *= a
        T += torch.matmul(b * (v - torch.matmul(T, k)), k.transpose(-1, -2))
        o[rows] = torch.matmul(T, q)[..., 0]
    back = torch.empty_like(S)
    back[torch.tensor(order, device=DEVICE)] = S
    return dict(o=o, state=back)


def _normed64(x, w):
    return x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) ** 0.5 * w.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("prefill", "step"):
        return _exact_tokens(s)
    if case["op"] == "gate":
        o, z = s["o"].double(), s["z"].double().view(s["o"].shape)
        silu = z * torch.sigmoid(z)
        y = _normed64(o * silu, s["weight"]) if case["first"] else _normed64(o, s["weight"]) * silu
        return dict(x=y.flatten(1))
    y = s["y"].double()
    h = s["h"].double() + s["scale"] * (y if s["post"] is None else _normed64(y, s["post"]))
    return dict(h=h, x=_normed64(h, s["pre"]))
