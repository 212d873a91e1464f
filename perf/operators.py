"""The attention and sampling operators of the verify pass: cases and plain forms.

Four entry points, as a decode loop with an attention layer calls them:

* ``w12_kv_append``          prompt rows into the paged 8-bit cache, rotated on the way;
* ``w12_kv_commit``          the accepted path of a draft tree into the cache;
* ``w12_tree_attention``     the tree rows' attention over the cache and their own root paths;
* ``w12_tree_verify_sampled`` acceptance against the target's probabilities from given random numbers.

The cache holds E4M3 codes: keys ``[block][head][token][d]``, values transposed ``[block][head][d][token]``,
and one power-of-two scale per block and head for each of the two.
"""
import math
import random

import torch

own = False
DEVICE = "cuda"

D = 128            # head dimension
TOP = 448.0        # largest E4M3 value
LOW = -32          # least exponent of a block's scale
FIX = 2.0 ** 40    # fixed-point unit of the sampling weights


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _append(name, n_req, tok, ctx, heads, block, rot=D, pairs="halves", shape=0):
    return dict(name=name, op="append", n_req=n_req, tok=tok, ctx=ctx, heads=heads, block=block, rot=rot, pairs=pairs,
                shape=shape)


def _tree(name, op, n_req, rows, ctx, heads, group, block, rot=D, pairs="halves", chain=False, shape=0):
    return dict(name=name, op=op, n_req=n_req, rows=rows, ctx=ctx, heads=heads, group=group, block=block, rot=rot,
                pairs=pairs, chain=chain, shape=shape)


def _sample(name, n_req, rows, vocab, f32, draft, chain=False, shape=0):
    return dict(name=name, op="sample", n_req=n_req, rows=rows, vocab=vocab, f32=f32, draft=draft, chain=chain, shape=shape)


def listed():
    return [
        # one prompt of 2048 tokens into an empty cache: first admission of a single request, 27B-like heads
        _append("append_prompt_2048", 1, 2048, 0, 8, 64),
        # 24 ragged continuations behind ragged contexts, partial rotation: chunked admission while others decode
        _append("append_ragged_24", 24, 701, 1003, 4, 32, rot=64, pairs="adjacent", shape=1),
        # sixteen prompts of up to 8192 tokens at once: the largest admission
        _append("append_large", 16, 8192, 0, 8, 128, shape=2),
        # plain decoding of one request: one token per step
        _tree("commit_single", "commit", 1, 1, 1000, 8, 5, 64, chain=True),
        # the 192-node batch of 24 requests after acceptance
        _tree("commit_batch_24", "commit", 24, 192, 4099, 8, 5, 64, shape=3),
        # plain decoding of one request behind a short context: where latency counts
        _tree("attend_short", "attend", 1, 1, 200, 4, 5, 64, chain=True),
        # the 32-node tree of one request behind a long context
        _tree("attend_tree_32", "attend", 1, 32, 32771, 8, 5, 64),
        # plain decoding behind a very long context
        _tree("attend_long", "attend", 1, 1, 131072, 8, 5, 128, chain=True),
        # 32 requests sharing 256 nodes behind ragged contexts of up to 16384 tokens: the largest step
        _tree("attend_batch_32", "attend", 32, 256, 16384, 8, 5, 64, shape=4),
        # plain sampled decoding of one request
        _sample("sample_single", 1, 1, 151936, False, False, chain=True),
        # the 192-node batch of 24 requests, a drafter that picks its candidates deterministically
        _sample("sample_batch_24", 24, 192, 151936, False, False, shape=5),
        # 32 chains of 8 sampled drafts each, with the drafter's own probabilities, 32-bit logits
        _sample("sample_draft_32", 32, 256, 151936, True, True, shape=6),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "commit", "attend", "attend", "sample", "sample"])
    shape = rng.randrange(1, 1 << 20)
    block, heads = rng.choice([32, 64, 128]), rng.choice([1, 2, 4, 8])
    rot, pairs = rng.choice([D, D, 64, 32, 0]), rng.choice(["halves", "adjacent"])
    n_req = _spread(rng, 1, 32)
    if op == "append":
        c = _append("", n_req, min(_spread(rng, 1, 8192), 65536 // n_req), rng.choice([0, _spread(rng, 1, 4096)]), heads,
                    block, rot, pairs, shape)
    elif op == "sample":
        rows = n_req * _spread(rng, 1, 8)
        c = _sample("", n_req, rows, _spread(rng, 1000, 151936), rng.random() < 0.5, rng.random() < 0.5,
                    rng.random() < 0.3, shape)
    else:
        rows = min(n_req * _spread(rng, 1, 32), 256)
        ctx = min(_spread(rng, 1, 131072), 24 * 16384 // n_req)
        c = _tree("", op, n_req, rows, ctx if op == "attend" else min(ctx, 8192), heads, rng.choice([1, 4, 5, 8]), block, rot,
                  pairs, rng.random() < 0.3, shape)
    del c["name"]
    return c


def _ragged(case, top, least):
    """Lengths of the requests: the first has `top`, the others between a quarter of it and all of it."""
    r = random.Random(case["shape"] * 7919 + top)
    return [top] + [max(least, int(top * r.uniform(0.25, 1.0))) for _ in range(case["n_req"] - 1)]


def _parents(case):
    """Rows per request and each row's parent (in the whole tree): chains, or trees at most 16 deep whose later rows
    hang under random earlier ones."""
    n, rows = case["n_req"], case["rows"]
    r = random.Random(case["shape"] * 104729 + rows)
    share = [1] * n
    for i in range(rows - n):
        share[r.randrange(n) if case["shape"] and not case["chain"] else i % n] += 1
    parent, depth, req, off = [], [], [], [0]
    for q in range(n):
        base = len(parent)
        for j in range(share[q]):
            if j == 0:
                parent.append(-1)
                depth.append(0)
            else:
                p = len(parent) - 1 if case["chain"] else base + r.randrange(j)
                if depth[p] >= 16:
                    p = base
                parent.append(p)
                depth.append(depth[p] + 1)
            req.append(q)
        off.append(len(parent))
    return parent, depth, req, off


def work(case):
    if case["op"] == "append":
        t = sum(_ragged(case, case["tok"], 1)) * case["heads"] * D
        return {"bytes": 2 * t * 2 + 2 * t, "flops": 6 * t}
    if case["op"] == "commit":
        _, depth, req, off = _parents(case)
        t = sum(depth[j] + 1 for j in _accepted(case, depth, off)) * case["heads"] * D
        return {"bytes": 2 * t * 2 + 2 * t, "flops": 6 * t}
    if case["op"] == "attend":
        _, depth, req, _ = _parents(case)
        lens = _ragged(case, case["ctx"], 0)
        hq = case["heads"] * case["group"]
        kv = sum(lens) * case["heads"] * 2 * D + 2 * 4 * case["heads"] * sum(-(-x // case["block"]) for x in lens)
        rows = len(req) * D * 2 * (2 * hq + 2 * case["heads"])
        keys = sum(lens[q] + d + 1 for q, d in zip(req, depth))
        return {"bytes": kv + rows, "flops": 4 * D * hq * keys}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (4 if case["f32"] else 2) + (4 * n if case["draft"] else 0), "flops": 8 * n}


def _accepted(case, depth, off):
    """The row each request ends on after acceptance: a random one of its rows."""
    r = random.Random(case["shape"] * 31 + 5)
    return [r.randrange(off[q], off[q + 1]) for q in range(case["n_req"])]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEVICE)


def _tables(case, n_pos):
    """cos and sin of every position and frequency, computed in 64 bits as a model's loader does."""
    half = case["rot"] // 2
    if half == 0:
        return None, None
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEVICE) / half)
    a = torch.arange(n_pos, dtype=torch.float64, device=DEVICE)[:, None] * freq
    return a.cos().float(), a.sin().float()


def _cache(case, lens, room, g):
    """A cache whose requests hold `lens` tokens in blocks scattered over the pool, with `room` more tokens each."""
    bt, H = case["block"], case["heads"]
    need = [-(-(x + m) // bt) for x, m in zip(lens, room)]
    n_blocks = sum(need) + 3
    order = torch.randperm(n_blocks, generator=torch.Generator().manual_seed(case["shape"])).tolist()
    table = torch.zeros(len(lens), max(max(need), 1), dtype=torch.int32)
    at = 0
    for q, m in enumerate(need):
        table[q, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
        at += m
    codes = []
    for shape in ((bt, D), (D, bt)):
        c = torch.empty((n_blocks, H) + shape, dtype=torch.uint8, device=DEVICE)
        for i in range(0, n_blocks, 1024):   # values N(0, 1) under scales that leave them up to a factor of 2 below the top
            x = torch.randn(c[i:i + 1024].shape, generator=g, device=DEVICE) * 80
            c[i:i + 1024] = x.clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)
        codes.append(c)
    ones = torch.ones(n_blocks, H, device=DEVICE)
    scales = [torch.ldexp(ones, torch.randint(-7, -5, (n_blocks, H), generator=g, device=DEVICE)) for _ in range(2)]
    return dict(k=codes[0], v=codes[1], k_scale=scales[0], v_scale=scales[1], table=table.to(DEVICE), len=_i32(lens))


def _logits(rows, vocab, g):
    """Rows of a language model's logits: a broad floor and a handful of likely tokens."""
    z = torch.randn(rows, vocab, generator=g, device=DEVICE) * 2
    hot = torch.randint(0, vocab, (rows, 12), generator=g, device=DEVICE)
    lift = torch.rand(rows, 12, generator=g, device=DEVICE) * 8 + 6
    return z.scatter_add_(1, hot, lift)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed * 1000003 + case["shape"])
    s = dict(case=case)
    n = case["n_req"]
    if case["op"] == "append":
        lens, cnt = _ragged(case, case["ctx"], 0), _ragged(case, case["tok"], 1)
        off = [0]
        for c in cnt:
            off.append(off[-1] + c)
        s.update(_cache(case, lens, cnt, g), row_off=_i32(off), n_tok=off[-1])
        s["cos"], s["sin"] = _tables(case, max(a + b for a, b in zip(lens, cnt)))
        w = case["heads"] * D
        qkv = torch.randn(off[-1], 2 * w, generator=g, device=DEVICE).bfloat16()   # as the key and value linears leave them
        s["kx"], s["vx"] = qkv[:, :w], qkv[:, w:]
    else:
        parent, depth, req, off = _parents(case)
        R = len(req)
        paths = []
        for j in range(R):
            paths.append((paths[parent[j]] if parent[j] >= 0 else []) + [j])
        s.update(parent=_i32(parent), depth=torch.tensor(depth, dtype=torch.uint8, device=DEVICE), req=_i32(req),
                 row_off=_i32(off), path=_i32([p + [-1] * (17 - len(p)) for p in paths]), p_max=16)
        if case["op"] in ("commit", "attend"):
            lens = _ragged(case, case["ctx"], 0)
            s.update(_cache(case, lens, [17] * n, g))
            s["cos"], s["sin"] = _tables(case, max(lens) + 17)
            w = case["heads"] * D
            wq = w * case["group"]
            qkv = torch.randn(R, wq + 2 * w, generator=g, device=DEVICE)
            qkv[:, :wq] *= 2
            qkv = qkv.bfloat16()   # one fused linear's rows
            s["q"], s["kx"], s["vx"] = qkv[:, :wq], qkv[:, wq:wq + w], qkv[:, wq + w:]
            s["acc_node"] = _i32(_accepted(case, depth, off))
            s["max_len"] = max(lens)
        else:
            V = case["vocab"]
            z = _logits(R, V, g)
            draft = torch.softmax(z + torch.randn(R, V, generator=g, device=DEVICE), 1)
            kids = [[] for _ in range(R)]
            for j, p in enumerate(parent):
                if p >= 0:
                    kids[p].append(j)
            most = max(1, max(len(k) for k in kids))
            pick = torch.multinomial(draft, most, replacement=True, generator=g) if case["draft"] else draft.topk(most, 1)[1]
            token = torch.randint(0, V, (R,), generator=g, device=DEVICE)
            for p in range(R):
                if kids[p]:
                    token[kids[p]] = pick[p, :len(kids[p])]
            s.update(token=token.int(), kids=_i32([k + [-1] * (most - len(k)) for k in kids]),
                     logits=z if case["f32"] else z.bfloat16(), draft=draft if case["draft"] else None,
                     temp=torch.rand(n, generator=g, device=DEVICE) * 0.6 + 0.6,
                     u_accept=torch.rand(R, generator=g, device=DEVICE), u_sample=torch.rand(R, generator=g, device=DEVICE))
            if n > 2:
                s["temp"][1] = 0   # a greedy request among the sampled ones
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a decode loop keeps between calls: the cache's, tree's and workspaces' handles and its output buffers."""
    import speculative_decoding_tree_w12_gb300 as w12
    case, n = s["case"], s["case"]["n_req"]
    new = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device=DEVICE)  # noqa: E731
    s["ws"] = w12.Workspace(1, 0, 0, n)
    if case["op"] != "append":
        s["tree"] = w12.DeviceTree.from_arrays(s["parent"], s["depth"], s["req"], s["row_off"], token=s.get("token"))
    if case["op"] == "sample":
        R = case["rows"]
        s["dist"] = w12.SampleRows(s["logits"], s["u_sample"], temperature=s["temp"], draft_p=s["draft"], u_accept=s["u_accept"])
        s["out"] = (new(n, s["p_max"] + 1), new(n), new(n), new(R), new(R, dtype=torch.float32))
    else:
        s["cache"] = w12.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["len"])
        s["rope"] = w12.Rope(s["cos"], s["sin"], adjacent=case["pairs"] == "adjacent") if case["rot"] else None
        s["len_out"] = new(n)
        if case["op"] == "attend":
            s["aws"] = w12.AttentionWorkspace(case["rows"], case["heads"] * case["group"], case["heads"], n)
            s["out"] = new(case["rows"], case["heads"] * case["group"], D, dtype=torch.bfloat16)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rotate(s, x, pos):
    """x [T][H][d] in 32 bits, turned by its position: pairs (i, i + rot/2), or (2 i, 2 i + 1)."""
    rot = s["case"]["rot"]
    if rot == 0:
        return x
    c, n = s["cos"][pos][:, None, :], s["sin"][pos][:, None, :]
    if s["case"]["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * c - b * n, b * c + a * n, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    y = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _scale_of(top):
    """The least power of two s with top <= 448 s, not under 2^-32."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=LOW)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), torch.full_like(top, 2.0 ** LOW))


def _codes(x):
    x = torch.where(torch.isfinite(x), x, torch.full_like(x, math.nan))
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _write(s, req, j, kx, vx):
    """Tokens j of request req behind its context: the two pools, their scales and the lengths, in place."""
    case, bt = s["case"], s["case"]["block"]
    H, n = case["heads"], case["n_req"]
    lens = s["len"].long()
    pos = lens[req] + j
    blk, slot = s["table"][req, pos // bt].long(), pos % bt
    k = _rotate(s, kx.reshape(-1, H, D).float(), pos)
    v = vx.reshape(-1, H, D).float()
    touched = torch.zeros(s["k"].shape[0], dtype=torch.bool, device=DEVICE)
    touched[blk] = True
    part = lens % bt                                   # tokens already in each request's last block
    last = s["table"].long().gather(1, (lens // bt).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0]
    held = torch.zeros(s["k"].shape[0], dtype=torch.long, device=DEVICE)
    held[last] = part
    held = torch.where(touched, held, 0)
    for name, x in (("k", k), ("v", v)):
        pool, scale = s[name], s[name + "_scale"]
        top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
        need = torch.zeros_like(scale).scatter_reduce(0, blk[:, None].expand(-1, H), top, "amax")
        need = _scale_of(need)
        now = torch.where(held[:, None] > 0, torch.maximum(scale, need), need)
        now = torch.where(touched[:, None], now, scale)
        pb = last[touched[last] & (part > 0)]          # blocks that already held tokens
        old = pool[pb].view(torch.float8_e4m3fn).float() * (scale[pb] / now[pb])[..., None, None]
        at = torch.arange(bt, device=DEVICE) < held[pb][:, None]
        at = at[:, None, :, None] if name == "k" else at[:, None, None, :]
        pool[pb] = torch.where(at, _codes(old), pool[pb])
        code = _codes(x / now[blk][..., None])
        if name == "k":
            pool[blk, :, slot] = code
        else:
            pool[blk, :, :, slot] = code
        scale.copy_(now)
    new = torch.zeros(n, dtype=torch.long, device=DEVICE).scatter_add(0, req, torch.ones_like(req))
    return _cache_out(s, (lens + new).int())


def _cache_out(s, lens):
    f8 = torch.float8_e4m3fn
    return dict(k=s["k"].view(f8), v=s["v"].view(f8), k_scale=s["k_scale"], v_scale=s["v_scale"], len=lens)


def _plain_append(s):
    off = s["row_off"].long()
    req = torch.repeat_interleave(torch.arange(s["case"]["n_req"], device=DEVICE), off[1:] - off[:-1], output_size=s["n_tok"])
    return _write(s, req, torch.arange(s["n_tok"], device=DEVICE) - off[req], s["kx"], s["vx"])


def _plain_commit(s):
    path = s["path"][s["acc_node"].long()].long()
    req, j = torch.nonzero(path >= 0, as_tuple=True)
    rows = path[req, j]
    return _write(s, req, j, s["kx"][rows], s["vx"][rows])


def _plain_attend(s):
    case = s["case"]
    H, G, bt, n, R = case["heads"], case["group"], case["block"], case["n_req"], case["rows"]
    lens, req, off = s["len"].long(), s["req"].long(), s["row_off"].long()
    pos = lens[req] + s["depth"].long()
    q = _rotate(s, s["q"].reshape(R, H * G, D).float(), pos).reshape(R, H, G, D) * D ** -0.5
    kt = _rotate(s, s["kx"].reshape(R, H, D).float(), pos)
    vt = s["vx"].reshape(R, H, D).float()
    L = s["max_len"]
    nb = -(-L // bt)
    blocks = s["table"][:, :nb].long()
    k = s["k"][blocks].view(torch.float8_e4m3fn).float() * s["k_scale"][blocks][..., None, None]     # [n][nb][H][bt][D]
    k = k.permute(0, 2, 1, 3, 4).reshape(n, H, nb * bt, D)
    v = s["v"][blocks].view(torch.float8_e4m3fn).float() * s["v_scale"][blocks][..., None, None]     # [n][nb][H][D][bt]
    v = v.permute(0, 2, 1, 4, 3).reshape(n, H, nb * bt, D)
    dead = torch.arange(nb * bt, device=DEVICE) >= lens[:, None]                                      # [n][nb * bt]
    v = v.masked_fill(dead[:, None, :, None], 0.0)
    most = int((off[1:] - off[:-1]).max())
    at = torch.arange(R, device=DEVICE) - off[req]
    qs = torch.zeros(n, most, H, G, D, device=DEVICE)
    qs[req, at] = q
    qs = qs.permute(0, 2, 1, 3, 4).reshape(n, H, most * G, D)
    sc = torch.matmul(qs, k.transpose(2, 3)).masked_fill(dead[:, None, None, :], -math.inf)
    sc = sc.reshape(n, H, most, G, nb * bt).permute(0, 2, 1, 3, 4)[req, at]                           # [R][H][G][nb * bt]
    path = s["path"].long()
    anc = torch.zeros(R, R + 1, dtype=torch.bool, device=DEVICE).scatter(1, torch.where(path < 0, R, path), True)[:, :R]
    st = torch.einsum("rhgd,jhd->rhgj", q, kt).masked_fill(~anc[:, None, None, :], -math.inf)
    m = torch.maximum(st.amax(-1), sc.amax(-1)) if nb else st.amax(-1)
    pt, pc = (st - m[..., None]).exp(), (sc - m[..., None]).exp()
    total = pt.sum(-1) + pc.sum(-1)
    ps = torch.zeros(n, most, H, G, nb * bt, device=DEVICE)
    ps[req, at] = pc
    oc = torch.matmul(ps.permute(0, 2, 1, 3, 4).reshape(n, H, most * G, nb * bt), v)
    oc = oc.reshape(n, H, most, G, D).permute(0, 2, 1, 3, 4)[req, at]
    o = (oc + torch.einsum("rhgj,jhd->rhgd", pt, vt)) / total[..., None]
    return o.reshape(R, H * G, D).bfloat16()


def _fixed(a):
    return (a * FIX).to(torch.int64)


def _plain_sample(s):
    case, R = s["case"], s["case"]["rows"]
    token, kids = s["token"].long(), s["kids"].long()
    t = s["temp"][s["req"].long()]
    z = s["logits"].float()
    z = torch.where(torch.isnan(z), -math.inf, z)
    ids = torch.arange(case["vocab"], device=DEVICE)
    top = torch.where(z == z.amax(1, keepdim=True), ids, case["vocab"]).amin(1, keepdim=True)
    greedy = torch.full_like(z, -math.inf).scatter(1, top, 0.0)
    z = torch.where(t[:, None] > 0, z * (1 / t)[:, None], greedy)
    m = z.amax(1, keepdim=True)
    a = torch.where(z == m, 1.0, (z - m).exp())
    w = _fixed(a)
    total = w.sum(1)
    first = total.float() / FIX
    accepted = torch.full((R,), -1, dtype=torch.long, device=DEVICE)
    if case["draft"]:
        for c in range(kids.shape[1]):     # each round needs the one before it
            kid = kids[:, c]
            x = token[kid.clamp(min=0)][:, None]
            inv = 1 / (total.float() / FIX)
            live = (kid >= 0) & (accepted < 0)
            yes = s["u_accept"][kid.clamp(min=0)] * s["draft"].gather(1, x)[:, 0] < a.gather(1, x)[:, 0] * inv
            accepted = torch.where(live & yes, kid, accepted)
            rest = (a * inv[:, None] - s["draft"]).clamp(min=0)
            left = _fixed(rest)
            sums = left.sum(1)
            turn = live & ~yes & (sums > 0)
            a, w = torch.where(turn[:, None], rest, a), torch.where(turn[:, None], left, w)
            total = torch.where(turn, sums, total)
    at = (s["u_sample"].double() * total.double()).to(torch.int64)
    at = torch.minimum(at, total - 1)
    drawn = (w.cumsum(1) <= at[:, None]).sum(1)
    if case["draft"]:
        tok = torch.where(accepted >= 0, token[accepted.clamp(min=0)], drawn)
    else:
        tok = drawn
        same = (kids >= 0) & (token[kids.clamp(min=0)] == drawn[:, None])
        accepted = torch.where(same.any(1), torch.where(same, kids, R).amin(1), accepted)
    logp = z.gather(1, tok[:, None])[:, 0] - m[:, 0] - first.log()
    # a row stands if every row on its root path was accepted at its parent; the deepest one that stands ends the path
    path, parent, n = s["path"].long(), s["parent"].long(), case["n_req"]
    taken = (parent < 0) | (accepted[parent.clamp(min=0)] == torch.arange(R, device=DEVICE))
    stands = (taken[path.clamp(min=0)] | (path < 0)).all(1)
    score = torch.where(stands, s["depth"].long(), -1)
    best = torch.full((n,), -1, dtype=torch.long, device=DEVICE).scatter_reduce(0, s["req"].long(), score, "amax")
    end = torch.zeros(n, dtype=torch.long, device=DEVICE)
    is_end = stands & (score == best[s["req"].long()])
    end[s["req"].long()[is_end]] = torch.nonzero(is_end)[:, 0]
    line = torch.cat([path[end][:, 1:], torch.full((n, 1), -1, device=DEVICE)], 1)
    acc = torch.where(line >= 0, token[line.clamp(min=0)], -1)
    acc.scatter_(1, best[:, None], tok[end][:, None])
    return dict(tok=acc.int(), len=(best + 1).int(), node=end.int(), row_tok=tok.int(), row_logp=logp)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return dict(append=_plain_append, commit=_plain_commit, attend=_plain_attend, sample=_plain_sample)[op](s)
    import speculative_decoding_tree_w12_gb300 as w12
    n = s["case"]["n_req"]
    if op == "append":
        w12.w12_kv_append(s["cache"], s["rope"], s["kx"], s["vx"], s["row_off"], s["ws"], len_out=s["len_out"])
        return _cache_out(s, s["len_out"])
    if op == "commit":
        w12.w12_kv_commit(s["cache"], s["rope"], s["tree"], n, s["acc_node"], s["kx"], s["vx"], s["ws"], len_out=s["len_out"])
        return _cache_out(s, s["len_out"])
    if op == "attend":
        return w12.w12_tree_attention(s["cache"], s["rope"], s["tree"], n, s["q"], s["kx"], s["vx"], s["ws"], s["aws"],
                                      out=s["out"])
    tok, length, node, row_tok, row_logp = s["out"]
    w12.w12_tree_verify_sampled(s["dist"], s["tree"], n, s["p_max"], s["ws"], row_tok, row_logp, tok, length, node)
    return dict(tok=tok, len=length, node=node, row_tok=row_tok, row_logp=row_logp)


# ---------------------------------------------------------------------------
# the same in 64 bits
# ---------------------------------------------------------------------------

def _turn64(s, x, pos):
    rot, x = s["case"]["rot"], x.double().clone()
    if rot:
        i = torch.arange(rot // 2, device=DEVICE)
        lo, hi = (i, i + rot // 2) if s["case"]["pairs"] == "halves" else (2 * i, 2 * i + 1)
        ang = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None, :]
        z = torch.complex(x[..., lo], x[..., hi]) * ang
        x[..., lo], x[..., hi] = z.real, z.imag
    return x


def _round8(y):
    """Nearest E4M3 value (ties to even) of 64-bit values within its range."""
    step = torch.ldexp(torch.ones_like(y), (torch.frexp(y)[1] - 4).clamp(min=-9))
    return torch.round(y / step) * step


def _exact_write(s, req, j, rows):
    """The pools token by token: blocks fill up in order, each with the scale its largest value needs."""
    case, bt, H = s["case"], s["case"]["block"], s["case"]["heads"]
    lens, table = s["len"].tolist(), s["table"].tolist()
    pos = s["len"].long()[req] + j
    new = {"k": _turn64(s, s["kx"][rows].reshape(-1, H, D), pos), "v": s["vx"][rows].reshape(-1, H, D).double()}
    out = {x: s[x].view(torch.float8_e4m3fn).double() for x in ("k", "v")}
    out.update({x + "_scale": s[x + "_scale"].double() for x in ("k", "v")})
    count = torch.bincount(req, minlength=case["n_req"]).tolist()
    first = 0
    for r, c in enumerate(count):
        at = lens[r]
        while at < lens[r] + c:
            upto = min((at // bt + 1) * bt, lens[r] + c)
            b, lo, hi = table[r][at // bt], at % bt, upto - at // bt * bt
            for x in ("k", "v"):
                y = new[x][first + at - lens[r]:first + upto - lens[r]].transpose(0, 1)          # [H][tokens][D]
                top = y.abs().amax((1, 2))
                e = torch.ceil(torch.log2(top / TOP)).clamp(min=LOW)
                e = torch.where(torch.ldexp(torch.full_like(top, TOP), e - 1) >= top, e - 1, e).clamp(min=LOW)
                sc = torch.ldexp(torch.ones_like(top), e)
                pool = out[x][b] if x == "k" else out[x][b].transpose(1, 2)                      # [H][bt][D]
                if lo:
                    sc = torch.maximum(sc, out[x + "_scale"][b])
                    pool[:, :lo] = _round8(pool[:, :lo] * (out[x + "_scale"][b] / sc)[:, None, None])
                pool[:, lo:hi] = _round8(y / sc[:, None, None])
                out[x + "_scale"][b] = sc
            at = upto
        first += c
    return dict(out, len=None)


def _exact_attend(s):
    case = s["case"]
    H, G, bt = case["heads"], case["group"], case["block"]
    lens, off, req = s["len"].tolist(), s["row_off"].tolist(), s["req"].long()
    R = case["rows"]
    pos = s["len"].long()[req] + s["depth"].long()
    q = _turn64(s, s["q"].reshape(R, H * G, D), pos).reshape(R, H, G, D)
    kt, vt = _turn64(s, s["kx"].reshape(R, H, D), pos), s["vx"].reshape(R, H, D).double()
    out = torch.empty(R, H, G, D, dtype=torch.float64, device=DEVICE)
    for r, n in enumerate(lens):
        b = s["table"][r, :-(-n // bt)].long()
        mine = slice(off[r], off[r + 1])
        path = s["path"][mine].long() - off[r]
        m = off[r + 1] - off[r]
        anc = torch.zeros(m, m + 1, dtype=torch.bool, device=DEVICE).scatter(1, torch.where(path < 0, m, path), True)[:, :m]
        for h in range(H):
            kc = (s["k"][b, h].view(torch.float8_e4m3fn).double() * s["k_scale"][b, h].double()[:, None, None]).reshape(-1, D)[:n]
            vc = (s["v"][b, h].view(torch.float8_e4m3fn).double() * s["v_scale"][b, h].double()[:, None, None])
            vc = vc.transpose(1, 2).reshape(-1, D)[:n]
            keys, vals = torch.cat([kc, kt[mine, h]]), torch.cat([vc, vt[mine, h]])
            sc = (q[mine, h].reshape(m * G, D) @ keys.T / math.sqrt(D)).reshape(m, G, -1)
            sc[:, :, n:] = sc[:, :, n:].masked_fill(~anc[:, None, :], -math.inf)
            out[mine, h] = (torch.softmax(sc, -1).reshape(m * G, -1) @ vals).reshape(m, G, D)
    return out.reshape(R, H * G, D)


def _exact_sample(s):
    """The log-probability under the target of the token each row ends with; the tokens are whole numbers and have none."""
    case, R = s["case"], s["case"]["rows"]
    kids, token = s["kids"].tolist(), s["token"].tolist()
    logp = torch.zeros(R, dtype=torch.float64, device=DEVICE)
    for i in range(R):
        t = float(s["temp"][s["req"][i]])
        z = s["logits"][i].double()
        lp = torch.log_softmax(z / t, 0) if t > 0 else torch.full_like(z, -math.inf).index_fill(0, torch.nonzero(z == z.max())[0], 0.0)
        p, x = lp.exp(), None
        for c in kids[i] if case["draft"] else []:
            if c < 0:
                break
            qd = s["draft"][i].double()
            if float(s["u_accept"][c]) * float(qd[token[c]]) < float(p[token[c]]):
                x = token[c]
                break
            rest = (p - qd).clamp(min=0)
            p = rest / rest.sum() if float(rest.sum()) > 0 else p
        if x is None:
            cum = p.cumsum(0)
            x = int((cum <= float(s["u_sample"][i]) * cum[-1]).sum().clamp(max=z.numel() - 1))
        logp[i] = lp[x]
    return dict(tok=None, len=None, node=None, row_tok=None, row_logp=logp)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        if sum(_ragged(case, case["tok"], 1)) // case["block"] > 4000:
            return None
        off = s["row_off"].long()
        req = torch.repeat_interleave(torch.arange(case["n_req"], device=DEVICE), off[1:] - off[:-1])
        rows = torch.arange(s["n_tok"], device=DEVICE)
        return _exact_write(s, req, rows - off[req], rows)
    if case["op"] == "commit":
        path = s["path"][s["acc_node"].long()].long()
        req, j = torch.nonzero(path >= 0, as_tuple=True)
        return _exact_write(s, req, j, path[req, j])
    return _exact_attend(s) if case["op"] == "attend" else _exact_sample(s)
