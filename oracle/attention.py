"""Plain 64-bit forms of the KV cache, the tree attention and the sampled
verification, in numpy.  They share no code with the library.

The position rotation is defined in FP32 with every product and sum rounded
(``turn``), so cache codes are exact values; everything else is computed in
64 bits."""
from __future__ import annotations

import numpy as np


def e4m3_values() -> np.ndarray:
    """The value of every E4M3 code (0x7F and 0xFF are NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c & 128, -v, v)


E4M3 = e4m3_values()
_POS = E4M3[:127]                      # ascending


def e4m3_encode(x) -> np.ndarray:
    """Nearest code, ties to even; |x| <= 448; not finite -> NaN."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    ok = np.isfinite(x)
    a = np.where(ok, a, 0.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code | np.where(np.signbit(x), 128, 0)
    return np.where(ok, code, 127).astype(np.uint8)


def block_scale(top: float) -> float:
    """The least power of two s with top <= 448 s, not under 2^-32."""
    s = 2.0 ** -32
    while top > 448.0 * s:
        s *= 2.0
    return s


def turn(x, pos, cos, sin, adjacent=False) -> np.ndarray:
    """x [..][d] (float32) turned by one position, FP32 rounded per operation."""
    x = np.array(x, np.float32)
    if cos is None:
        return x
    half = cos.shape[1]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
    c, s = cos[pos], sin[pos]
    with np.errstate(over="ignore", invalid="ignore"):
        xa, xb = x[..., a].copy(), x[..., b].copy()
        x[..., a] = xa * c - xb * s
        x[..., b] = xb * c + xa * s
    return x


def kv_write(cache, r, rows_k, rows_v, cos, sin, adjacent=False):
    """Append rows [n][H][d] (float32) to request r of cache (a dict of numpy
    arrays k, v, k_scale, v_scale, table, len), in place."""
    bt = cache["k"].shape[2]
    H = cache["k"].shape[1]
    n, at = len(rows_k), int(cache["len"][r])
    end = at + n
    keys = np.stack([turn(rows_k[j], at + j, cos, sin, adjacent) for j in range(n)]) if n else rows_k
    first = at
    while at < end:
        upto = min((at // bt + 1) * bt, end)
        b, lo, hi = int(cache["table"][r, at // bt]), at % bt, upto - at // bt * bt
        for name, x in (("k", keys), ("v", rows_v)):
            for h in range(H):
                y = np.asarray(x[at - first:upto - first, h], np.float64)            # [m][d]
                fin = np.abs(y[np.isfinite(y)])
                s = block_scale(fin.max() if fin.size else 0.0)
                code = cache[name][b, h] if name == "k" else cache[name][b, h].T     # [bt][d]
                old = float(cache[name + "_scale"][b, h])
                if lo and old >= s:
                    s = old
                elif lo:
                    code[:lo] = e4m3_encode(E4M3[code[:lo]] * (old / s))
                code[lo:hi] = e4m3_encode(y / s)
                cache[name + "_scale"][b, h] = s
        at = upto
    cache["len"][r] = end


def root_path(parent, row):
    p = [row]
    while parent[p[-1]] >= 0:
        p.append(int(parent[p[-1]]))
    return p[::-1]


def cached(cache, r):
    """Keys and values [len][H][d] of request r, in 64 bits."""
    bt, n = cache["k"].shape[2], int(cache["len"][r])
    b = [int(x) for x in cache["table"][r, :-(-n // bt)]]
    H, d = cache["k"].shape[1], cache["k"].shape[3]
    if not b:
        return np.zeros((0, H, d)), np.zeros((0, H, d))
    k = E4M3[cache["k"][b]] * cache["k_scale"][b].astype(np.float64)[:, :, None, None]
    v = E4M3[cache["v"][b]] * cache["v_scale"][b].astype(np.float64)[:, :, None, None]
    return k.transpose(0, 2, 1, 3).reshape(-1, H, d)[:n], v.transpose(0, 3, 1, 2).reshape(-1, H, d)[:n]


def tree_attention(cache, parent, depth, req, q, k, v, cos, sin, adjacent, scale):
    """-> (out [R][Hq][d], slack [R][Hq][d]).

    slack bounds how far a kernel may be off that rounds q to twelve significant
    bits (and to 2^-17 of the head's largest |q|), the weights to eleven bits and
    the output to BF16, and sums in FP32: a relative weight error of at most
    2 |ds| + 2^-10 with |ds| the score's, times sum p |v|, plus 2^-8 |out|."""
    R, Hq, d = q.shape
    H = k.shape[1]
    G = Hq // H
    out, slack = np.zeros((R, Hq, d)), np.zeros((R, Hq, d))
    ctx = {}
    for i in range(R):
        r = int(req[i])
        if r not in ctx:
            ctx[r] = cached(cache, r)
        n = int(cache["len"][r])
        qi = turn(q[i], n + int(depth[i]), cos, sin, adjacent).astype(np.float64)
        path = root_path(parent, i)
        kp = np.stack([turn(k[j], n + int(depth[j]), cos, sin, adjacent) for j in path]).astype(np.float64)
        vp = np.stack([v[j] for j in path]).astype(np.float64)
        keys, vals = np.concatenate([ctx[r][0], kp]), np.concatenate([ctx[r][1], vp])
        for hq in range(Hq):
            kh, vh = keys[:, hq // G], vals[:, hq // G]
            s = kh @ qi[hq] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, hq] = p @ vh
            ds = scale * (np.abs(kh) @ np.abs(qi[hq]) * 2.0 ** -12 + 2.0 ** -17 * np.abs(qi[hq]).max() * np.abs(kh).sum(1)).max()
            slack[i, hq] = (2 * ds + 2.0 ** -10) * (p @ np.abs(vh)) + 2.0 ** -8 * np.abs(out[i, hq])
    return out, slack


def target(logits, temperature):
    """The target's probabilities in 64 bits (temperature 0: one-hot at the lowest largest)."""
    z = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    if temperature == 0:
        p = np.zeros_like(z)
        p[int(np.argmax(z))] = 1.0
        return p
    z = z / temperature
    e = np.where(z == z.max(), 1.0, np.exp(z - z.max()))
    return e / e.sum()


def sample_row(p, kids, q, u_accept, u_sample, eps):
    """The tokens that a row may emit: one, or several where a decision is
    closer than eps (relative to the whole mass) to its boundary.  kids: the
    children's tokens in row order; q: the drafter's probabilities or None."""
    p = p.copy()
    if q is not None:
        for j, x in enumerate(kids):
            a, b = float(u_accept[j]) * q[x], p[x]
            if abs(a - b) <= eps:
                return None
            if a < b:
                return {int(x)}
            rest = np.maximum(p - q, 0.0)
            if rest.sum() <= 64 * eps:
                return None
            eps = 4 * eps / rest.sum()
            p = rest / rest.sum()
    cum = np.cumsum(p)
    lo, hi = (float(u_sample) - eps) * cum[-1], (float(u_sample) + eps) * cum[-1]
    a, b = np.searchsorted(cum, lo, side="right"), np.searchsorted(cum, hi, side="right")
    return {int(t) for t in range(min(a, len(p) - 1), min(b, len(p) - 1) + 1) if p[t] > 0 or t in (a, b)}
