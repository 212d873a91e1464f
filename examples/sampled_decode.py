"""Speculative decoding with sampling on a small random decoder.

Every step drafts a tree per request, runs the layers over all rows of all
trees at once (``w12_gemm`` for the linears, ``w12_tree_attention`` over the
paged cache, ``w12_block_norm`` between them), verifies the drafts against the model's own distribution
(``w12_tree_verify_sampled``) and moves the accepted paths into the cache
(``w12_kv_commit``).  Prompts enter through the same layers in chunks, which
``w12_kv_append`` appends.

    python examples/sampled_decode.py [--steps 8] [--requests 3] [--temperature 0.8]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import speculative_decoding_tree_w12_gb300 as w12

D = 128            # of a head
CHUNK = 16         # prompt tokens of a request to a pass


class Decoder:
    """`layers` of attention with a residual, and a head; random weights."""

    def __init__(self, hidden=512, vocab=2048, layers=2, heads=6, kv_heads=2, seed=0, device="cuda"):
        self.hidden, self.vocab, self.heads, self.kv_heads, self.device = hidden, vocab, heads, kv_heads, device
        rng = np.random.default_rng(seed)
        self.qkv, self.o, self.dense = [], [], []

        def linear(n, k, gain=1.0):
            w = torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32) * gain / k ** 0.5).bfloat16()
            self.dense.append(w)
            return w12.DeviceWeight(w12.w12_pack(w.view(torch.int16).numpy().view(np.uint16)))

        for _ in range(layers):
            self.qkv.append(linear((heads + 2 * kv_heads) * D, hidden))
            self.o.append(linear(hidden, heads * D))
        self.head = linear(vocab, hidden, 3.0)
        self.one = torch.ones(hidden, dtype=torch.bfloat16, device=device)     # the norms' weights
        self.embed = torch.from_numpy(rng.standard_normal((vocab, hidden)).astype(np.float32)).bfloat16().to(device)
        # the drafter: every token's two likeliest successors with no context but itself
        self.draft = (norm(self.embed).float() @ self.dense[-1].to(device).float().T).topk(2).indices.cpu()

    def rope(self, positions):
        f = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))
        a = torch.arange(positions, dtype=torch.float64)[:, None] * f
        return w12.Rope(a.cos().float().to(self.device), a.sin().float().to(self.device))


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Session:
    """Requests in flight: their caches (one to a layer), and what a step's calls need."""

    def __init__(self, model: Decoder, n_req: int, max_tokens: int, block=64):
        self.m, self.n = model, n_req
        max_rows = n_req * CHUNK
        per = -(-max_tokens // block)
        table = torch.arange(n_req * per, dtype=torch.int32, device=model.device).view(n_req, per)
        self.caches = [w12.KvCache.empty(n_req * per, model.kv_heads, block, table) for _ in model.qkv]
        self.rope = model.rope(max_tokens + 64)
        self.ws = w12.Workspace(max_rows, max((model.heads + 2 * model.kv_heads) * D, model.vocab), model.vocab, n_req)
        self.aws = w12.AttentionWorkspace(max_rows, model.heads, model.kv_heads, n_req)

    def forward(self, tree, tokens):
        """Logits of the tree's rows, and every layer's fused rows (its keys and values among them)."""
        m, rows = self.m, []
        x, n = w12.w12_block_norm(m.embed[tokens.long()], pre=m.one)
        wq, wk = m.heads * D, m.kv_heads * D
        for qkv, o, cache in zip(m.qkv, m.o, self.caches):
            r = w12.w12_gemm(qkv, n, self.ws)
            a = w12.w12_tree_attention(cache, self.rope, tree, self.n, r[:, :wq], r[:, wq:wq + wk], r[:, wq + wk:], self.ws,
                                       self.aws)
            x, n = w12.w12_block_norm(x, w12.w12_gemm(o, a.view(len(tokens), wq), self.ws), pre=m.one)
            rows.append((r[:, wq:wq + wk], r[:, wq + wk:]))
        return w12.w12_gemm(m.head, n, self.ws), rows

    def prefill(self, prompts):
        """All prompt tokens but the last of each request into the caches."""
        for at in range(0, max(len(p) for p in prompts) - 1, CHUNK):
            part = [p[:-1][at:at + CHUNK] for p in prompts]
            tree, tokens, off = make_tree([[(t, i - 1) for i, t in enumerate(c)] for c in part], self.m.device)
            _, rows = self.forward(tree, tokens)
            for cache, (k, v) in zip(self.caches, rows):
                w12.w12_kv_append(cache, self.rope, k, v, off, self.ws)

    def step(self, last, temperature, rng):
        """One verification step from each request's last token: the accepted tokens of every request."""
        drafts = []
        for t in last:                     # the last token, two successors, one successor of each
            a, b = self.m.draft[t].tolist()
            drafts.append([(t, -1), (a, 0), (b, 0), (int(self.m.draft[a, 0]), 1), (int(self.m.draft[b, 0]), 2)])
        tree, tokens, _ = make_tree(drafts, self.m.device)
        logits, rows = self.forward(tree, tokens)
        u = torch.from_numpy(rng.random(len(tokens), dtype=np.float32)).to(self.m.device)
        dist = w12.SampleRows(logits, u, temperature=temperature)
        tok, n, node = w12.w12_tree_verify_sampled(dist, tree, self.n, 2, self.ws)
        for cache, (k, v) in zip(self.caches, rows):
            w12.w12_kv_commit(cache, self.rope, tree, self.n, node, k, v, self.ws)
        out = [t[:c] for t, c in zip(tok.tolist(), n.tolist())]          # (waits for the step)
        if self.ws.status():
            raise RuntimeError(w12.status_str(self.ws.status()))
        return out, logits


def make_tree(requests, device):
    """Rows (token, parent among the request's own, -1 for its root) of every request -> tree, tokens, row offsets."""
    parent, token, depth, req, off = [], [], [], [], [0]
    for r, nodes in enumerate(requests):
        lo = len(parent)
        for t, p in nodes:
            parent.append(-1 if p < 0 else lo + p)
            depth.append(0 if p < 0 else depth[lo + p] + 1)
            token.append(t)
            req.append(r)
        off.append(len(parent))
    dev = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device=device)
    token, off = dev(token), dev(off)
    return w12.DeviceTree.from_arrays(dev(parent), dev(depth, torch.uint8), dev(req), off, token=token), token, off


def run(requests=3, steps=8, temperature=0.8, seed=0, model=None):
    """Decodes; the texts (lists of tokens) and the session."""
    model = model or Decoder(seed=seed)
    rng = np.random.default_rng(seed + 1)
    texts = [rng.integers(0, model.vocab, 5 + 20 * r).tolist() for r in range(requests)]
    s = Session(model, requests, max_tokens=max(map(len, texts)) + 3 * steps + 8)
    s.prefill(texts)
    temp = torch.full((requests,), temperature, device=model.device)
    for _ in range(steps):
        out, _ = s.step([t[-1] for t in texts], temp, rng)
        for t, o in zip(texts, out):
            t += o
    return texts, s


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--requests", type=int, default=3)
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args()
    texts, s = run(a.requests, a.steps, a.temperature, a.seed)
    for r, t in enumerate(texts):
        new = t[5 + 20 * r:]
        print(f"request {r}: {len(new)} tokens in {a.steps} steps: {new}")
    print("cached tokens:", s.caches[0].len.tolist())


if __name__ == "__main__":
    main()
