"""The sampled decoding example: the attention layer, sampled verification and
the cache running together."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def ex():
    pytest.importorskip("torch")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sampled_decode.py")
    spec = importlib.util.spec_from_file_location("sampled_decode", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_texts_and_lengths(ex):
    model = ex.Decoder()
    texts, s = ex.run(requests=3, steps=6, temperature=0.8, seed=3, model=model)
    again, _ = ex.run(requests=3, steps=6, temperature=0.8, seed=3, model=model)
    assert texts == again                                   # no call's result depends on the order of its threads
    for r, t in enumerate(texts):
        assert len(t) >= 5 + 20 * r + 6 and all(0 <= x < model.vocab for x in t)
        for c in s.caches:                                  # everything but the last token is cached
            assert c.len[r].item() == len(t) - 1


def rotate(x, cos, sin):
    a, b = x[..., :D // 2], x[..., D // 2:]
    return np.concatenate([a * cos - b * sin, b * cos + a * sin], -1)


def dense_logits(model, s, tokens, parent, depth, req):
    """The forward pass over the tree in 64 bits, from the cached codes."""
    f64 = lambda t: t.detach().cpu().double().numpy()
    cos, sin = f64(s.rope.cos), f64(s.rope.sin)
    norm = lambda x: x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    H, Hq = model.kv_heads, model.heads
    x = f64(model.embed)[tokens]
    w = [f64(t) for t in model.dense]
    for layer, cache in enumerate(s.caches):
        import torch
        kc, vc = (f64(t.view(torch.float8_e4m3fn).float()) for t in (cache.k, cache.v))
        kc, vc = kc * f64(cache.k_scale)[:, :, None, None], vc * f64(cache.v_scale)[:, :, None, None]
        table, lens = cache.block_table.cpu().numpy(), cache.len.cpu().numpy()
        qkv = norm(x) @ w[2 * layer].T
        out = np.zeros((len(tokens), Hq, D))
        pos = lens[req] + depth
        turn = lambda y, n: rotate(y.reshape(len(tokens), n, D), cos[pos][:, None], sin[pos][:, None])
        q, k = turn(qkv[:, :Hq * D], Hq), turn(qkv[:, Hq * D:(Hq + H) * D], H)
        v = qkv[:, (Hq + H) * D:].reshape(len(tokens), H, D)
        for i in range(len(tokens)):
            path, j = [], i
            while j >= 0:
                path.append(j)
                j = parent[j]
            n, blocks = lens[req[i]], table[req[i]]
            for h in range(Hq):
                g = h // (Hq // H)
                keys = np.concatenate([kc[blocks, g].reshape(-1, D)[:n], k[path, g]])
                vals = np.concatenate([vc[blocks, g].transpose(0, 2, 1).reshape(-1, D)[:n], v[path, g]])
                z = keys @ q[i, h] / D ** 0.5
                e = np.exp(z - z.max())
                out[i, h] = e @ vals / e.sum()
        x = x + out.reshape(len(tokens), -1) @ w[2 * layer + 1].T
    return norm(x) @ w[-1].T


def test_logits_against_64_bits(ex):
    # Eight roundings to BF16 on a row's way (2^-9 each, at random), none of
    # which the 64-bit pass makes: under 1% of the logits' scale, bound 3%.
    model = ex.Decoder()
    texts, s = ex.run(requests=2, steps=3, temperature=0.0, seed=5, model=model)
    nodes = [[(t[-1], -1), (11, 0), (12, 0), (13, 1), (14, 3)] for t in texts]
    tree, tokens, _ = ex.make_tree(nodes, model.device)
    got = s.forward(tree, tokens)[0].float().cpu().double().numpy()
    h = tree.host()
    ref = dense_logits(model, s, tokens.cpu().numpy(), h["parent"], h["depth"].astype(int), h["req"])
    assert np.abs(got - ref).max() <= 3e-2 * np.abs(ref).max()
