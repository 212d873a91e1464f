"""The attention and sampling calls turn host tensors, tensors of several
devices and trees of too few requests away: a kernel gets bare addresses."""
from __future__ import annotations

import types

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def w12():
    from speculative_decoding_tree_w12_gb300 import build
    build.build()
    import speculative_decoding_tree_w12_gb300 as m
    m.lib()
    return m


def parts(w12, device, n_req=2):
    """What the calls of a step of 4 rows take, by name; every value may be replaced."""
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device=device)
    i = lambda a, dt=torch.int32: torch.tensor(a, dtype=dt, device=device)
    cuda = device != "cpu"
    ws = w12.Workspace(4, 0, 0, n_req) if cuda else types.SimpleNamespace(addr=0, nbytes=0, dev=-1)
    aws = w12.AttentionWorkspace(4, 4, 2, n_req, device=device)
    table = i([[0, 1], [2, 3]])
    rows = lambda w: z(4, w, dt=torch.bfloat16)
    return dict(cache=w12.KvCache.empty(4, 2, 32, table, device=device), rope=w12.Rope(z(60, 32, dt=torch.float32) + 1, z(60, 32, dt=torch.float32)),
                tree=w12.DeviceTree.from_arrays(i([-1, 0, -1, 2]), i([0, 1, 0, 1], torch.uint8), i([0, 0, 1, 1]), i([0, 2, 4]),
                                                token=i([1, 2, 3, 4])),
                q=rows(512), k=rows(256), v=rows(256), off=i([0, 2, 4]), node=i([1, 2]), len_out=z(2), out=z(4, 4, 128, dt=torch.bfloat16),
                dist=w12.SampleRows(z(4, 50, dt=torch.float32), z(4, dt=torch.float32), z(2, dt=torch.float32) + 1),
                row_tok=z(4), row_logp=z(4, dt=torch.float32), acc_tok=z(2, 3), acc_len=z(2), acc_node=z(2), ws=ws, aws=aws)


CALLS = dict(
    append=(lambda m, a: m.w12_kv_append(a["cache"], a["rope"], a["k"], a["v"], a["off"], a["ws"], len_out=a["len_out"]),
            ("rope", "k", "v", "off", "ws", "len_out")),
    commit=(lambda m, a: m.w12_kv_commit(a["cache"], a["rope"], a["tree"], 2, a["node"], a["k"], a["v"], a["ws"], len_out=a["len_out"]),
            ("rope", "tree", "node", "k", "v", "ws", "len_out")),
    attend=(lambda m, a: m.w12_tree_attention(a["cache"], a["rope"], a["tree"], 2, a["q"], a["k"], a["v"], a["ws"], a["aws"], out=a["out"]),
            ("rope", "tree", "q", "k", "v", "ws", "aws", "out")),
    sample=(lambda m, a: m.w12_tree_sample(a["dist"], a["tree"], 2, a["ws"], a["row_tok"], a["row_logp"]),
            ("tree", "ws", "row_tok", "row_logp")),
    verify=(lambda m, a: m.w12_tree_verify_sampled(a["dist"], a["tree"], 2, 2, a["ws"], a["row_tok"], a["row_logp"], a["acc_tok"],
                                                   a["acc_len"], a["acc_node"]),
            ("tree", "ws", "row_tok", "row_logp", "acc_tok", "acc_len", "acc_node")),
)


@pytest.mark.parametrize("call", CALLS)
def test_host_handles(w12, call):
    a = parts(w12, "cpu")
    with pytest.raises(ValueError):
        CALLS[call][0](w12, a)


@pytest.mark.gpu
@pytest.mark.parametrize("call", CALLS)
def test_a_host_tensor_among_device_tensors(w12, call):
    run, names = CALLS[call]
    a, host = parts(w12, "cuda"), parts(w12, "cpu")
    for name in names:
        with pytest.raises(ValueError):
            run(w12, {**a, name: host[name]})
    run(w12, a)
    torch.cuda.synchronize()
    assert a["ws"].status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["commit", "attend", "sample", "verify"])
def test_a_tree_of_fewer_requests(w12, call):
    a = parts(w12, "cuda")
    i = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device="cuda")
    a["tree"] = w12.DeviceTree.from_arrays(i([-1, 0, 1, 2]), i([0, 1, 2, 3], torch.uint8), i([0] * 4), i([0, 4]), token=i([1, 2, 3, 4]))
    with pytest.raises(ValueError):
        CALLS[call][0](w12, a)


@pytest.mark.gpu
def test_handles_of_several_devices(w12):
    z = lambda *s, dt=torch.uint8, dev="cuda": torch.zeros(s, dtype=dt, device=dev)
    good = [z(3, 2, 64, 128), z(3, 2, 128, 64), z(3, 2, dt=torch.float32), z(3, 2, dt=torch.float32), z(2, 2, dt=torch.int32),
            z(2, dt=torch.int32)]
    w12.KvCache(*good)
    for j in range(1, 6):
        with pytest.raises(ValueError):
            w12.KvCache(*good[:j], good[j].cpu(), *good[j + 1:])
    f = lambda *s, dev="cuda": z(*s, dt=torch.float32, dev=dev)
    with pytest.raises(ValueError):
        w12.Rope(f(4, 8), f(4, 8, dev="cpu"))
    for kw in (dict(u_sample=f(2, dev="cpu")), dict(temperature=f(1, dev="cpu")), dict(draft_p=f(2, 8, dev="cpu"), u_accept=f(2)),
               dict(draft_p=f(2, 8), u_accept=f(2, dev="cpu"))):
        with pytest.raises(ValueError):
            w12.SampleRows(f(2, 8), **{"u_sample": f(2), **kw})
