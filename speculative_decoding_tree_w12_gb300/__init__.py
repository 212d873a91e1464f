"""W12 tree-verify pass on GB300 (sm_103a): Python binding of ``libw12.so``.

A thin ctypes layer over the C ABI in ``include/w12.h``: it marshals torch
tensors (device memory) and numpy arrays (host memory) into the C structs and
calls the library.  Every step of the pass runs in the library's CUDA
kernels; if ``libw12.so`` is missing or cannot load, importing the functions
below raises -- there is no fallback.

Entry points (same names as the C ABI): ``w12_pack``, ``w12_unpack``,
``w12_load_check``, ``w12_gemm``, ``w12_lmhead_argmax``, ``w12_tree_build``,
``w12_tree_accept``, ``w12_verify_step``, the TLV calls (``w12_verify_step_q``,
``w12_tlv_chain``, ``w12_tlv_splice``), the recurrent layer's
``w12_gdn_tree_verify``, ``w12_gdn_commit``, ``w12_gdn_prefill`` and
``w12_gdn_step``, the norms ``w12_gdn_norm`` and ``w12_block_norm``, the attention
layer's ``w12_kv_append``, ``w12_tree_attention``, ``w12_kv_commit``, and
``w12_tree_verify_sampled``, plus the workspace helpers.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
from typing import List, Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw12.so")

W12_OK, W12_E_INVAL, W12_E_UNSUPPORTED, W12_E_MISMATCH, W12_E_CUDA, W12_E_TIMEOUT, W12_E_WORKSPACE = \
    0, -1, -2, -3, -4, -5, -6

TILE_N, TILE_K, REC_BYTES = 128, 64, 12288


class W12Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        detail = ""
        if status == W12_E_CUDA:
            buf = C.create_string_buffer(96)
            code = lib().w12_debug_last_cuda_error(buf, 96)
            detail = f" [{buf.value.decode()} = {code}]"
        super().__init__(f"{what}: {status_str(status)} ({status}){detail}")


# ---------------------------------------------------------------------------
# C structs (mirror include/w12.h)
# ---------------------------------------------------------------------------

class Layout(C.Structure):
    _fields_ = [("n", C.c_int64), ("k", C.c_int64), ("n_tiles", C.c_int64), ("k_tiles", C.c_int64),
                ("n_escapes", C.c_int64), ("rec_bytes", C.c_size_t), ("base_bytes", C.c_size_t),
                ("esc_off_bytes", C.c_size_t), ("esc_bytes", C.c_size_t)]


class Weight(C.Structure):
    _fields_ = [("rec", C.c_void_p), ("base", C.c_void_p), ("esc_tile_off", C.c_void_p), ("esc", C.c_void_p),
                ("n", C.c_int64), ("k", C.c_int64), ("n_escapes", C.c_int64)]


class LatticeC(C.Structure):
    _fields_ = [("n_req", C.c_int32), ("p_max", C.c_int32), ("n_cand", C.c_int32), ("conditional", C.c_int32),
                ("p_r", C.c_void_p), ("root_tok", C.c_void_p), ("cand_tok", C.c_void_p), ("cand_logp", C.c_void_p)]


class TreeC(C.Structure):
    _fields_ = [("R", C.c_int32), ("parent", C.c_void_p), ("token", C.c_void_p), ("depth", C.c_void_p),
                ("req", C.c_void_p), ("score", C.c_void_p), ("rank", C.c_void_p), ("req_row_off", C.c_void_p)]


class StepC(C.Structure):
    _fields_ = [("n_linear", C.c_int32), ("lin", C.c_void_p), ("x", C.c_void_p), ("y", C.c_void_p),
                ("head", C.c_void_p), ("h", C.c_void_p), ("argmax", C.c_void_p)]


_lib = None


def lib():
    """Load libw12.so (raises if it is missing: no fallback path exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "speculative_decoding_tree_w12_gb300.build.build()")
        L = C.CDLL(LIB_PATH)
        p, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
        sigs = {
            "w12_status_str": ([C.c_int], C.c_char_p),
            "w12_abi_version": ([], C.c_int),
            "w12_pack_query": ([p, i64, i64, p], C.c_int),
            "w12_pack": ([p, i64, i64, p, p, p, p, p], C.c_int),
            "w12_workspace_bytes": ([i32, i64, i64, i32], sz),
            "w12_workspace_init": ([p, sz, p], C.c_int),
            "w12_status_fetch": ([p, p], C.c_int),
            "w12_unpack": ([p, p, p], C.c_int),
            "w12_load_check": ([p, p, p, p, sz, p], C.c_int),
            "w12_gemm": ([p, p, i32, p, p, sz, p], C.c_int),
            "w12_gemm_static_scratch": ([p, p, i32, p, p], C.c_int),
            "w12_lmhead_argmax": ([p, p, i32, p, p, p, sz, p], C.c_int),
            "w12_gemm_q": ([p, p, i32, p, p, sz, p], C.c_int),
            "w12_lmhead_argmax_q": ([p, p, i32, p, p, p, sz, p], C.c_int),
            "w12_head_cert_norms": ([p, p, p], C.c_int),
            "w12_cert_workspace_bytes": ([i32, i64], sz),
            "w12_lmhead_argmax_certified": ([p, p, p, i32, p, p, p, p, sz, p, sz, p], C.c_int),
            "w12_tree_build": ([p, i32, p, p, sz, p], C.c_int),
            "w12_tree_accept": ([p, i32, i32, p, p, p, p, p], C.c_int),
            "w12_verify_step": ([p, p, i32, i32, p, p, p, p, sz, p], C.c_int),
            "w12_verify_step_q": ([p, p, i32, i32, p, p, p, p, sz, p], C.c_int),
            "w12_tlv_chain": ([p, p, i32, i32, p, p], C.c_int),
            "w12_gdn_tree_verify": ([p, p, i32, i32, p, p, sz, p], C.c_int),
            "w12_gdn_commit": ([p, p, i32, p, p, p, sz, p], C.c_int),
            "w12_gdn_wy_verify": ([p, p, i32, p, p, p, sz, p], C.c_int),
            "w12_gdn_wy_commit": ([p, p, i32, p, p, p, p, sz, p], C.c_int),
            "w12_gdn_prefill": ([p, i32, p, p, p, p, p, sz, p], C.c_int),
            "w12_gdn_scratch_bytes": ([i32, i32], sz),
            "w12_gdn_step": ([p, p, p, p, p], C.c_int),
            "w12_gdn_norm": ([p, i32, i32, i32, p, i64, p, C.c_float, i32, p, i64, p], C.c_int),
            "w12_block_norm": ([p, p], C.c_int),
            "w12_tlv_splice": ([p, p, p, p, i32, i32, p, p, p, p, sz, p], C.c_int),
            "w12_kv_append": ([p, p, i32, p, i64, p, i64, i32, p, p, p, sz, p], C.c_int),
            "w12_kv_commit": ([p, p, p, i32, p, p, i64, p, i64, p, p, sz, p], C.c_int),
            "w12_attn_workspace_bytes": ([i32, i32, i32, i32], sz),
            "w12_tree_attention": ([p, p, p, i32, i32, p, i64, p, i64, p, i64, C.c_float, p, p, sz, p, sz, p], C.c_int),
            "w12_sample_max_vocab": ([], i64),
            "w12_sample_scratch_bytes": ([i32, i64], sz),
            "w12_tree_sample": ([p, p, i32, p, p, p, sz, p], C.c_int),
            "w12_tree_verify_sampled": ([p, p, i32, i32, p, p, p, p, p, p, sz, p], C.c_int),
            "w12_debug_set": ([i32, C.c_uint64], None),
            "w12_debug_num_sms": ([], i32),
            "w12_debug_attn_registers": ([i32, p], i32),
            "w12_debug_gdn_inverse_conflicts": ([], i32),
            "w12_debug_profile": ([i32], None),
            "w12_debug_last_cuda_error": ([p, i32], i32),
            "w12_debug_profile_read": ([p, i32], i32),
            "w12_debug_chain_trace": ([p, sz], None),
            "w12_debug_chain_parts": ([i32], i32),
        }
        for name, (args, res) in sigs.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def status_str(s: int) -> str:
    return lib().w12_status_str(int(s)).decode()


def _check(s: int, what: str):
    if s != W12_OK:
        raise W12Error(s, what)


def _stream(stream=None):
    import torch
    st = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(st.cuda_stream)


# What the calls of a decode loop look up once: the types they accept and the
# runtime's own query of the current stream (a call of some 0.2 us; building a
# torch.cuda.Stream object takes fifteen times that).
_torch = _raw_stream = _device = None


def _runtime():
    global _torch, _raw_stream, _device
    if _torch is None:
        import torch
        current = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", None)
        if current is not None and device is not None:
            _raw_stream = lambda: current(device())
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream
        _device = device if device is not None else torch.cuda.current_device
        _torch = torch
    return _torch


def _st(stream) -> int:
    return _raw_stream() if stream is None else stream.cuda_stream


def _st_on(dev, stream) -> int:
    """_st of a call whose tensors are on cuda:dev: it has to be the current device, on which the library launches."""
    if _device() != dev:
        raise ValueError(f"tensors on cuda:{dev}: it has to be the current device")
    return _raw_stream() if stream is None else stream.cuda_stream


def _under(stream, make):
    """make() -> tensors for a call on `stream` (None: the current one).  Memory of the current stream may still be in use there
    when another stream's kernel writes it, so it is that stream's own (what fills it runs there too); and since its
    reader may be on the current one, it is nobody else's before both have passed its end."""
    torch = _runtime()
    if stream is None or stream.cuda_stream == _raw_stream():
        return make()
    with torch.cuda.stream(stream):
        made = make()
    for t in made.tensors() if isinstance(made, DeviceTree) else (made,):
        t.record_stream(torch.cuda.current_stream(t.device))
    return made


def _empty(shape, dtype, device, stream):
    """torch.empty for a call on `stream`."""
    if stream is None:
        return _runtime().empty(shape, dtype=dtype, device=device)
    return _under(stream, lambda: _torch.empty(shape, dtype=dtype, device=device))


def _used_on(streams, st, stream, scratch):
    """A call on `stream` (its handle: st) uses scratch that its object holds: the allocator learns of every such stream."""
    if scratch.numel() and scratch.is_cuda:
        scratch.record_stream(_torch.cuda.current_stream() if stream is None else stream)
    streams.add(st)


def _dp(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _np(a: np.ndarray):
    return a.ctypes.data_as(C.c_void_p)


# ---------------------------------------------------------------------------
# host packing
# ---------------------------------------------------------------------------

class HostPacked:
    """W12 buffers in host memory (numpy), as produced by ``w12_pack``."""

    def __init__(self, n, k, rec, base, esc_tile_off, esc):
        self.n, self.k = n, k
        self.rec, self.base, self.esc_tile_off, self.esc = rec, base, esc_tile_off, esc

    @property
    def n_escapes(self) -> int:
        return int(self.esc.shape[0])

    @property
    def nbytes(self) -> int:
        return self.rec.nbytes + self.base.nbytes + self.esc_tile_off.nbytes + self.esc.nbytes


def w12_pack(w_bf16_bits: np.ndarray) -> HostPacked:
    """Pack a host BF16 tensor (uint16 bits, [n][k]) into W12.  The library
    checks its own output bit for bit before returning."""
    w = np.ascontiguousarray(w_bf16_bits, dtype=np.uint16)
    n, k = w.shape
    L = Layout()
    _check(lib().w12_pack_query(_np(w), n, k, C.byref(L)), "w12_pack_query")
    rec = np.empty(L.rec_bytes, np.uint8)
    base = np.empty(L.base_bytes, np.uint8)
    off = np.empty(L.esc_off_bytes // 4, np.int32)
    esc = np.empty(L.esc_bytes // 4, np.uint32)
    _check(lib().w12_pack(_np(w), n, k, C.byref(L), _np(rec), _np(base), _np(off),
                          _np(esc) if esc.size else None), "w12_pack")
    return HostPacked(n, k, rec, base, off, esc)


# ---------------------------------------------------------------------------
# device tensors
# ---------------------------------------------------------------------------

class DeviceWeight:
    """A packed W12 tensor resident on the GPU (torch tensors) plus its C view."""

    def __init__(self, hp: HostPacked, device="cuda", rec=None):
        import torch
        self.n, self.k, self.n_escapes = hp.n, hp.k, hp.n_escapes
        self.rec = rec if rec is not None else torch.from_numpy(hp.rec).to(device)
        self.base = torch.from_numpy(hp.base).to(device)
        self.esc_tile_off = torch.from_numpy(hp.esc_tile_off).to(device)
        self.esc = torch.from_numpy(hp.esc.view(np.int32)).to(device) if hp.n_escapes else None
        self.c = Weight(self.rec.data_ptr(), self.base.data_ptr(), self.esc_tile_off.data_ptr(),
                        _dp(self.esc), self.n, self.k, self.n_escapes)

    @property
    def nbytes(self) -> int:
        b = self.rec.numel() + self.base.numel() + 4 * self.esc_tile_off.numel()
        return b + (4 * self.esc.numel() if self.esc is not None else 0)


class Workspace:
    """Zero-initialised device workspace sized for the given call shapes."""

    def __init__(self, R: int, max_n: int = 0, vocab: int = 0, n_req: int = 1, device="cuda"):
        import torch
        nbytes = int(lib().w12_workspace_bytes(int(R), int(max_n), int(vocab), int(n_req)))
        if nbytes == 0:
            raise W12Error(W12_E_UNSUPPORTED, "w12_workspace_bytes")
        self.buf = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        self.nbytes, self.addr, self.dev = nbytes, self.buf.data_ptr(), self.buf.get_device()
        _check(lib().w12_workspace_init(self.ptr, nbytes, _stream()), "w12_workspace_init")

    @property
    def ptr(self):
        return C.c_void_p(self.buf.data_ptr())

    def status(self, stream=None) -> int:
        return int(lib().w12_status_fetch(self.ptr, _stream(stream)))


def w12_unpack(w: DeviceWeight, out=None, stream=None):
    import torch
    if out is None:
        out = _empty((w.n, w.k), torch.bfloat16, w.rec.device, stream)
    _check(lib().w12_unpack(C.byref(w.c), C.c_void_p(out.data_ptr()), _stream(stream)), "w12_unpack")
    return out


def w12_load_check(w: DeviceWeight, src_bf16, ws: Workspace, stream=None) -> int:
    """Bit-exact device check against the source tensor; returns the number of
    differing weights (0 = identical).  Synchronises the stream."""
    mism = C.c_int64(0)
    s = lib().w12_load_check(C.byref(w.c), C.c_void_p(src_bf16.data_ptr()), C.byref(mism), ws.ptr, ws.nbytes,
                             _stream(stream))
    if s not in (W12_OK, W12_E_MISMATCH):
        raise W12Error(s, "w12_load_check")
    return int(mism.value)


def w12_gemm(w: DeviceWeight, x, ws: Workspace, y=None, stream=None, quick: bool = False):
    """``y = x . W^T`` (x: bf16 [R][k] on the device) -> bf16 [R][n].
    ``quick``: the quick pass (``w12_gemm_q``, view planes only)."""
    import torch
    R = x.shape[0]
    if y is None:
        y = _empty((R, w.n), torch.bfloat16, x.device, stream)
    fn, name = (lib().w12_gemm_q, "w12_gemm_q") if quick else (lib().w12_gemm, "w12_gemm")
    _check(fn(C.byref(w.c), C.c_void_p(x.data_ptr()), R, C.c_void_p(y.data_ptr()), ws.ptr, ws.nbytes,
              _stream(stream)), name)
    return y


def w12_lmhead_argmax(head: DeviceWeight, h, ws: Workspace, argmax=None, maxlogit=None, stream=None,
                      quick: bool = False):
    """Argmax over ``h . W_head^T`` per row -> int32 [R].  ``quick``: the quick
    pass (``w12_lmhead_argmax_q``, view planes only)."""
    import torch
    R = h.shape[0]
    if argmax is None:
        argmax = _empty((R,), torch.int32, h.device, stream)
    fn, name = (lib().w12_lmhead_argmax_q, "w12_lmhead_argmax_q") if quick else \
        (lib().w12_lmhead_argmax, "w12_lmhead_argmax")
    _check(fn(C.byref(head.c), C.c_void_p(h.data_ptr()), R, C.c_void_p(argmax.data_ptr()),
              C.c_void_p(_dp(maxlogit)) if maxlogit is not None else None, ws.ptr, ws.nbytes,
              _stream(stream)), name)
    return argmax


def w12_head_cert_norms(head: DeviceWeight, out=None, stream=None):
    """Per token: ||w_v - w^_v|| and ||w^_v|| (w^: quick weights) -> float32
    [2][n] on the device (load time, for the certified head)."""
    import torch
    if out is None:
        out = _empty((2, head.n), torch.float32, "cuda", stream)
    _check(lib().w12_head_cert_norms(C.byref(head.c), C.c_void_p(out.data_ptr()), _stream(stream)),
           "w12_head_cert_norms")
    return out


class CertWorkspace:
    """Device buffer for the certified head's quick logits and survivor lists."""

    def __init__(self, R: int, vocab: int, device="cuda"):
        import torch
        self.nbytes = int(lib().w12_cert_workspace_bytes(int(R), int(vocab)))
        if self.nbytes == 0:
            raise W12Error(W12_E_INVAL, "w12_cert_workspace_bytes")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)

    @property
    def ptr(self):
        return C.c_void_p(self.buf.data_ptr())


def w12_lmhead_argmax_certified(head: DeviceWeight, norms, h, ws: Workspace, cws: CertWorkspace, argmax=None,
                                maxlogit=None, survivors=None, stream=None):
    """Certified argmax over ``h . W_head^T`` per row -> int32 [R]: quick-pass
    logits, per-row Cauchy-Schwarz bound, exact FP64 rescoring of the
    survivors.  ``survivors`` (int32 [R], optional) gets the survivor counts."""
    import torch
    R = h.shape[0]
    if argmax is None:
        argmax = _empty((R,), torch.int32, h.device, stream)
    _check(lib().w12_lmhead_argmax_certified(C.byref(head.c), C.c_void_p(norms.data_ptr()), C.c_void_p(h.data_ptr()),
                                             R, C.c_void_p(argmax.data_ptr()),
                                             C.c_void_p(_dp(maxlogit)) if maxlogit is not None else None,
                                             C.c_void_p(_dp(survivors)) if survivors is not None else None,
                                             ws.ptr, ws.nbytes, cws.ptr, cws.nbytes, _stream(stream)),
           "w12_lmhead_argmax_certified")
    return argmax


class DeviceLattice:
    def __init__(self, lat, device="cuda"):
        import torch
        self.n_req, self.p_max, self.n_cand = int(lat.n_req), int(lat.p_max), int(lat.n_cand)
        self.conditional = int(bool(lat.conditional))
        self.p_r = np.ascontiguousarray(lat.p_r, np.int32)        # host memory by contract
        self.root_tok = torch.from_numpy(np.ascontiguousarray(lat.root_tok, np.int32)).to(device)
        self.cand_tok = torch.from_numpy(np.ascontiguousarray(lat.cand_tok, np.int32)).to(device)
        self.cand_logp = torch.from_numpy(np.ascontiguousarray(lat.cand_logp, np.float32)).to(device)
        self.c = LatticeC(self.n_req, self.p_max, self.n_cand, self.conditional, _np(self.p_r).value,
                          self.root_tok.data_ptr(), self.cand_tok.data_ptr(), self.cand_logp.data_ptr())


class DeviceTree:
    def __init__(self, budget: int, n_req: int, device="cuda"):
        import torch
        z = lambda dt, n: torch.zeros(n, dtype=dt, device=device)
        self.parent, self.token, self.req = z(torch.int32, budget), z(torch.int32, budget), z(torch.int32, budget)
        self.depth, self.rank = z(torch.uint8, budget), z(torch.uint8, budget)
        self.score = z(torch.float32, budget)
        self.req_row_off = z(torch.int32, n_req + 1)
        self.n_req, self.dev = int(n_req), self.parent.get_device()
        self.c = TreeC(0, *(t.data_ptr() for t in self.tensors()))

    def tensors(self):
        return self.parent, self.token, self.depth, self.req, self.score, self.rank, self.req_row_off

    @classmethod
    def from_arrays(cls, parent, depth, req, req_row_off, token=None):
        """A tree from its device arrays (a tree built elsewhere, a chain of
        single tokens): parent, req (int32 [R]), depth (uint8 [R]), req_row_off
        (int32 [n_req + 1]) and optionally the rows' tokens (int32 [R])."""
        import torch
        R, n_req = int(parent.shape[0]), int(req_row_off.shape[0]) - 1
        t = cls(R, n_req, device=parent.device)
        for dst, src, dt in ((t.parent, parent, torch.int32), (t.depth, depth, torch.uint8), (t.req, req, torch.int32),
                             (t.req_row_off, req_row_off, torch.int32), (t.token, token, torch.int32)):
            if src is None:
                continue
            if src.dtype != dt or src.shape != dst.shape:
                raise ValueError("tree arrays: int32 [R] (depth: uint8), req_row_off int32 [n_req + 1]")
            dst.copy_(src)
        t.c.R = R
        return t

    @property
    def R(self) -> int:
        return int(self.c.R)

    def host(self):
        R = self.R
        return dict(parent=self.parent[:R].cpu().numpy(), token=self.token[:R].cpu().numpy(),
                    depth=self.depth[:R].cpu().numpy(), req=self.req[:R].cpu().numpy(),
                    score=self.score[:R].cpu().numpy(), rank=self.rank[:R].cpu().numpy(),
                    req_row_off=self.req_row_off.cpu().numpy())


def w12_tree_build(lat: DeviceLattice, budget: int, ws: Workspace, tree: Optional[DeviceTree] = None,
                   stream=None) -> DeviceTree:
    if tree is None:
        tree = _under(stream, lambda: DeviceTree(budget, lat.n_req, device=lat.root_tok.device))
    _check(lib().w12_tree_build(C.byref(lat.c), int(budget), C.byref(tree.c), ws.ptr, ws.nbytes, _stream(stream)),
           "w12_tree_build")
    return tree


def w12_tree_accept(tree: DeviceTree, n_req: int, p_max: int, argmax, acc_tok=None, acc_len=None, acc_node=None,
                    stream=None):
    import torch
    dev = argmax.device
    acc_tok = acc_tok if acc_tok is not None else _empty((n_req, p_max + 1), torch.int32, dev, stream)
    acc_len = acc_len if acc_len is not None else _empty((n_req,), torch.int32, dev, stream)
    acc_node = acc_node if acc_node is not None else _empty((n_req,), torch.int32, dev, stream)
    _check(lib().w12_tree_accept(C.byref(tree.c), n_req, p_max, C.c_void_p(argmax.data_ptr()),
                                 C.c_void_p(acc_tok.data_ptr()), C.c_void_p(acc_len.data_ptr()),
                                 C.c_void_p(acc_node.data_ptr()), _stream(stream)), "w12_tree_accept")
    return acc_tok, acc_len, acc_node


class VerifyStep:
    """Marshalled arguments of ``w12_verify_step`` (kept alive between calls so
    the call can be captured in a CUDA graph and replayed)."""

    def __init__(self, linears: Sequence[DeviceWeight], xs, ys, head: DeviceWeight, h, argmax):
        self.linears, self.xs, self.ys, self.head, self.h, self.argmax = list(linears), list(xs), list(ys), head, h, argmax
        n = len(self.linears)
        self._lin = (Weight * max(n, 1))(*[w.c for w in self.linears])
        self._x = (C.c_void_p * max(n, 1))(*[x.data_ptr() for x in self.xs])
        self._y = (C.c_void_p * max(n, 1))(*[y.data_ptr() for y in self.ys])
        self.c = StepC(n, C.cast(self._lin, C.c_void_p), C.cast(self._x, C.c_void_p), C.cast(self._y, C.c_void_p),
                       C.cast(C.pointer(head.c), C.c_void_p), h.data_ptr(), argmax.data_ptr())


def w12_verify_step(step: VerifyStep, tree: DeviceTree, n_req: int, p_max: int, ws: Workspace, acc_tok, acc_len,
                    acc_node=None, stream=None):
    _check(lib().w12_verify_step(C.byref(step.c), C.byref(tree.c), n_req, p_max, C.c_void_p(acc_tok.data_ptr()),
                                 C.c_void_p(acc_len.data_ptr()), C.c_void_p(_dp(acc_node)) if acc_node is not None
                                 else None, ws.ptr, ws.nbytes, _stream(stream)), "w12_verify_step")


def w12_verify_step_q(step: VerifyStep, tree: DeviceTree, n_req: int, p_max: int, ws: Workspace, acc_tok,
                      acc_len, acc_node=None, stream=None):
    """The TLV Q pass: ``w12_verify_step`` on the quick weights; its
    acceptance outputs are the commit chain."""
    _check(lib().w12_verify_step_q(C.byref(step.c), C.byref(tree.c), n_req, p_max, C.c_void_p(acc_tok.data_ptr()),
                                   C.c_void_p(acc_len.data_ptr()), C.c_void_p(_dp(acc_node)) if acc_node is not None
                                   else None, ws.ptr, ws.nbytes, _stream(stream)), "w12_verify_step_q")


def w12_tlv_chain(c_len_host, t1_row_off_host, budget: int):
    """Host call: chain tokens committed per request and the subtree budget."""
    c_len = np.ascontiguousarray(c_len_host, np.int32)
    off = np.ascontiguousarray(t1_row_off_host, np.int32)
    n_req = len(c_len)
    if len(off) != n_req + 1:
        raise ValueError("t1_row_off needs n_req + 1 entries")
    m = np.empty(n_req, np.int32)
    sub = C.c_int32(0)
    _check(lib().w12_tlv_chain(_np(c_len), _np(off), n_req, int(budget), _np(m), C.byref(sub)), "w12_tlv_chain")
    return m, int(sub.value)


def w12_tlv_splice(t1: DeviceTree, c_tok, c_len, c_node, m_host, t2: DeviceTree, ws: Workspace,
                   out: Optional[DeviceTree] = None, stream=None) -> DeviceTree:
    """The combined tree of one TLV cycle (device)."""
    m = np.ascontiguousarray(m_host, np.int32)
    n_req = len(m)
    p1_max = int(c_tok.shape[1]) - 1
    if out is None:
        out = _under(stream, lambda: DeviceTree(max(1, int(m.sum()) + t2.R), n_req, device=c_tok.device))
    _check(lib().w12_tlv_splice(C.byref(t1.c), C.c_void_p(c_tok.data_ptr()), C.c_void_p(c_len.data_ptr()),
                                C.c_void_p(c_node.data_ptr()), n_req, p1_max, _np(m), C.byref(t2.c),
                                C.byref(out.c), ws.ptr, ws.nbytes, _stream(stream)), "w12_tlv_splice")
    return out


class GdnLayerC(C.Structure):
    _fields_ = [("n_heads", C.c_int32), ("head_dim", C.c_int32), ("S0", C.c_void_p), ("q", C.c_void_p),
                ("k", C.c_void_p), ("v", C.c_void_p), ("alpha", C.c_void_p), ("beta", C.c_void_p)]


W12_GDN_WY, W12_GDN_PATH = 0, 1


class GdnLayer:
    """Device inputs of one recurrent layer over a tree: committed states
    S0 (float32 [n_req][H][d][d]), q/k/v (bfloat16 [R][H][d]), alpha/beta
    (float32 [R][H]); kept alive with the marshalled struct."""

    def __init__(self, S0, q, k, v, alpha, beta):
        self.S0, self.q, self.k, self.v, self.alpha, self.beta = S0, q, k, v, alpha, beta
        self.H, self.d = int(q.shape[1]), int(q.shape[2])
        self.c = GdnLayerC(self.H, self.d, S0.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                           alpha.data_ptr(), beta.data_ptr())


def w12_gdn_tree_verify(layer: GdnLayer, tree: DeviceTree, n_req: int, ws: Workspace, method: int = W12_GDN_WY,
                        out=None, stream=None):
    import torch
    if out is None:
        out = _empty((tree.R, layer.H, layer.d), torch.float32, layer.q.device, stream)
    _check(lib().w12_gdn_tree_verify(C.byref(layer.c), C.byref(tree.c), int(n_req), int(method),
                                     C.c_void_p(out.data_ptr()), ws.ptr, ws.nbytes, _stream(stream)),
           "w12_gdn_tree_verify")
    return out


def w12_gdn_commit(layer: GdnLayer, tree: DeviceTree, n_req: int, acc_node, ws: Workspace, state=None, stream=None):
    import torch
    if state is None:
        state = _empty(layer.S0.shape, torch.float32, layer.S0.device, stream)
    _check(lib().w12_gdn_commit(C.byref(layer.c), C.byref(tree.c), int(n_req), C.c_void_p(acc_node.data_ptr()),
                                C.c_void_p(state.data_ptr()), ws.ptr, ws.nbytes, _stream(stream)), "w12_gdn_commit")
    return state


def w12_gdn_wy_verify(layer: GdnLayer, tree: DeviceTree, n_req: int, ws: Workspace, out=None, u=None, stream=None):
    """WY-form outputs and the WY vectors u (both float32 [R][H][d])."""
    import torch
    if out is None:
        out = _empty((tree.R, layer.H, layer.d), torch.float32, layer.q.device, stream)
    if u is None:
        u = _empty((tree.R, layer.H, layer.d), torch.float32, layer.q.device, stream)
    _check(lib().w12_gdn_wy_verify(C.byref(layer.c), C.byref(tree.c), int(n_req), C.c_void_p(out.data_ptr()),
                                   C.c_void_p(u.data_ptr()), ws.ptr, ws.nbytes, _stream(stream)), "w12_gdn_wy_verify")
    return out, u


def w12_gdn_wy_commit(layer: GdnLayer, tree: DeviceTree, n_req: int, acc_node, u, ws: Workspace, state=None,
                      stream=None):
    """The committed states from the WY vectors u of w12_gdn_wy_verify."""
    import torch
    if state is None:
        state = _empty(layer.S0.shape, torch.float32, layer.S0.device, stream)
    _check(lib().w12_gdn_wy_commit(C.byref(layer.c), C.byref(tree.c), int(n_req), C.c_void_p(acc_node.data_ptr()),
                                   C.c_void_p(u.data_ptr()), C.c_void_p(state.data_ptr()), ws.ptr, ws.nbytes,
                                   _stream(stream)), "w12_gdn_wy_commit")
    return state


# ---------------------------------------------------------------------------
# attention over a paged 8-bit KV cache
# ---------------------------------------------------------------------------

class KvCacheC(C.Structure):
    _fields_ = [("n_kv_heads", C.c_int32), ("head_dim", C.c_int32), ("block_tokens", C.c_int32),
                ("n_blocks", C.c_int32), ("max_blocks", C.c_int32), ("k", C.c_void_p), ("v", C.c_void_p),
                ("k_scale", C.c_void_p), ("v_scale", C.c_void_p), ("block_table", C.c_void_p), ("len", C.c_void_p)]


class RopeC(C.Structure):
    _fields_ = [("rot_dim", C.c_int32), ("adjacent", C.c_int32), ("max_pos", C.c_int32), ("cos", C.c_void_p),
                ("sin", C.c_void_p)]


def _want(t, dtype, shape, what):
    """A contiguous device tensor of this type and shape (None: any size)."""
    if t.dtype != dtype or t.dim() != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)) \
            or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous {dtype} {shape} wanted, got {t.dtype} {tuple(t.shape)}")


def _same_device(dev, what, *tensors):
    """All of a handle's tensors lie where its first one does."""
    if any(t is not None and t.get_device() != dev for t in tensors):
        raise ValueError(f"{what}: tensors of one device wanted")


def _refuse(dev, n_req, tree, *handles):
    """What a call turns away: a kernel gets bare addresses, so every handle's tensors have to lie on the call's GPU, and
    a tree has to have row offsets for every request.  (The calls compare by themselves, which takes them 0.1 us.)"""
    if dev < 0:
        raise ValueError("tensors of a CUDA device wanted")
    if tree is not None and tree.n_req < n_req:
        raise ValueError(f"tree: row offsets of {n_req} requests wanted, got {tree.n_req}")
    raise ValueError(f"{', '.join(type(h).__name__ for h in (tree, *handles) if h is not None)}: on cuda:{dev} wanted")


def _ints(t, n, what, dev) -> int:
    """The address of n contiguous int32."""
    if t.dtype is not _torch.int32 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{what}: contiguous int32 [{n}] on cuda:{dev} wanted, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t, rows, width, what, dev):
    """(address, elements between rows) of `rows` or more bfloat16 rows of `width` contiguous elements."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not _torch.bfloat16 or len(shape) != 2 or shape[1] != width or shape[0] < rows \
            or (stride[1] != 1 and shape[0]) or t.get_device() != dev:
        raise ValueError(f"{what}: bfloat16 rows [>= {rows}][{width}] with contiguous elements on cuda:{dev} wanted, got "
                         f"{t.dtype} {tuple(shape)} on {t.device}")
    return t.data_ptr(), stride[0] if shape[0] > 1 else max(stride[0], width)


class KvCache:
    """A paged KV cache: E4M3 codes k (uint8 [n_blocks][H][block_tokens][128])
    and v (uint8 [n_blocks][H][128][block_tokens]), power-of-two scales
    (float32 [n_blocks][H]), the block table (int32 [n_req][max_blocks]) and
    the committed lengths (int32 [n_req]).  The tensors stay the caller's."""

    def __init__(self, k, v, k_scale, v_scale, block_table, length):
        torch = _runtime()
        lib()
        n, H, bt, d = k.shape
        _want(k, torch.uint8, (n, H, bt, d), "k")
        _want(v, torch.uint8, (n, H, d, bt), "v")
        _want(k_scale, torch.float32, (n, H), "k_scale")
        _want(v_scale, torch.float32, (n, H), "v_scale")
        _want(block_table, torch.int32, (None, None), "block_table")
        _want(length, torch.int32, (block_table.shape[0],), "length")
        self.dev = k.get_device()
        _same_device(self.dev, "cache", v, k_scale, v_scale, block_table, length)
        self.k, self.v, self.k_scale, self.v_scale, self.block_table, self.len = k, v, k_scale, v_scale, block_table, length
        self.n_req, self.H, self.bt, self.d = int(block_table.shape[0]), int(H), int(bt), int(d)
        self.c = KvCacheC(H, d, bt, n, block_table.shape[1], k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                          v_scale.data_ptr(), block_table.data_ptr(), length.data_ptr())
        self.ref = C.byref(self.c)

    @classmethod
    def empty(cls, n_blocks, n_kv_heads, block_tokens, block_table, device="cuda"):
        """A zeroed pool of n_blocks blocks; every request starts without tokens."""
        import torch
        z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt, device=device)
        return cls(z(n_blocks, n_kv_heads, block_tokens, 128), z(n_blocks, n_kv_heads, 128, block_tokens),
                   torch.ones(n_blocks, n_kv_heads, device=device), torch.ones(n_blocks, n_kv_heads, device=device),
                   block_table, z(block_table.shape[0], dt=torch.int32))


class Rope:
    """Position tables: cos and sin, float32 [max_pos][rot_dim / 2]; pairs
    (i, i + rot_dim / 2), or (2 i, 2 i + 1) with ``adjacent``."""

    def __init__(self, cos, sin, adjacent: bool = False):
        import torch
        _want(cos, torch.float32, (None, None), "cos")
        _want(sin, torch.float32, tuple(cos.shape), "sin")
        self.cos, self.sin, self.dev = cos, sin, cos.get_device()
        _same_device(self.dev, "position tables", sin)
        self.c = RopeC(2 * cos.shape[1], int(adjacent), cos.shape[0], cos.data_ptr(), sin.data_ptr())
        self.ref = C.byref(self.c)


class AttentionWorkspace:
    """Device scratch of ``w12_tree_attention`` for up to R rows of n_req requests."""

    def __init__(self, R: int, n_heads: int, n_kv_heads: int, n_req: int, device="cuda"):
        import torch
        self.nbytes = int(lib().w12_attn_workspace_bytes(int(R), int(n_heads), int(n_kv_heads), int(n_req)))
        if self.nbytes == 0:
            raise W12Error(W12_E_UNSUPPORTED, "w12_attn_workspace_bytes")
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.addr, self.dev = self.buf.data_ptr(), self.buf.get_device()


def w12_kv_append(cache: KvCache, rope: Optional[Rope], k, v, row_off, ws: Workspace, len_out=None, stream=None):
    """Append rows row_off[r]..row_off[r+1]-1 of k and v (bfloat16 [T][H * 128],
    row slices allowed) to every request's tokens; the new lengths go to
    ``len_out`` (default: in place)."""
    n, T, width = cache.n_req, k.shape[0], cache.H * cache.d
    if v.shape[0] != T:
        raise ValueError("k and v: the same number of rows wanted")
    if len_out is None:
        len_out = cache.len
    dev = cache.dev
    if dev < 0 or ws.dev != dev or (rope is not None and rope.dev != dev):
        _refuse(dev, n, None, rope, ws)
    s = _lib.w12_kv_append(cache.ref, rope.ref if rope else None, n, *_rows(k, T, width, "k", dev), *_rows(v, T, width, "v", dev),
                           T, _ints(row_off, n + 1, "row_off", dev), _ints(len_out, n, "len_out", dev), ws.addr, ws.nbytes,
                           _st(stream))
    if s:
        raise W12Error(s, "w12_kv_append")
    return len_out


def w12_kv_commit(cache: KvCache, rope: Optional[Rope], tree: DeviceTree, n_req: int, acc_node, k, v, ws: Workspace,
                  len_out=None, stream=None):
    """Append the accepted path of every request (root .. acc_node[r]) to its
    tokens; k and v are the tree's rows."""
    if n_req != cache.n_req:
        raise ValueError("the cache's table and the tree: the same requests wanted")
    if len_out is None:
        len_out = cache.len
    R, width = tree.c.R, cache.H * cache.d
    dev = cache.dev
    if dev < 0 or ws.dev != dev or tree.dev != dev or tree.n_req < n_req or (rope is not None and rope.dev != dev):
        _refuse(dev, n_req, tree, rope, ws)
    s = _lib.w12_kv_commit(cache.ref, rope.ref if rope else None, C.byref(tree.c), n_req, _ints(acc_node, n_req, "acc_node", dev),
                           *_rows(k, R, width, "k", dev), *_rows(v, R, width, "v", dev), _ints(len_out, n_req, "len_out", dev),
                           ws.addr, ws.nbytes, _st(stream))
    if s:
        raise W12Error(s, "w12_kv_commit")
    return len_out


def w12_tree_attention(cache: KvCache, rope: Optional[Rope], tree: DeviceTree, n_req: int, q, k, v, ws: Workspace,
                       aws: AttentionWorkspace, scale: Optional[float] = None, out=None, stream=None):
    """Attention of the tree's rows over the cache and their root paths ->
    bfloat16 [R][n_heads][128].  q (bfloat16 [R][n_heads * 128]), k, v: the
    linears' rows before rotation (slices of a fused row are fine); scale:
    default 128 ** -0.5."""
    if n_req != cache.n_req:
        raise ValueError("the cache's table and the tree: the same requests wanted")
    R, d, width, width_q = tree.c.R, cache.d, cache.H * cache.d, q.shape[-1]
    Hq = width_q // d
    dev = cache.dev
    if dev < 0 or ws.dev != dev or aws.dev != dev or tree.dev != dev or tree.n_req < n_req or \
            (rope is not None and rope.dev != dev):
        _refuse(dev, n_req, tree, rope, ws, aws)
    if out is None:
        out = _empty((R, Hq, d), _torch.bfloat16, q.device, stream)
    elif out.shape[0] < R or out.shape[1:] != (Hq, d) or out.dtype is not _torch.bfloat16 or not out.is_contiguous() \
            or out.get_device() != dev:
        raise ValueError(f"out: contiguous bfloat16 [{R}][{Hq}][{d}] on cuda:{dev} wanted")
    s = _lib.w12_tree_attention(cache.ref, rope.ref if rope else None, C.byref(tree.c), n_req, Hq, *_rows(q, R, Hq * d, "q", dev),
                                *_rows(k, R, width, "k", dev), *_rows(v, R, width, "v", dev),
                                d ** -0.5 if scale is None else scale, out.data_ptr(), ws.addr, ws.nbytes, aws.addr, aws.nbytes,
                                _st(stream))
    if s:
        raise W12Error(s, "w12_tree_attention")
    return out


# ---------------------------------------------------------------------------
# the recurrent layer over prompts and single tokens, norms around a block
# ---------------------------------------------------------------------------

class GdnRowsC(C.Structure):
    _fields_ = [("n_heads", C.c_int32), ("n_qk_heads", C.c_int32), ("head_dim", C.c_int32), ("n_rows", C.c_int32),
                ("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("q_stride", C.c_int64), ("k_stride", C.c_int64),
                ("v_stride", C.c_int64), ("alpha", C.c_void_p), ("beta", C.c_void_p), ("scratch", C.c_void_p),
                ("scratch_bytes", C.c_size_t)]


class GdnScratch:
    """Device buffer for ``w12_gdn_prefill`` on rows of up to n_rows tokens and n_heads heads (20 MB at most), for several
    layers' ``GdnRows`` whose calls run in order."""

    def __init__(self, n_heads: int, n_rows: int, device="cuda"):
        torch = _runtime()
        self.nbytes = int(lib().w12_gdn_scratch_bytes(int(n_heads), int(n_rows)))
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        self.streams = set()                     # on which it has been used


class GdnRows:
    """A recurrent layer's token rows: q and k (bfloat16 [T][n_qk_heads * 128]),
    v (bfloat16 [T][H * 128]; slices of a fused row are fine), gates alpha and
    write strengths beta (float32 [T][H]).  Value head h reads query/key head
    h // (H // n_qk_heads).  The tensors stay the caller's.
    Holds the scratch of ``w12_gdn_prefill``, its own or one that other layers' rows share; the calls that use one
    run in order, and a captured call needs the object for as long as its graph is replayed."""

    def __init__(self, q, k, v, alpha, beta, scratch: Optional[GdnScratch] = None):
        torch = _runtime()
        lib()
        _want(alpha, torch.float32, (None, None), "alpha")
        T, H = alpha.shape
        _want(beta, torch.float32, (T, H), "beta")
        self.dev = alpha.get_device()
        if q.dim() != 2 or q.shape[0] != T or k.shape[0] != T or v.shape[0] != T:
            raise ValueError(f"q, k, v: {T} rows wanted, as alpha has")
        if H < 1 or q.shape[1] < 128 or q.shape[1] % 128 or H % (q.shape[1] // 128):
            raise ValueError(f"q: rows of whole heads of 128 wanted that {H} value heads share evenly, got {q.shape[1]}")
        _same_device(self.dev, "rows", beta, q, k, v)
        self.q, self.k, self.v, self.alpha, self.beta = q, k, v, alpha, beta
        self.T, self.H, self.d = int(T), int(H), 128
        (qa, qs), (ka, ks), (va, vs) = (_rows(t, T, w, n, self.dev) for t, w, n in
                                        ((q, q.shape[1], "q"), (k, q.shape[1], "k"), (v, H * 128, "v")))
        self.c = GdnRowsC(H, q.shape[1] // 128, 128, T, qa, ka, va, qs, ks, vs, alpha.data_ptr(), beta.data_ptr(), None, 0)
        self.scratch, self._streams = None, set()   # for w12_gdn_prefill, made by its first call; on which it has been used
        if scratch is not None:
            need = int(_lib.w12_gdn_scratch_bytes(self.H, self.T))
            if scratch.nbytes < need or scratch.buf.get_device() != self.dev:
                raise ValueError(f"scratch: {need} bytes on cuda:{self.dev} wanted, got {scratch.nbytes} on {scratch.buf.device}")
            self.scratch, self._streams = scratch.buf, scratch.streams
            if scratch.nbytes:
                self.c.scratch, self.c.scratch_bytes = scratch.buf.data_ptr(), scratch.nbytes
        self.ref = C.byref(self.c)

    def _scratch_on(self, st, stream):
        """The scratch, made by the first call.  The allocator learns of every stream that uses it, so that it becomes nobody
        else's while a call still runs."""
        if self.scratch is None:
            nbytes = int(_lib.w12_gdn_scratch_bytes(self.H, self.T))
            self.scratch = _empty((nbytes,), _torch.uint8, self.alpha.device, stream)
            if nbytes:
                self.c.scratch, self.c.scratch_bytes = self.scratch.data_ptr(), nbytes
        _used_on(self._streams, st, stream, self.scratch)

    def _buffers(self, n_req, S0, state, out, stream):
        """The calls' state and output tensors, made or checked."""
        dev, shape = self.dev, (n_req, self.H, self.d, self.d)
        if dev < 0:
            _refuse(dev, n_req, None, self)
        new = lambda *s: _empty(s, _torch.float32, self.alpha.device, stream)
        state = new(*shape) if state is None else state
        out = new(self.T, self.H, self.d) if out is None else out
        for t, what, want in ((S0, "S0", shape), (state, "state", shape), (out, "out", (self.T, self.H, self.d))):
            if t is not None and (t.dtype is not _torch.float32 or t.shape != want or not t.is_contiguous()
                                  or t.get_device() != dev):
                raise ValueError(f"{what}: contiguous float32 {tuple(want)} on cuda:{dev} wanted, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}")
        return state, out


def w12_gdn_prefill(rows: GdnRows, row_off, ws: Workspace, S0=None, state=None, out=None, stream=None):
    """Rows row_off[r]..row_off[r+1]-1 (int32 [n_req + 1]) continue request
    r's state -> (out, state): every row's output (float32 [T][H][128]) and the
    states behind the last rows (float32 [n_req][H][128][128] as S[v][k]).  S0: the
    states in front (default: zero); state may be S0 itself."""
    n = row_off.shape[0] - 1
    if n < 1:
        raise ValueError("row_off: int32 [n_req + 1] wanted")
    state, out = rows._buffers(n, S0, state, out, stream)
    if ws.dev != rows.dev:
        _refuse(rows.dev, n, None, ws)
    st = _st_on(rows.dev, stream)
    if st not in rows._streams:
        rows._scratch_on(st, stream)
    s = _lib.w12_gdn_prefill(rows.ref, n, _ints(row_off, n + 1, "row_off", rows.dev), _dp(S0), state.data_ptr(),
                             out.data_ptr(), ws.addr, ws.nbytes, st)
    if s:
        raise W12Error(s, "w12_gdn_prefill")
    return out, state


def w12_gdn_step(rows: GdnRows, S0=None, state=None, out=None, stream=None):
    """One token of every request: row r continues request r's state -> (out,
    state), as for ``w12_gdn_prefill``."""
    state, out = rows._buffers(rows.T, S0, state, out, stream)
    s = _lib.w12_gdn_step(rows.ref, _dp(S0), state.data_ptr(), out.data_ptr(), _st_on(rows.dev, stream))
    if s:
        raise W12Error(s, "w12_gdn_step")
    return out, state


def w12_gdn_norm(o, weight, z=None, eps: float = 1e-6, gate_first: bool = False, out=None, stream=None):
    """The recurrent layer's outputs o (float32 [R][H][128]) as the next linear
    reads them -> bfloat16 [R][H * 128]: rms(o) * weight * silu(z) per head, with
    ``gate_first`` rms(o * silu(z)) * weight.  weight: bfloat16 [128]; z:
    bfloat16 rows [R][H * 128] (slices of a fused row are fine), optional."""
    if _torch is None:
        _runtime()
        lib()
    shape, dev = o.shape, o.get_device()
    if len(shape) != 3 or shape[2] != 128 or o.dtype is not _torch.float32 or dev < 0 or not o.is_contiguous():
        raise ValueError(f"o: contiguous float32 [rows][heads][128] of a CUDA device wanted, got {o.dtype} {tuple(shape)} on {o.device}")
    R, H, _ = shape
    width = H * 128
    if out is None:
        out = _empty((R, width), _torch.bfloat16, o.device, stream)
    za, zs = (None, 0) if z is None else _rows(z, R, width, "z", dev)
    oa, os_ = _rows(out, R, width, "out", dev)
    s = _lib.w12_gdn_norm(o.data_ptr(), R, H, 128, za, zs, _vector(weight, 128, "weight", dev), eps, gate_first, oa, os_,
                          _st_on(dev, stream))
    if s:
        raise W12Error(s, "w12_gdn_norm")
    return out


def _vector(t, n, what, dev):
    """The address of n contiguous bfloat16."""
    if t.dtype is not _torch.bfloat16 or t.shape != (n,) or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous bfloat16 [{n}] on cuda:{dev} wanted, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


class ResidualC(C.Structure):
    _fields_ = [("n_rows", C.c_int32), ("h_f32", C.c_int32), ("n", C.c_int64), ("h", C.c_void_p), ("h_stride", C.c_int64),
                ("h_out", C.c_void_p), ("h_out_stride", C.c_int64), ("y", C.c_void_p), ("y_stride", C.c_int64),
                ("post", C.c_void_p), ("scale", C.c_float), ("pre", C.c_void_p), ("eps", C.c_float), ("x", C.c_void_p),
                ("x_stride", C.c_int64)]


_residual = struct.Struct("@iiqPqPqPqPfPfPq").pack      # ResidualC's bytes (a third of the time that filling one takes)


def _stream_rows(t, rows, width, f32, what, dev):
    """_rows of a residual stream, bfloat16 or float32."""
    if not f32:
        return _rows(t, rows, width, what, dev)
    shape, stride = t.shape, t.stride()
    if t.dtype is not _torch.float32 or len(shape) != 2 or shape[1] != width or shape[0] < rows \
            or (stride[1] != 1 and shape[0]) or t.get_device() != dev:
        raise ValueError(f"{what}: float32 rows [>= {rows}][{width}] with contiguous elements on cuda:{dev} wanted, got "
                         f"{t.dtype} {tuple(shape)} on {t.device}")
    return t.data_ptr(), stride[0] if shape[0] > 1 else max(stride[0], width)


def w12_block_norm(h, y=None, pre=None, post=None, scale: float = 1.0, eps: float = 1e-6, h_out=None, out=None, stream=None):
    """Between two blocks -> (h', x): h' = h + scale * t with t = y, or
    rms(y) * post; x = rms(h') * pre (bfloat16), of h' before it is rounded.
    h: the residual stream, bfloat16 or float32 rows [R][n]; y: the block's
    output, bfloat16 rows (None: h' = h); pre, post: bfloat16 [n] (None: no norm
    there, and without pre no x).  h' goes to ``h_out`` (default: new rows; may
    be h), x to ``out``."""
    if _torch is None:
        _runtime()
        lib()
    shape, dev, f32 = h.shape, h.get_device(), h.dtype is _torch.float32
    if len(shape) != 2 or dev < 0:
        raise ValueError("h: rows of a CUDA device wanted")
    R, n = shape
    ha, hs = _stream_rows(h, R, n, f32, "h", dev)
    ya = ys = oa = os_ = xa = xs = posta = prea = 0
    if y is None:
        if h_out is not None or post is not None:
            raise ValueError("h_out and post: only with y")
        h_out = h
    else:
        ya, ys = _rows(y, R, n, "y", dev)
        if post is not None:
            posta = _vector(post, n, "post", dev)
        if h_out is None:
            h_out = _empty((R, n), h.dtype, h.device, stream)
        oa, os_ = _stream_rows(h_out, R, n, f32, "h_out", dev)
    if pre is not None:
        if out is None:
            out = _empty((R, n), _torch.bfloat16, h.device, stream)
        xa, xs = _rows(out, R, n, "out", dev)
        prea = _vector(pre, n, "pre", dev)
    elif out is not None:
        raise ValueError("out: only with pre")
    s = _lib.w12_block_norm(_residual(R, f32, n, ha, hs, oa, os_, ya, ys, posta, scale, prea, eps, xa, xs), _st_on(dev, stream))
    if s:
        raise W12Error(s, "w12_block_norm")
    return h_out, out


# ---------------------------------------------------------------------------
# sampled verification
# ---------------------------------------------------------------------------

class SamplingC(C.Structure):
    _fields_ = [("logits", C.c_void_p), ("logits_f32", C.c_int32), ("vocab", C.c_int64), ("logits_stride", C.c_int64),
                ("temperature", C.c_void_p), ("draft_p", C.c_void_p), ("draft_stride", C.c_int64),
                ("u_accept", C.c_void_p), ("u_sample", C.c_void_p), ("scratch", C.c_void_p), ("scratch_rows", C.c_int32)]


class SampleRows:
    """The target's logits (bfloat16 or float32 [R][vocab]) and the random
    numbers of one sampled verification: u_sample (float32 [R]), temperature
    (float32 [n_req], optional; 0 = greedy) and, for a drafter that samples,
    its probabilities draft_p (float32 [R][vocab]) with u_accept (float32 [R]).
    Holds the calls' scratch; one object's calls run in order."""

    def __init__(self, logits, u_sample, temperature=None, draft_p=None, u_accept=None):
        torch = _runtime()
        lib()
        R, V = logits.shape
        if logits.dtype not in (torch.bfloat16, torch.float32) or logits.stride(1) != 1:
            raise ValueError("logits: bfloat16 or float32 [R][vocab] with contiguous elements wanted")
        _want(u_sample, torch.float32, (R,), "u_sample")
        if temperature is not None:
            _want(temperature, torch.float32, (None,), "temperature")
        if draft_p is not None:
            if draft_p.dtype != torch.float32 or draft_p.shape != logits.shape or draft_p.stride(1) != 1:
                raise ValueError("draft_p: float32 [R][vocab] with contiguous elements wanted")
            if u_accept is None:
                raise ValueError("draft_p needs u_accept")
        if u_accept is not None:
            _want(u_accept, torch.float32, (R,), "u_accept")
        self.dev = logits.get_device()
        _same_device(self.dev, "logits and random numbers", u_sample, temperature, draft_p, u_accept)
        self.logits, self.u_sample, self.temperature, self.draft_p, self.u_accept = \
            logits, u_sample, temperature, draft_p, u_accept
        row = lambda t: t.stride(0) if R > 1 else max(t.stride(0), V)
        rows = min(R, 512)                       # of a tree at most
        nbytes = int(lib().w12_sample_scratch_bytes(rows, V))
        if nbytes == 0:
            raise W12Error(W12_E_UNSUPPORTED, "w12_sample_scratch_bytes")
        self.scratch, self._streams = torch.empty(nbytes, dtype=torch.uint8, device=logits.device), set()
        self.c = SamplingC(logits.data_ptr(), int(logits.dtype == torch.float32), V, row(logits), _dp(temperature),
                           _dp(draft_p), row(draft_p) if draft_p is not None else 0, _dp(u_accept), _dp(u_sample),
                           self.scratch.data_ptr(), rows)
        self.ref = C.byref(self.c)
        self.rows = R
        self.requests = None if temperature is None else int(temperature.shape[0])

    def _fits(self, tree, n_req, ws):
        dev = self.dev
        if dev < 0 or ws.dev != dev or tree.dev != dev or tree.n_req < n_req:
            _refuse(dev, n_req, tree, ws)
        if self.rows < tree.c.R or (self.requests is not None and self.requests < n_req):
            raise ValueError("logits: a row for every row of the tree wanted, and a temperature for every request")
        return dev


def w12_tree_sample(dist: SampleRows, tree: DeviceTree, n_req: int, ws: Workspace, row_tok=None, row_logp=None,
                    stream=None):
    """One token per tree row, distributed as the target's probabilities
    there -> int32 [R]; its log-probability to ``row_logp`` (float32 [R])."""
    dev = dist._fits(tree, n_req, ws)
    R = tree.c.R
    if row_tok is None:
        row_tok = _empty((R,), _torch.int32, dist.logits.device, stream)
    st = _st(stream)
    if st not in dist._streams:
        _used_on(dist._streams, st, stream, dist.scratch)
    s = _lib.w12_tree_sample(dist.ref, C.byref(tree.c), n_req, _ints(row_tok, R, "row_tok", dev), _floats(row_logp, R, dev),
                             ws.addr, ws.nbytes, st)
    if s:
        raise W12Error(s, "w12_tree_sample")
    return row_tok


def _floats(t, n, dev):
    if t is None:
        return None
    if t.dtype is not _torch.float32 or t.shape != (n,) or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"row_logp: contiguous float32 [{n}] on cuda:{dev} wanted")
    return t.data_ptr()


def w12_tree_verify_sampled(dist: SampleRows, tree: DeviceTree, n_req: int, p_max: int, ws: Workspace, row_tok=None,
                            row_logp=None, acc_tok=None, acc_len=None, acc_node=None, stream=None):
    """``w12_tree_sample`` and the acceptance of the children that carry their
    parent's token -> acc_tok, acc_len, acc_node."""
    dev = dist._fits(tree, n_req, ws)
    R = tree.c.R
    if row_tok is None or acc_tok is None or acc_len is None or acc_node is None:
        new = lambda *s: _empty(s, _torch.int32, dist.logits.device, stream)
        row_tok = row_tok if row_tok is not None else new(R)
        acc_tok = acc_tok if acc_tok is not None else new(n_req, p_max + 1)
        acc_len = acc_len if acc_len is not None else new(n_req)
        acc_node = acc_node if acc_node is not None else new(n_req)
    if acc_tok.shape != (n_req, p_max + 1) or acc_tok.dtype is not _torch.int32 or not acc_tok.is_contiguous() \
            or acc_tok.get_device() != dev:
        raise ValueError(f"acc_tok: contiguous int32 [{n_req}][{p_max + 1}] on cuda:{dev} wanted")
    st = _st(stream)
    if st not in dist._streams:
        _used_on(dist._streams, st, stream, dist.scratch)
    s = _lib.w12_tree_verify_sampled(dist.ref, C.byref(tree.c), n_req, p_max, _ints(row_tok, R, "row_tok", dev),
                                     _floats(row_logp, R, dev), acc_tok.data_ptr(), _ints(acc_len, n_req, "acc_len", dev),
                                     _ints(acc_node, n_req, "acc_node", dev), ws.addr, ws.nbytes, st)
    if s:
        raise W12Error(s, "w12_tree_verify_sampled")
    return acc_tok, acc_len, acc_node


def debug_set(flags: int = 0, timeout_ns: int = 0):
    lib().w12_debug_set(int(flags), int(timeout_ns))


def profile(enable: bool):
    lib().w12_debug_profile(1 if enable else 0)


def profile_read(max_launches: int = 1024) -> List[float]:
    buf = (C.c_float * max_launches)()
    n = int(lib().w12_debug_profile_read(buf, max_launches))
    if n < 0:
        raise W12Error(n, "w12_debug_profile_read")
    return [float(buf[i]) for i in range(min(n, max_launches))]


def num_sms() -> int:
    return int(lib().w12_debug_num_sms())


class ChainTrace:
    """Per-GEMM end times inside the verify step's GEMM chain (debug hook):
    while enabled, each chain launch stamps the global timer per CTA at its
    start and when the CTA has written its last output of each GEMM."""

    def __init__(self, n_gemms: int, device="cuda"):
        import torch
        self.n = int(n_gemms)
        self.parts = int(lib().w12_debug_chain_parts(self.n))
        self.S = num_sms()
        self.buf = torch.zeros(((self.n + self.parts) * self.S,), dtype=torch.int64, device=device)

    def __enter__(self):
        lib().w12_debug_chain_trace(C.c_void_p(self.buf.data_ptr()), self.buf.numel())
        return self

    def __exit__(self, *exc):
        lib().w12_debug_chain_trace(None, 0)

    def gemm_us(self) -> List[float]:
        """Per GEMM: the time from the previous GEMM's end (for each launch's
        first GEMM, from the launch's first CTA start) to the last CTA's stamp."""
        t = self.buf.view(self.n + self.parts, self.S).cpu().numpy().astype(np.float64)
        out, j0 = [], 0
        for k in range(self.parts):
            m = (self.n - j0) // (self.parts - k)
            rows = t[j0 + k: j0 + k + m]
            start = t[j0 + k + m]
            starts = start[start > 0]
            prev = starts.min() if starts.size else rows[0].max()
            for r in rows:
                end = r.max()
                out.append((end - prev) / 1e3)
                prev = end
            j0 += m
        return out
