"""MoBA (Mixture of Block Attention) causal prefill on B200: Python binding of libmoba.so.

The binding only marshals arguments: every step of the forward pass runs in the
library's sm_100a kernels.  PyTorch provides device memory and streams.  There is
no fallback: if the CUDA library is missing, every call raises.

C-ABI entry points (same names here): ``moba_pool_keys``, ``moba_gate_topk``,
``moba_attn_fwd``, ``moba_fwd``, ``moba_workspace_size``, ``moba_kbar_elems``.
The paged 8-bit KV cache: ``moba_cache_tables``, ``moba_cache_append``,
``moba_cache_decode_fwd``, and ``MobaCache``, which owns one cache's buffers.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoba.so")
_lib = None

STATUS = {0: "MOBA_OK", 1: "MOBA_ERR_INVALID_ARG", 2: "MOBA_ERR_UNSUPPORTED",
          3: "MOBA_ERR_ALIGNMENT", 4: "MOBA_ERR_WORKSPACE", 5: "MOBA_ERR_CUDA",
          6: "MOBA_ERR_DEVICE"}

EXPORTS = ("moba_kbar_elems", "moba_workspace_size", "moba_pool_keys", "moba_gate_topk",
           "moba_attn_fwd", "moba_fwd", "moba_route", "moba_attn_past", "moba_attn_self_merge",
           "moba_launches_per_forward", "moba_read_device_error", "moba_status_string",
           "moba_last_error", "moba_gate_topk_noalloc", "moba_selftest_bounded_wait",
           "moba_host_staging_size", "moba_fwd_host", "moba_attn_naive", "moba_decode_workspace_size",
           "moba_decode_fwd", "moba_pool_last_block", "moba_bwd_workspace_size", "moba_attn_bwd",
           "moba_cache_tables", "moba_cache_append", "moba_cache_decode_workspace_size", "moba_cache_decode_fwd")

CACHE_FORMATS = {"e4m3": 0, "int8": 1}


class MobaError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__("%s: %s" % (STATUS.get(status, status), detail))
        self.status = status


class _CParams(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("cu_seqlens_host", ctypes.POINTER(ctypes.c_int32)),
        ("cu_seqlens", ctypes.c_void_p),
        ("max_seqlen", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
    ]


class _CCacheParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("max_seqs", "max_seqlen", "num_pages", "page_size", "num_q_heads", "num_kv_heads", "head_dim",
                 "block_size", "top_k", "format")] + [("softmax_scale", ctypes.c_float)]


def load():
    """Load libmoba.so (built in-tree by ``build.py``); raise if it is absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoba.so is not built (%s); run block_sparse_attention_gate_b200/build.py"
                               % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(_CParams)
        vp = ctypes.c_void_p
        sz = ctypes.c_size_t
        lib.moba_kbar_elems.argtypes = [P]
        lib.moba_kbar_elems.restype = sz
        lib.moba_workspace_size.argtypes = [P]
        lib.moba_workspace_size.restype = sz
        lib.moba_pool_keys.argtypes = [P, vp, vp, vp]
        lib.moba_gate_topk.argtypes = [P, vp, vp, vp, vp, sz, vp]
        lib.moba_attn_fwd.argtypes = [P, vp, vp, vp, vp, vp, sz, vp, vp, vp]
        lib.moba_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp]
        lib.moba_route.argtypes = [P, vp, vp, sz, vp]
        lib.moba_attn_past.argtypes = [P, vp, vp, vp, vp, sz, vp]
        lib.moba_attn_self_merge.argtypes = [P, vp, vp, vp, vp, vp, sz, vp, vp, vp]
        lib.moba_bwd_workspace_size.argtypes = [P]
        lib.moba_bwd_workspace_size.restype = sz
        lib.moba_attn_bwd.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp, vp]
        lib.moba_attn_bwd.restype = ctypes.c_int
        lib.moba_decode_workspace_size.argtypes = [P]
        lib.moba_decode_workspace_size.restype = sz
        lib.moba_decode_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp]
        lib.moba_decode_fwd.restype = ctypes.c_int
        lib.moba_pool_last_block.argtypes = [P, vp, vp, vp]
        lib.moba_pool_last_block.restype = ctypes.c_int
        lib.moba_attn_naive.argtypes = [P, vp, vp, vp, vp, vp, vp, vp]
        lib.moba_attn_naive.restype = ctypes.c_int
        lib.moba_gate_topk_noalloc.argtypes = [P, vp, vp, vp, vp]
        lib.moba_gate_topk_noalloc.restype = ctypes.c_int
        lib.moba_host_staging_size.argtypes = [P, ctypes.c_int]
        lib.moba_host_staging_size.restype = sz
        lib.moba_fwd_host.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, ctypes.POINTER(ctypes.c_void_p), ctypes.c_int]
        lib.moba_fwd_host.restype = ctypes.c_int
        lib.moba_launches_per_forward.argtypes = [P]
        lib.moba_launches_per_forward.restype = ctypes.c_int
        for f in ("moba_pool_keys", "moba_gate_topk", "moba_attn_fwd", "moba_fwd", "moba_route",
                  "moba_attn_past", "moba_attn_self_merge"):
            getattr(lib, f).restype = ctypes.c_int
        C = ctypes.POINTER(_CCacheParams)
        i64 = ctypes.c_int64
        i32 = ctypes.c_int32
        lib.moba_cache_tables.argtypes = [C] + [vp] * 9 + [i32, vp, vp]
        lib.moba_cache_tables.restype = ctypes.c_int
        lib.moba_cache_append.argtypes = [C, vp, i64, vp, i64, i32] + [vp] * 10
        lib.moba_cache_append.restype = ctypes.c_int
        lib.moba_cache_decode_workspace_size.argtypes = [C]
        lib.moba_cache_decode_workspace_size.restype = sz
        lib.moba_cache_decode_fwd.argtypes = [C] + [vp] * 10 + [sz, vp, vp, vp]
        lib.moba_cache_decode_fwd.restype = ctypes.c_int
        lib.moba_selftest_bounded_wait.argtypes = [ctypes.POINTER(ctypes.c_int32)]
        lib.moba_selftest_bounded_wait.restype = ctypes.c_int
        lib.moba_read_device_error.argtypes = [ctypes.POINTER(ctypes.c_int32), ctypes.c_int]
        lib.moba_read_device_error.restype = ctypes.c_int
        lib.moba_status_string.argtypes = [ctypes.c_int]
        lib.moba_status_string.restype = ctypes.c_char_p
        lib.moba_last_error.argtypes = []
        lib.moba_last_error.restype = ctypes.c_char_p
        _lib = lib
    return _lib


class MobaParams:
    """Host-side moba_params plus the buffers it points at (kept alive here)."""

    def __init__(self, cu_seqlens_host, num_q_heads: int, num_kv_heads: int, head_dim: int,
                 block_size: int, top_k: int, cu_seqlens_device=None, softmax_scale: float = 0.0,
                 num_seqs: int | None = None, max_seqlen: int = 0):
        c = _CParams()
        if cu_seqlens_host is not None:
            self.cu_host = np.ascontiguousarray(np.asarray(cu_seqlens_host), dtype=np.int32)
            c.num_seqs = self.cu_host.size - 1
            c.cu_seqlens_host = self.cu_host.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
            if cu_seqlens_device is None:
                import torch
                cu_seqlens_device = torch.from_numpy(self.cu_host.copy()).cuda()
            self.cu_dev = cu_seqlens_device
            c.cu_seqlens = cu_seqlens_device.data_ptr()
            self.total_tokens = int(self.cu_host[-1])
        else:
            self.cu_host = None
            self.cu_dev = None
            c.num_seqs = int(num_seqs)
            c.max_seqlen = int(max_seqlen)
            self.total_tokens = int(num_seqs) * int(max_seqlen)
        c.num_q_heads = num_q_heads
        c.num_kv_heads = num_kv_heads
        c.head_dim = head_dim
        c.block_size = block_size
        c.top_k = top_k
        c.softmax_scale = softmax_scale
        self.c = c

    def ref(self):
        return ctypes.byref(self.c)

    @property
    def kbar_elems(self) -> int:
        return moba_kbar_elems(self)

    @property
    def workspace_bytes(self) -> int:
        return moba_workspace_size(self)

    @property
    def max_blocks(self) -> int:
        h, d = self.c.num_kv_heads, self.c.head_dim
        return self.kbar_elems // (self.c.num_seqs * h * d)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _check(rc: int):
    if rc != 0:
        raise MobaError(rc, load().moba_last_error().decode())


def moba_kbar_elems(p: MobaParams) -> int:
    return int(load().moba_kbar_elems(p.ref()))


def moba_workspace_size(p: MobaParams) -> int:
    return int(load().moba_workspace_size(p.ref()))


def moba_pool_keys(p: MobaParams, K, Kbar, stream=None) -> None:
    _check(load().moba_pool_keys(p.ref(), _ptr(K), _ptr(Kbar), _stream(stream)))


def moba_gate_topk(p: MobaParams, Q, Kbar, sel, workspace, stream=None) -> None:
    _check(load().moba_gate_topk(p.ref(), _ptr(Q), _ptr(Kbar), _ptr(sel), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))


def moba_attn_fwd(p: MobaParams, Q, K, V, sel, workspace, O, LSE, stream=None) -> None:
    _check(load().moba_attn_fwd(p.ref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(sel), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _ptr(O), _ptr(LSE),
                                _stream(stream)))


def moba_fwd(p: MobaParams, Q, K, V, workspace, O, LSE, Kbar=None, sel=None, stream=None) -> None:
    _check(load().moba_fwd(p.ref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(Kbar), _ptr(sel), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), _ptr(O), _ptr(LSE),
                           _stream(stream)))


def moba_route(p: MobaParams, sel, workspace, stream=None) -> None:
    _check(load().moba_route(p.ref(), _ptr(sel), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream)))


def moba_attn_past(p: MobaParams, Q, K, V, workspace, stream=None) -> None:
    _check(load().moba_attn_past(p.ref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))


def moba_attn_self_merge(p: MobaParams, Q, K, V, sel, workspace, O, LSE, stream=None) -> None:
    _check(load().moba_attn_self_merge(p.ref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(sel), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(O), _ptr(LSE),
                                       _stream(stream)))


def moba_attn_naive(p: MobaParams, Q, K, V, sel, O, LSE, stream=None) -> None:
    """Mask-based attention over every causal key with the selection as a block mask
    (a baseline for moba_attn_fwd; same results up to rounding)."""
    _check(load().moba_attn_naive(p.ref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(sel), _ptr(O), _ptr(LSE),
                                  _stream(stream)))


def moba_bwd_workspace_size(p: MobaParams) -> int:
    return int(load().moba_bwd_workspace_size(p.ref()))


def moba_attn_bwd(p: MobaParams, Q, K, V, O, LSE, dO, sel, workspace, dQ, dK, dV, stream=None) -> None:
    """Gradients dQ [T,Hq,D], dK, dV [T,Hkv,D] (bf16) of MoBA attention for dO, with the
    forward's selection held fixed."""
    _check(load().moba_attn_bwd(p.ref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), _ptr(dO), _ptr(sel),
                                _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dQ),
                                _ptr(dK), _ptr(dV), _stream(stream)))


def moba_decode_workspace_size(p: MobaParams) -> int:
    return int(load().moba_decode_workspace_size(p.ref()))


def moba_decode_fwd(p: MobaParams, Q, K, V, Kbar, workspace, O, LSE, sel=None, stream=None) -> None:
    """Gated decode: Q [num_seqs, Hq, D] (the newest token of each cached sequence) against
    the caches K, V [T, Hkv, D] described by p; O [num_seqs, Hq, D], LSE [num_seqs, Hq]."""
    _check(load().moba_decode_fwd(p.ref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(Kbar), _ptr(sel), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _ptr(O), _ptr(LSE),
                                  _stream(stream)))


def moba_pool_last_block(p: MobaParams, K, Kbar, stream=None) -> None:
    """Re-pool each sequence's last block into Kbar (after appending to a KV cache)."""
    _check(load().moba_pool_last_block(p.ref(), _ptr(K), _ptr(Kbar), _stream(stream)))


def moba_gate_topk_noalloc(p: MobaParams, Q, Kbar, sel, stream=None) -> None:
    """moba_gate_topk for callers without an allocator: scratch is a fixed array in the library."""
    _check(load().moba_gate_topk_noalloc(p.ref(), _ptr(Q), _ptr(Kbar), _ptr(sel), _stream(stream)))


def moba_host_staging_size(p: MobaParams, nstreams: int) -> int:
    return int(load().moba_host_staging_size(p.ref(), nstreams))


def moba_fwd_host(p: MobaParams, Q, K, V, O, LSE, staging, streams) -> None:
    """Forward on pinned HOST tensors (Q, K, V in; O, LSE out), copies overlapped with the
    kernels over the given CUDA streams; asynchronous (synchronise the streams afterwards)."""
    arr = (ctypes.c_void_p * len(streams))(*[_stream(s) for s in streams])
    _check(load().moba_fwd_host(p.ref(), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), _ptr(staging),
                                staging.numel() * staging.element_size(), arr, len(streams)))


def moba_launches_per_forward(p: MobaParams) -> int:
    return int(load().moba_launches_per_forward(p.ref()))


def moba_read_device_error(clear: bool = False) -> int:
    """Device error word of the current device (non-zero: a kernel wait gave up)."""
    v = ctypes.c_int32(0)
    _check(load().moba_read_device_error(ctypes.byref(v), 1 if clear else 0))
    return int(v.value)


def moba_selftest_bounded_wait() -> int:
    """Run the bounded-wait failure path once; returns the device error word it produced."""
    v = ctypes.c_int32(0)
    _check(load().moba_selftest_bounded_wait(ctypes.byref(v)))
    return int(v.value)


class MobaCacheParams:
    """Geometry of a paged 8-bit KV cache (moba_cache_params) and the shapes of its buffers."""

    def __init__(self, max_seqs: int, max_seqlen: int, num_pages: int, page_size: int, num_q_heads: int,
                 num_kv_heads: int, head_dim: int, block_size: int, top_k: int, format: str = "e4m3",
                 softmax_scale: float = 0.0):
        if format not in CACHE_FORMATS:
            raise MobaError(2, "format must be one of %s (got %r)" % (", ".join(CACHE_FORMATS), format))
        sizes = (max_seqs, max_seqlen, num_pages, page_size, num_q_heads, num_kv_heads, head_dim, block_size, top_k)
        for (name, _), n in zip(_CCacheParams._fields_, sizes):
            if not -(1 << 31) <= n < 1 << 31:  # ctypes would take it modulo 2^32
                raise MobaError(2, "%s does not fit in 32 bits (got %d)" % (name, n))
        self.c = _CCacheParams(*sizes, CACHE_FORMATS[format], softmax_scale)
        self._ref = ctypes.byref(self.c)
        self.format = format
        # an append of no tokens checks the parameters and does nothing else
        _check(load().moba_cache_append(self._ref, None, 0, None, 0, 0, *[None] * 9, None))
        self.workspace_bytes = int(load().moba_cache_decode_workspace_size(self._ref))
        self.pages_per_seq = -(-max_seqlen // page_size)
        self.max_blocks = -(-max_seqlen // block_size)
        import torch
        i32, f32, bf16 = torch.int32, torch.float32, torch.bfloat16
        code = torch.float8_e4m3fn if format == "e4m3" else torch.int8
        pool = (num_pages, num_kv_heads)
        # dtype and shape of every buffer (None: any length)
        self.buffers = {
            "add": (i32, (max_seqs,)), "lens": (i32, (max_seqs,)), "lens_out": (i32, (max_seqs,)),
            "tables": (i32, (max_seqs, self.pages_per_seq)), "free_pages": (i32, (num_pages,)),
            "free_state": (i32, (2,)), "free_state_out": (i32, (2,)), "cu_new": (i32, (max_seqs + 1,)),
            "slots": (i32, (None,)), "status": (i32, (1,)),
            "K": (bf16, (None, num_kv_heads, head_dim)), "V": (bf16, (None, num_kv_heads, head_dim)),
            "Kc": (code, pool + (page_size, head_dim)), "Vc": (code, pool + (page_size, head_dim)),
            "Ks": (f32, pool), "Vs": (f32, pool),
            "Kbar": (f32, (max_seqs, self.max_blocks, num_kv_heads, head_dim)),
            "Q": (bf16, (max_seqs, num_q_heads, head_dim)), "O": (bf16, (max_seqs, num_q_heads, head_dim)),
            "LSE": (f32, (max_seqs, num_q_heads)), "sel": (i32, (max_seqs, num_q_heads, top_k)),
        }

        def specs(*names):
            return tuple((n,) + self.buffers[n] for n in names)

        self._tables = specs("add", "lens", "tables", "free_pages", "free_state", "lens_out", "free_state_out", "cu_new",
                             "status")
        self._append = specs("cu_new", "lens", "tables", "Kc", "Vc", "Ks", "Vs", "Kbar")
        self._decode = specs("Q", "Kc", "Vc", "Ks", "Vs", "Kbar", "lens", "tables", "O", "LSE")
        self._decode_sel = self._decode + specs("sel")
        self._cuda, self._raw_stream = torch.cuda, getattr(torch._C, "_cuda_getCurrentRawStream", None)

    def ref(self):
        return self._ref

    def check(self, device, **tensors):
        """Every tensor has its dtype and shape, lies on `device` and is contiguous (K and V: in
        their last two dimensions)."""
        for name, t in tensors.items():
            dtype, shape = self.buffers[name]
            if t.dtype != dtype:
                raise MobaError(1, "%s must be %s (got %s)" % (name, dtype, t.dtype))
            if len(t.shape) != len(shape) or any(w is not None and w != n for w, n in zip(shape, t.shape)):
                raise MobaError(1, "%s must have shape %s (got %s)" % (
                    name, tuple("n" if w is None else w for w in shape), tuple(t.shape)))
            if t.device != device:
                raise MobaError(1, "%s is on %s, the call's tensors are on %s" % (name, t.device, device))
            if name in ("K", "V"):
                if t.shape[0] and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2])):
                    raise MobaError(1, "%s must be contiguous in its last two dimensions" % name)
            elif not t.is_contiguous():
                raise MobaError(1, "%s must be contiguous" % name)

    def _pointers(self, index, specs, tensors):
        """Addresses of tensors that pass check(); the checks of a call are most of its time on the
        host, so this form of them makes no strings and no device objects."""
        out = []
        for (name, dtype, shape), t in zip(specs, tensors):
            if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
                self._check_one(name, t, index)
            out.append(t.data_ptr())
        return out

    def _check_one(self, name, t, index):
        import torch
        self.check(torch.device("cuda", index), **{name: t})

    def _slots(self, index, slots):
        if slots.dim() != 1 or slots.dtype is not self.buffers["slots"][0] or slots.get_device() != index or not slots.is_contiguous():
            self._check_one("slots", slots, index)
        if slots.shape[0] >= 1 << 31:
            raise MobaError(2, "slots must have less than 2^31 entries (got %d)" % slots.shape[0])
        return slots.data_ptr()


def _on(t):
    """The CUDA device index of a call's first tensor."""
    index = t.get_device()
    if index < 0:
        raise MobaError(1, "the tensors must be on a CUDA device (got %s)" % t.device)
    return index


def _call(p, index, stream, fn, *args):
    """fn(*args, stream) with device `index` current, on the given stream or its current one."""
    cuda = p._cuda
    if stream is None:
        # the address alone, where torch gives it without a Stream object
        stream = p._raw_stream(index) if p._raw_stream is not None else cuda.current_stream(index).cuda_stream
    else:
        stream = getattr(stream, "cuda_stream", stream)
    if cuda.current_device() == index:
        rc = fn(*args, stream)
    else:
        with cuda.device(index):
            rc = fn(*args, stream)
    if rc != 0:
        raise MobaError(rc, load().moba_last_error().decode())


def moba_cache_tables(p: MobaCacheParams, add, lens, tables, free_pages, free_state, lens_out, free_state_out,
                      cu_new, slots, status, stream=None) -> None:
    """Block tables, slot map and free-page ring for the next step: add[s] new tokens for request s
    (0: none, negative: it ends).  lens_out may be lens, free_state_out may be free_state."""
    index = _on(add)
    ptr = p._pointers(index, p._tables, (add, lens, tables, free_pages, free_state, lens_out, free_state_out, cu_new,
                                         status))
    _call(p, index, stream, load().moba_cache_tables, p._ref, *ptr[:8], p._slots(index, slots), slots.shape[0], ptr[8])


def moba_cache_append(p: MobaCacheParams, K, V, cu_new, lens, slots, tables, Kc, Vc, Ks, Vs, Kbar,
                      stream=None) -> None:
    """Writes the new tokens K, V [n, Hkv, D] (rows any multiple of 8 elements apart) into their
    slots and pools the keys of blocks that become complete; lens are those after the step."""
    index = _on(K)
    dtype, (_, heads, dims) = p.buffers["K"]
    size, (k_stride, *k_inner), (v_stride, *v_inner) = K.shape, K.stride(), V.stride()
    n, inner = size[0], [dims, 1]
    if K.dtype is not dtype or size != (n, heads, dims) or k_inner != inner:
        p._check_one("K", K, index)
    if V.dtype is not dtype or V.shape != size or v_inner != inner or V.get_device() != index:
        p._check_one("V", V, index)
    if n <= 1:
        k_stride = v_stride = heads * dims
    ptr = p._pointers(index, p._append, (cu_new, lens, tables, Kc, Vc, Ks, Vs, Kbar))
    slot_ptr = p._slots(index, slots)
    if V.shape[0] != n or slots.shape[0] != n:
        raise MobaError(1, "K, V and slots must have the same number of tokens (got %d, %d, %d)"
                        % (n, V.shape[0], slots.shape[0]))
    _call(p, index, stream, load().moba_cache_append, p._ref, K.data_ptr(), k_stride, V.data_ptr(), v_stride, n,
          ptr[0], ptr[1], slot_ptr, *ptr[2:])


def moba_cache_decode_workspace_size(p: MobaCacheParams) -> int:
    return p.workspace_bytes


def moba_cache_decode_fwd(p: MobaCacheParams, Q, Kc, Vc, Ks, Vs, Kbar, lens, tables, workspace, O, LSE, sel=None,
                          stream=None) -> None:
    """Gated decode: Q [max_seqs, Hq, D] (the newest token of each request) against the paged 8-bit
    cache; O [max_seqs, Hq, D], LSE [max_seqs, Hq], and sel [max_seqs, Hq, top_k] if given."""
    index = _on(Q)
    if sel is None:
        ptr = p._pointers(index, p._decode, (Q, Kc, Vc, Ks, Vs, Kbar, lens, tables, O, LSE)) + [None]
    else:
        ptr = p._pointers(index, p._decode_sel, (Q, Kc, Vc, Ks, Vs, Kbar, lens, tables, O, LSE, sel))
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise MobaError(1, "workspace must be contiguous and on %s" % Q.device)
    _call(p, index, stream, load().moba_cache_decode_fwd, p._ref, *ptr[:8], ptr[10], workspace.data_ptr(), workspace.nbytes,
          ptr[8], ptr[9])


def alloc_cache_workspace(p: MobaCacheParams, device="cuda"):
    import torch
    return torch.empty(p.workspace_bytes, dtype=torch.uint8, device=device)


class MobaCache:
    """The paged 8-bit KV cache of one layer: its pool, with the block tables, lengths and free
    pages of up to ``max_seqs`` requests.  A step is ``extend`` (how many tokens each request
    gets), ``append`` (their keys and values) and ``decode``.  The calls run on the current stream
    and enqueue kernels only, so a step can be captured into a CUDA graph.  (More layers share the
    tables and lengths: call the functions with each layer's pool.)"""

    def __init__(self, p: MobaCacheParams, device="cuda"):
        import torch
        self.p, self.device = p, torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())

        def zeros(name):
            dtype, shape = p.buffers[name]
            return torch.zeros(shape, dtype=dtype, device=self.device)

        self.Kc, self.Vc, self.Ks, self.Vs, self.Kbar = (zeros(n) for n in ("Kc", "Vc", "Ks", "Vs", "Kbar"))
        self.lens, self.tables, self.cu_new, self.status = (zeros(n) for n in ("lens", "tables", "cu_new", "status"))
        self.free_pages = torch.arange(p.c.num_pages, dtype=torch.int32, device=self.device)
        self.free_state = torch.tensor([0, p.c.num_pages], dtype=torch.int32, device=self.device)
        self.workspace = alloc_cache_workspace(p, self.device)

    def extend(self, add, max_tokens: int):
        """Tables and slots for add[s] new tokens a request (negative: it ends), at most
        ``max_tokens`` in all.  Returns the slot map; ``status`` tells whether it was done."""
        import torch
        slots = torch.empty(max_tokens, dtype=torch.int32, device=self.device)
        moba_cache_tables(self.p, add, self.lens, self.tables, self.free_pages, self.free_state, self.lens,
                          self.free_state, self.cu_new, slots, self.status)
        return slots

    def append(self, K, V, slots) -> None:
        """The new tokens' keys and values, packed in the order of the requests."""
        moba_cache_append(self.p, K, V, self.cu_new, self.lens, slots, self.tables, self.Kc, self.Vc, self.Ks,
                          self.Vs, self.Kbar)

    def decode(self, Q, sel=None):
        """(O, LSE) of the newest token of every request."""
        import torch
        O = torch.empty_like(Q)
        LSE = torch.empty(Q.shape[:2], dtype=torch.float32, device=self.device)
        moba_cache_decode_fwd(self.p, Q, self.Kc, self.Vc, self.Ks, self.Vs, self.Kbar, self.lens, self.tables,
                              self.workspace, O, LSE, sel=sel)
        return O, LSE


def alloc_workspace(p: MobaParams, device="cuda"):
    import torch
    return torch.empty(max(p.workspace_bytes, 256), dtype=torch.uint8, device=device)


def moba_attention(Q, K, V, cu_seqlens_host, block_size: int, top_k: int, softmax_scale: float = 0.0,
                   workspace=None, stream=None):
    """MoBA causal prefill on packed bf16 Q [T,Hq,D], K/V [T,Hkv,D]; returns (O, LSE)."""
    import torch
    T, hq, D = Q.shape
    p = MobaParams(cu_seqlens_host, hq, K.shape[1], D, block_size, top_k, softmax_scale=softmax_scale)
    if workspace is None:
        workspace = alloc_workspace(p, Q.device)
    O = torch.empty_like(Q)
    LSE = torch.empty((T, hq), dtype=torch.float32, device=Q.device)
    moba_fwd(p, Q, K, V, workspace, O, LSE, stream=stream)
    return O, LSE
