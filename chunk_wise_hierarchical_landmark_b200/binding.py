"""Thin Python binding of libhils.so (include/hils.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  Tensors are torch CUDA tensors (torch provides
device memory and the current stream); outputs are allocated here with torch
and passed to the library as device pointers.  There is no fallback: if
libhils.so is missing or fails to load, every call raises.
"""
from __future__ import annotations

import contextlib
import copyreg
import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhils.so")

HILS_OK = 0
HILS_F32, HILS_BF16 = 0, 1
HILS_OP_PREFILL, HILS_OP_DECODE, HILS_OP_DECODE_CACHE = 0, 1, 2
HILS_CACHE_PAGED, HILS_CACHE_Q8 = 0, 1


class HilsError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"hils status {status}: {msg}")
        self.status = status


class Params(ctypes.Structure):
    """Mirror of hils_params."""
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("L", ctypes.c_int), ("d", ctypes.c_int), ("chunk", ctypes.c_int),
                ("topk", ctypes.c_int), ("M", ctypes.c_int), ("scale", ctypes.c_float),
                ("dtype", ctypes.c_int), ("debug_checks", ctypes.c_int)]


class _CacheStruct(ctypes.Structure):
    """Mirror of hils_kv_cache."""
    _fields_ = [("format", ctypes.c_int), ("max_pages", ctypes.c_int), ("lmk_rows", ctypes.c_int),
                ("num_pages", ctypes.c_int64), ("k_pages", ctypes.c_void_p),
                ("v_pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("lmk", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_tail", ctypes.c_void_p),
                ("v_tail", ctypes.c_void_p)]


class _RowsStruct(ctypes.Structure):
    """Mirror of hils_rows."""
    _fields_ = [("data", ctypes.c_void_p), ("stride_b", ctypes.c_int64),
                ("stride_h", ctypes.c_int64), ("stride_t", ctypes.c_int64)]


_lib = None
EXPORTS = ["hils_workspace_size", "hils_select", "hils_union_capacity", "hils_union",
           "hils_attn_fwd", "hils_prefill", "hils_decode_fwd", "hils_decode_fwd_paged",
           "hils_decode_fwd_noalloc", "hils_hope", "hils_qcal_workspace_size", "hils_qcal_query",
           "hils_prefill_qcal", "hils_hope_rope_pairs", "hils_test_set_wait_limit",
           "hils_attn_bwd_workspace_size", "hils_attn_bwd", "hils_prefill_hope",
           "hils_kv_append", "hils_decode_fwd_cache",
           "hils_status_string", "hils_last_error", "hils_launch_count"]


def lib():
    """Load libhils.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m chunk_wise_hierarchical_landmark_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, PP, I, I64, SZ = ctypes.c_void_p, ctypes.POINTER(Params), ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        L.hils_workspace_size.argtypes = [PP, I]
        L.hils_workspace_size.restype = SZ
        L.hils_select.argtypes = [PP, P, P, P, P, P, P, SZ, P]
        L.hils_union_capacity.argtypes = [PP]
        L.hils_union_capacity.restype = I64
        L.hils_union.argtypes = [PP, P, P, P, I64, P, SZ, P]
        L.hils_attn_fwd.argtypes = [PP, P, P, P, P, P, P, P, P, P, SZ, P]
        L.hils_prefill.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.hils_decode_fwd.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.hils_decode_fwd_paged.argtypes = [PP, P, P, P, I64, P, I, P, P, P, P, P, P, P, SZ, P]
        L.hils_decode_fwd_noalloc.argtypes = [PP, P, P, P, P, P, P, P, P, P, P]
        L.hils_hope.argtypes = [P, I, I, I, I, I, I, I, ctypes.c_double, P]
        L.hils_prefill_hope.argtypes = [PP, P, P, P, P, I, I, ctypes.c_double, P, P, P, P, P, P,
                                        SZ, P]
        L.hils_prefill_hope.restype = I
        L.hils_attn_bwd_workspace_size.argtypes = [PP]
        L.hils_attn_bwd_workspace_size.restype = SZ
        L.hils_attn_bwd.argtypes = [PP, P, P, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.hils_attn_bwd.restype = I
        L.hils_test_set_wait_limit.argtypes = [ctypes.c_uint64, I]
        L.hils_test_set_wait_limit.restype = None
        L.hils_hope_rope_pairs.argtypes = [I, ctypes.c_double, ctypes.c_double]
        L.hils_hope_rope_pairs.restype = I
        L.hils_qcal_workspace_size.argtypes = [PP, I]
        L.hils_qcal_workspace_size.restype = SZ
        L.hils_qcal_query.argtypes = [PP, P, P, P, P, I, I, P, P, SZ, P]
        L.hils_prefill_qcal.argtypes = [PP, P, P, P, P, P, P, P, I, I, P, P, P, P, P, P, P, SZ, P]
        CP, RP = ctypes.POINTER(_CacheStruct), ctypes.POINTER(_RowsStruct)
        L.hils_kv_append.argtypes = [PP, CP, I, RP, RP, P, P, RP, P, I, ctypes.c_double, P, P, SZ, P]
        L.hils_kv_append.restype = I
        L.hils_decode_fwd_cache.argtypes = [PP, CP, P, P, P, P, P, P, P, P, SZ, P]
        L.hils_decode_fwd_cache.restype = I
        for f in ("hils_select", "hils_union", "hils_attn_fwd", "hils_prefill", "hils_decode_fwd",
                  "hils_decode_fwd_paged", "hils_decode_fwd_noalloc", "hils_hope",
                  "hils_qcal_query", "hils_prefill_qcal"):
            getattr(L, f).restype = I
        L.hils_status_string.argtypes = [I]
        L.hils_status_string.restype = ctypes.c_char_p
        L.hils_last_error.argtypes = []
        L.hils_last_error.restype = ctypes.c_char_p
        L.hils_launch_count.argtypes = []
        L.hils_launch_count.restype = I64
        _lib = L
    return _lib


def _check(status):
    if status != HILS_OK:
        L = lib()
        raise HilsError(status, f"{L.hils_status_string(status).decode()}: "
                                f"{L.hils_last_error().decode()}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def make_params(B, Hq, Hkv, L, d, topk, M=64, chunk=64, scale=None, dtype=torch.bfloat16,
                debug_checks=False) -> Params:
    return Params(B, Hq, Hkv, L, d, chunk, topk, M,
                  float(scale if scale is not None else 1.0 / d ** 0.5),
                  HILS_BF16 if dtype == torch.bfloat16 else HILS_F32, int(bool(debug_checks)))


def params_for(q, k, topk, M=64, chunk=64, scale=None, debug_checks=False, decode=False):
    """hils_params from tensors: prefill q [B,Hq,L,d] or decode q [B,Hq,d];
    k [B,Hkv,L,d]."""
    B, Hkv, L, d = k.shape
    Hq = q.shape[1]
    return make_params(B, Hq, Hkv, L, d, topk, M, chunk, scale, q.dtype, debug_checks)


def workspace(p: Params, op: int, device=None) -> torch.Tensor | None:
    n = lib().hils_workspace_size(ctypes.byref(p), op)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _ws_args(ws):
    return (_ptr(ws), 0 if ws is None else ws.numel())


def hils_select(p: Params, q, lmk_k, sel_idx, chunk_w, lse_lmk=None, ws=None, stream=None):
    _check(lib().hils_select(ctypes.byref(p), _ptr(q), _ptr(lmk_k), _ptr(sel_idx), _ptr(chunk_w),
                             _ptr(lse_lmk), *_ws_args(ws), _stream(stream)))


def hils_union_capacity(p: Params) -> int:
    return int(lib().hils_union_capacity(ctypes.byref(p)))


def hils_union(p: Params, sel_idx, u_off, u_idx, ws=None, stream=None):
    _check(lib().hils_union(ctypes.byref(p), _ptr(sel_idx), _ptr(u_off), _ptr(u_idx),
                            u_idx.numel(), *_ws_args(ws), _stream(stream)))


def hils_attn_fwd(p: Params, q, k, v, sel_idx, chunk_w, out, lse, w_final=None, ws=None,
                  stream=None):
    _check(lib().hils_attn_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(sel_idx),
                               _ptr(chunk_w), _ptr(out), _ptr(lse), _ptr(w_final),
                               *_ws_args(ws), _stream(stream)))


def hils_prefill(p: Params, q, k, v, lmk_k, sel_idx, chunk_w, lse_lmk, out, lse, ws=None,
                 stream=None):
    _check(lib().hils_prefill(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(lmk_k),
                              _ptr(sel_idx), _ptr(chunk_w), _ptr(lse_lmk), _ptr(out), _ptr(lse),
                              *_ws_args(ws), _stream(stream)))


def hils_decode_fwd(p: Params, q, k_cache, v_cache, lmk_k, sel_idx, chunk_w, lse_lmk, out, lse,
                    ws=None, stream=None):
    _check(lib().hils_decode_fwd(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                 _ptr(lmk_k), _ptr(sel_idx), _ptr(chunk_w), _ptr(lse_lmk),
                                 _ptr(out), _ptr(lse), *_ws_args(ws), _stream(stream)))


def hils_decode_fwd_paged(p: Params, q, k_pages, v_pages, page_table, lmk_k, sel_idx, chunk_w,
                          lse_lmk, out, lse, ws=None, stream=None):
    """k_pages / v_pages [num_pages, Hkv, C, d]; page_table [B, max_pages] int32."""
    _check(lib().hils_decode_fwd_paged(ctypes.byref(p), _ptr(q), _ptr(k_pages), _ptr(v_pages),
                                       int(k_pages.shape[0]), _ptr(page_table),
                                       int(page_table.shape[1]), _ptr(lmk_k), _ptr(sel_idx),
                                       _ptr(chunk_w), _ptr(lse_lmk), _ptr(out), _ptr(lse),
                                       *_ws_args(ws), _stream(stream)))


def hils_decode_fwd_noalloc(p: Params, q, k_cache, v_cache, lmk_k, sel_idx, chunk_w, lse_lmk,
                            out, lse, stream=None):
    _check(lib().hils_decode_fwd_noalloc(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                         _ptr(lmk_k), _ptr(sel_idx), _ptr(chunk_w), _ptr(lse_lmk),
                                         _ptr(out), _ptr(lse), _stream(stream)))


def hils_hope(x, n_rope_pairs: int, pos0: int = 0, base: float = 10000.0, stream=None):
    """HoPE in place on x [B,H,L,d] (or a decode query [B,H,d], one position)."""
    if x.dim() == 3:
        B, H, d = x.shape
        L = 1
    else:
        B, H, L, d = x.shape
    dt = HILS_BF16 if x.dtype == torch.bfloat16 else HILS_F32
    _check(lib().hils_hope(_ptr(x), dt, B, H, L, d, int(pos0), int(n_rope_pairs), float(base),
                           _stream(stream)))


def qcal_workspace(p: Params, r: int, device=None) -> torch.Tensor:
    n = lib().hils_qcal_workspace_size(ctypes.byref(p), int(r))
    if n == 0:
        raise HilsError(1, "hils_qcal_workspace_size rejected the parameters")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def hils_qcal_query(p: Params, q, h, w_down, w_up, q_cal, ws, stream=None):
    r, D = w_down.shape
    _check(lib().hils_qcal_query(ctypes.byref(p), _ptr(q), _ptr(h), _ptr(w_down), _ptr(w_up),
                                 int(D), int(r), _ptr(q_cal), *_ws_args(ws), _stream(stream)))


def hils_prefill_qcal(p: Params, q, k, v, lmk_k, h, w_down, w_up, q_cal, sel_idx, chunk_w,
                      lse_lmk, out, lse, ws, stream=None):
    r, D = w_down.shape
    _check(lib().hils_prefill_qcal(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(lmk_k),
                                   _ptr(h), _ptr(w_down), _ptr(w_up), int(D), int(r), _ptr(q_cal),
                                   _ptr(sel_idx), _ptr(chunk_w), _ptr(lse_lmk), _ptr(out),
                                   _ptr(lse), *_ws_args(ws), _stream(stream)))


def prefill_qcal(q, k, v, lmk_k, h, w_down, w_up, topk, M=64, scale=None, debug_checks=False):
    """Prefill with the Q-Cal scoring query (h [B,L,D], w_down [r,D], w_up
    [Hq,d,r]): returns dict(out, lse, sel_idx, chunk_w, lse_lmk, q_cal)."""
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    p = make_params(B, Hq, Hkv, L, d, topk, M, 64, scale, q.dtype, debug_checks)
    dev = q.device
    sel = torch.empty((B, Hq, L, topk), dtype=torch.int32, device=dev)
    w = torch.empty((B, Hq, L, topk), dtype=torch.float32, device=dev)
    lse_lmk = torch.empty((B, Hq, L), dtype=torch.float32, device=dev)
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, L), dtype=torch.float32, device=dev)
    q_cal = torch.empty_like(q)
    ws = qcal_workspace(p, w_down.shape[0], dev)
    hils_prefill_qcal(p, q, k, v, lmk_k, h, w_down, w_up, q_cal, sel, w, lse_lmk, out, lse, ws)
    return dict(out=out, lse=lse, sel_idx=sel, chunk_w=w, lse_lmk=lse_lmk, q_cal=q_cal)


def hils_attn_bwd(p: Params, q, k, v, lmk_k, sel_idx, chunk_w, lse, dout, dlse, dq, dk, dv,
                  dlmk, ws, stream=None):
    _check(lib().hils_attn_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(lmk_k),
                               _ptr(sel_idx), _ptr(chunk_w), _ptr(lse), _ptr(dout), _ptr(dlse),
                               _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dlmk), *_ws_args(ws),
                               _stream(stream)))


def attn_bwd(q, k, v, lmk_k, sel_idx, chunk_w, lse, dout, dlse=None, scale=None,
             debug_checks=False):
    """Backward pass for a forward's selection: returns fp32 (dq, dk, dv, dlmk)."""
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    topk = sel_idx.shape[-1]
    p = make_params(B, Hq, Hkv, L, d, topk, 64, 64, scale, q.dtype, debug_checks)
    dev = q.device
    dq = torch.empty(q.shape, dtype=torch.float32, device=dev)
    dk = torch.empty(k.shape, dtype=torch.float32, device=dev)
    dv = torch.empty(v.shape, dtype=torch.float32, device=dev)
    dl = torch.empty(lmk_k.shape, dtype=torch.float32, device=dev)
    n = lib().hils_attn_bwd_workspace_size(ctypes.byref(p))
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    hils_attn_bwd(p, q, k, v, lmk_k, sel_idx, chunk_w, lse, dout, dlse, dq, dk, dv, dl, ws)
    return dq, dk, dv, dl


def hils_prefill_hope(p: Params, q, k, v, lmk_k, pos0, n_rope_pairs, base, sel_idx, chunk_w,
                      lse_lmk, out, lse, ws=None, stream=None):
    _check(lib().hils_prefill_hope(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(lmk_k),
                                   int(pos0), int(n_rope_pairs), float(base), _ptr(sel_idx),
                                   _ptr(chunk_w), _ptr(lse_lmk), _ptr(out), _ptr(lse),
                                   *_ws_args(ws), _stream(stream)))


def prefill_hope(q, k, v, lmk_k, topk, n_rope_pairs, base, pos0=0, M=64, scale=None,
                 debug_checks=False):
    """Prefill with HoPE applied to the (unrotated) queries inside the kernels;
    k holds rotated keys.  Returns dict(out, lse, sel_idx, chunk_w, lse_lmk)."""
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    p = make_params(B, Hq, Hkv, L, d, topk, M, 64, scale, q.dtype, debug_checks)
    dev = q.device
    sel = torch.empty((B, Hq, L, topk), dtype=torch.int32, device=dev)
    w = torch.empty((B, Hq, L, topk), dtype=torch.float32, device=dev)
    lse_lmk = torch.empty((B, Hq, L), dtype=torch.float32, device=dev)
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, L), dtype=torch.float32, device=dev)
    hils_prefill_hope(p, q, k, v, lmk_k, pos0, n_rope_pairs, base, sel, w, lse_lmk, out, lse,
                      workspace(p, HILS_OP_PREFILL, dev))
    return dict(out=out, lse=lse, sel_idx=sel, chunk_w=w, lse_lmk=lse_lmk)


def rope_pairs_for(d: int, base: float, train_len: int) -> int:
    """The HoPE split of the library (hils_hope_rope_pairs): the pairs whose
    wavelength fits in the pre-training length get RoPE."""
    n = lib().hils_hope_rope_pairs(int(d), float(base), float(train_len))
    if n < 0:
        raise HilsError(1, "hils_hope_rope_pairs rejected its arguments")
    return n


# ---------------------------------------------------------------------------
# the cache of a serving loop (hils_kv_cache): append and decode

class _CacheFields:
    __slots__ = ("k_pages", "v_pages", "page_table", "lmk", "k_scale", "v_scale", "k_tail", "v_tail",
                 "B", "Hkv", "d", "q8", "dtype", "device", "max_len", "_dev", "_c")


class KVCache(_CacheFields):
    """A KV cache that grows token by token (hils_kv_cache), as torch tensors.

    k_pages, v_pages [num_pages,Hkv,64,d] in the keys' dtype, or, for the 8-bit
    form, torch.float8_e4m3fn codes with k_scale, v_scale [num_pages,Hkv] fp32
    and k_tail, v_tail [B,2,Hkv,64,d] in the keys' dtype; page_table
    [B,max_pages] int32; lmk [B,Hkv,rows,d] landmark keys (None: none kept).

    The tensors are checked against each other once, here (the C ABI sees
    pointers only); a handle keeps its tensors, whose contents the calls
    change, and its attributes are fixed.  replace() makes a handle with other
    tensors, copy.copy one with the same; a deep copy and a saved one (torch.save)
    hold tensors of their own.  A subclass may add fields."""
    __slots__ = ()

    def __new__(cls, k_pages, v_pages, page_table, lmk=None, k_scale=None, v_scale=None,
                k_tail=None, v_tail=None):
        shape, ty, dev = k_pages.shape, k_pages.dtype, k_pages.get_device()
        if len(shape) != 4 or shape[2] != 64:
            raise ValueError("k_pages must be [num_pages, Hkv, 64, d]")
        if page_table.dim() != 2:
            raise ValueError("page_table must be [B, max_pages] int32")
        npg, H, _, d = shape
        B, mp = page_table.shape
        if B * mp >= 1 << 31:
            raise ValueError("page_table must have fewer than 2^31 entries")
        q8 = ty is torch.float8_e4m3fn
        dt = k_tail.dtype if q8 and k_tail is not None else ty
        if dt is not torch.bfloat16 and dt is not torch.float32:
            raise ValueError(f"a cache holds bf16 or fp32 keys, got {dt}")

        def ptr(name, t, want, ty):
            if t is None or t.dtype is not ty or t.shape != want:
                raise ValueError(f"{name} must be {tuple(want)} {ty}")
            if t.get_device() != dev or not t.is_contiguous():
                raise ValueError("the cache's tensors must be contiguous and on one device")
            return t.data_ptr()
        rows = 0
        if lmk is not None:
            rows = lmk.shape[2] if lmk.dim() == 4 else -1
        ptrs = [ptr("k_pages", k_pages, shape, ty), ptr("v_pages", v_pages, shape, ty),
                ptr("page_table", page_table, (B, mp), torch.int32),
                None if lmk is None else ptr("lmk", lmk, (B, H, rows, d), dt)]
        if q8:
            tail = (B, 2, H, 64, d)
            ptrs += (ptr("k_scale", k_scale, (npg, H), torch.float32),
                     ptr("v_scale", v_scale, (npg, H), torch.float32),
                     ptr("k_tail", k_tail, tail, dt), ptr("v_tail", v_tail, tail, dt))
        self = object.__new__(_CacheFields)  # open while it is filled
        self.k_pages, self.v_pages, self.page_table, self.lmk = k_pages, v_pages, page_table, lmk
        self.k_scale, self.v_scale, self.k_tail, self.v_tail = k_scale, v_scale, k_tail, v_tail
        self.B, self.Hkv, self.d, self.q8, self.dtype, self.max_len = B, H, d, q8, dt, mp * 64
        self.device, self._dev = k_pages.device, dev
        self._c = _CacheStruct(HILS_CACHE_Q8 if q8 else HILS_CACHE_PAGED, mp, rows, npg, *ptrs)
        if cls is KVCache:
            self.__class__ = cls  # a step makes handles: 7 us this way, 10 us filling a sealed one
            return self
        handle = object.__new__(cls)  # a subclass may have fields of its own
        for name in _CacheFields.__slots__:
            object.__setattr__(handle, name, getattr(self, name))
        return handle

    def __setattr__(self, name, value):
        self._fixed(name)
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        self._fixed(name)
        object.__delattr__(self, name)

    def _fixed(self, name):  # _c holds the tensors' pointers
        if name in _CacheFields.__slots__:
            raise AttributeError(f"KVCache.{name} is fixed; replace() makes a handle with other tensors")

    def _tensors(self):
        return {n: getattr(self, n) for n in _CacheFields.__slots__[:8]}

    def __reduce__(self):
        return copyreg.__newobj__, (type(self), *self._tensors().values()), getattr(self, "__dict__", None)

    def replace(self, **tensors) -> "KVCache":
        cls = type(self)
        handle = cls.__new__(cls, **{**self._tensors(), **tensors})
        if cls is not KVCache and hasattr(self, "__dict__"):
            handle.__dict__.update(self.__dict__)
        return handle


def alloc_kv_cache(B, Hkv, d, max_len, num_pages=None, page_table=None, q8=True,
                   dtype=torch.bfloat16, device="cuda") -> KVCache:
    """An empty cache for B sequences of up to max_len tokens.  Without a
    page_table each sequence owns ceil(max_len/64) pages in order; with one
    ([B, at least that many]) num_pages gives the size of the pool."""
    mp = -(-max_len // 64)
    if (page_table is None) != (num_pages is None):
        raise ValueError("page_table and num_pages come together")
    if page_table is not None and (page_table.dim() != 2 or page_table.shape[0] != B or page_table.shape[1] < mp):
        raise ValueError(f"page_table must be [{B}, at least {mp}] for {max_len} tokens")
    if page_table is None:
        page_table = torch.arange(B * mp, dtype=torch.int32, device=device).view(B, mp)
        num_pages = B * mp
    shape = (num_pages, Hkv, 64, d)
    z = dict(device=device)
    ty = torch.float8_e4m3fn if q8 else dtype
    pages = [torch.zeros(shape, dtype=ty, **z) for _ in range(2)]
    lmk = torch.zeros((B, Hkv, page_table.shape[1], d), dtype=dtype, **z)
    more = [torch.zeros(shape[:2], **z) for _ in range(2)]
    more += [torch.zeros((B, 2, Hkv, 64, d), dtype=dtype, **z) for _ in range(2)]
    return KVCache(*pages, page_table, lmk, *(more if q8 else ()))


def _c_int(x):
    """x as the library sees it: past 32 bits still out of its bounds (ctypes would
    pass the low bits)."""
    return min(max(x, -1), (1 << 31) - 1)


# A serving loop calls with the same sizes again and again: the parameter block
# of a call (read only) and its workspace bytes are kept by its arguments.
@functools.lru_cache(maxsize=1024)
def _params(B, Hq, Hkv, L, d, topk, *rest):
    return make_params(B, Hq, Hkv, _c_int(L), d, _c_int(topk), *rest)


@functools.lru_cache(maxsize=1024)
def _decode_cache_params(*args):
    p = _params(*args)
    return p, lib().hils_workspace_size(p, HILS_OP_DECODE_CACHE)


def _on(cache):
    """Calls go to the tensors' device, whichever is current."""
    if cache._dev < 0:
        raise ValueError(f"the cache must be on a CUDA device, not {cache.device}")
    if cache._dev == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(cache._dev)


def _current_stream(cache):
    return torch._C._cuda_getCurrentRawStream(cache._dev)


def _rows(x, shape, cache, name):
    if x.shape != shape or x.dtype is not cache.dtype or x.get_device() != cache._dev:
        raise ValueError(f"{name} must be {shape} {cache.dtype} on {cache.device}")
    sb, sh, st, sd = x.stride()
    if sd != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    # the stride of a dimension of one is never used
    return _RowsStruct(x.data_ptr(), sb if shape[0] > 1 else 0, sh if shape[1] > 1 else 0,
                       st if shape[2] > 1 else 0)


def _lens(x, cache, name):
    if x.dtype is not torch.int32 or x.shape != (cache.B,) or not x.is_contiguous() or x.get_device() != cache._dev:
        raise ValueError(f"{name} must be a contiguous [{cache.B}] int32 tensor on {cache.device}")
    return x.data_ptr()


def kv_append(cache: KVCache, k, v, pos, n_new=None, q=None, n_rope_pairs=0, base=10000.0,
              max_len=None, seq_lens=None, q_out=None, debug_checks=False):
    """Append new tokens (hils_kv_append): k, v [B,Hkv,T,d] and optionally q
    [B,Hq,T,d], any strides with d contiguous, at positions pos [B] int32
    (n_new [B] int32: tokens of each sequence, default T).  Keys and queries
    are rotated by HoPE, the values stored as they are; landmark rows of
    completed chunks are their mean key.  max_len: the longest length any
    sequence may reach (default: what the page table holds).  Returns dict(q =
    the rotated queries [B,Hq,T,d] or None, seq_lens = pos + n_new)."""
    B, H, d = cache.B, cache.Hkv, cache.d
    if k.dim() != 4:
        raise ValueError("k must be [B, Hkv, T, d]")
    T, Hq, rq = k.shape[2], H, None
    rk, rv = _rows(k, (B, H, T, d), cache, "k"), _rows(v, (B, H, T, d), cache, "v")
    if q is not None:
        if q.dim() != 4:
            raise ValueError("q must be [B, Hq, T, d]")
        Hq = q.shape[1]
        rq = _rows(q, (B, Hq, T, d), cache, "q")
        if q_out is not None and (not q_out.is_contiguous() or _rows(q_out, (B, Hq, T, d), cache, "q_out") is None):
            raise ValueError("q_out must be contiguous")
    pos_p = _lens(pos, cache, "pos")
    n_p = None if n_new is None else _lens(n_new, cache, "n_new")
    lens_p = None if seq_lens is None else _lens(seq_lens, cache, "seq_lens")
    p = _params(B, Hq, H, cache.max_len if max_len is None else int(max_len), d, 1, 64, 64, 1.0,
                cache.dtype, bool(debug_checks))
    with _on(cache):
        if rq is not None and q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        if lens_p is None:
            seq_lens = torch.empty_like(pos)
            lens_p = seq_lens.data_ptr()
        ws = torch.empty(256, dtype=torch.uint8, device=cache.device) if debug_checks else None
        _check(lib().hils_kv_append(p, cache._c, T, rk, rv, pos_p, n_p, rq,
                                    None if q_out is None else q_out.data_ptr(),
                                    n_rope_pairs if -1 < n_rope_pairs < 1 << 31 else -1, base,
                                    lens_p, *_ws_args(ws), _current_stream(cache)))
    return dict(q=q_out, seq_lens=seq_lens)


def hils_decode_fwd_cache(p: Params, cache: KVCache, q, seq_lens, sel_idx, chunk_w, lse_lmk, out,
                          lse, ws, stream=None):
    _check(lib().hils_decode_fwd_cache(
        p, cache._c, q.data_ptr(), seq_lens.data_ptr(), sel_idx.data_ptr(), chunk_w.data_ptr(),
        None if lse_lmk is None else lse_lmk.data_ptr(), out.data_ptr(), lse.data_ptr(),
        *_ws_args(ws), _current_stream(cache) if stream is None else stream.cuda_stream))


def decode_cache(q, cache: KVCache, seq_lens, topk, max_len=None, scale=None,
                 debug_checks=False):
    """One decode step (q [B,Hq,d], rotated) over a KVCache with a length per
    sequence (seq_lens [B] int32, 0: an empty row of the batch), each at most
    max_len (default: what the page table holds): returns dict(out, lse,
    sel_idx, chunk_w, lse_lmk)."""
    B, d, dt, dev = cache.B, cache.d, cache.dtype, cache.device
    if q.dim() != 3 or q.shape[0] != B or q.shape[2] != d or q.dtype is not dt \
            or q.get_device() != cache._dev or not q.is_contiguous():
        raise ValueError(f"q must be a contiguous [{B}, Hq, {d}] {dt} tensor on {dev}")
    _lens(seq_lens, cache, "seq_lens")
    Hq = q.shape[1]
    topk = int(topk)
    p, ws_bytes = _decode_cache_params(B, Hq, cache.Hkv, cache.max_len if max_len is None else int(max_len),
                                       d, topk, 64, 64, None if scale is None else float(scale), dt,
                                       bool(debug_checks))
    with _on(cache):
        # allocations are half of a small step's host time; with strides they take less
        K = topk if ws_bytes else 1  # sizes without a workspace are refused by the call
        w = torch.empty_strided((B, Hq, K), (Hq * K, K, 1), dtype=torch.float32, device=dev)
        sel = torch.empty_like(w, dtype=torch.int32)
        lse = torch.empty_strided((B, Hq), (Hq, 1), dtype=torch.float32, device=dev)
        lse_lmk, out = torch.empty_like(lse), torch.empty_like(q)
        ws = torch.empty_strided((ws_bytes,), (1,), dtype=torch.uint8, device=dev) if ws_bytes else None
        hils_decode_fwd_cache(p, cache, q, seq_lens, sel, w, lse_lmk, out, lse, ws)
    return dict(out=out, lse=lse, sel_idx=sel, chunk_w=w, lse_lmk=lse_lmk)


def launch_count() -> int:
    return int(lib().hils_launch_count())


# ---------------------------------------------------------------------------
# allocation helpers (outputs allocated with torch, then one C-ABI call)

def select(q, lmk_k, topk, M=64, scale=None, with_lse_lmk=True, debug_checks=False, k_shape=None):
    """Landmark scoring + top-k for a prefill: returns (sel_idx, chunk_w, lse_lmk)."""
    B, Hq, L, d = q.shape
    Hkv = lmk_k.shape[1]
    p = make_params(B, Hq, Hkv, L, d, topk, M, 64, scale, q.dtype, debug_checks)
    sel = torch.empty((B, Hq, L, topk), dtype=torch.int32, device=q.device)
    w = torch.empty((B, Hq, L, topk), dtype=torch.float32, device=q.device)
    lse_lmk = torch.empty((B, Hq, L), dtype=torch.float32, device=q.device) if with_lse_lmk else None
    hils_select(p, q, lmk_k, sel, w, lse_lmk, workspace(p, HILS_OP_PREFILL, q.device))
    return sel, w, lse_lmk


def attn_fwd(q, k, v, sel_idx, chunk_w, M=64, scale=None, with_w_final=False, debug_checks=False):
    """Intra-chunk attention + fusion: returns (out, lse, w_final or None)."""
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    topk = sel_idx.shape[-1]
    p = make_params(B, Hq, Hkv, L, d, topk, M, 64, scale, q.dtype, debug_checks)
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, L), dtype=torch.float32, device=q.device)
    wf = torch.empty((B, Hq, L, topk + 1), dtype=torch.float32, device=q.device) if with_w_final else None
    hils_attn_fwd(p, q, k, v, sel_idx, chunk_w, out, lse, wf, workspace(p, HILS_OP_PREFILL, q.device))
    return out, lse, wf


def prefill(q, k, v, lmk_k, topk, M=64, scale=None, debug_checks=False):
    """Full prefill forward: returns dict(out, lse, sel_idx, chunk_w, lse_lmk)."""
    B, Hq, L, d = q.shape
    Hkv = k.shape[1]
    p = make_params(B, Hq, Hkv, L, d, topk, M, 64, scale, q.dtype, debug_checks)
    dev = q.device
    sel = torch.empty((B, Hq, L, topk), dtype=torch.int32, device=dev)
    w = torch.empty((B, Hq, L, topk), dtype=torch.float32, device=dev)
    lse_lmk = torch.empty((B, Hq, L), dtype=torch.float32, device=dev)
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq, L), dtype=torch.float32, device=dev)
    hils_prefill(p, q, k, v, lmk_k, sel, w, lse_lmk, out, lse, workspace(p, HILS_OP_PREFILL, dev))
    return dict(out=out, lse=lse, sel_idx=sel, chunk_w=w, lse_lmk=lse_lmk)


def decode(q, k_cache, v_cache, lmk_k, topk, scale=None, debug_checks=False):
    """One decode step (q [B,Hq,d], cache [B,Hkv,N,d]): returns dict(out, lse, sel_idx, chunk_w, lse_lmk)."""
    B, Hq, d = q.shape
    _, Hkv, N, _ = k_cache.shape
    p = make_params(B, Hq, Hkv, N, d, topk, 64, 64, scale, q.dtype, debug_checks)
    dev = q.device
    sel = torch.empty((B, Hq, topk), dtype=torch.int32, device=dev)
    w = torch.empty((B, Hq, topk), dtype=torch.float32, device=dev)
    lse_lmk = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    hils_decode_fwd(p, q, k_cache, v_cache, lmk_k, sel, w, lse_lmk, out, lse,
                    workspace(p, HILS_OP_DECODE, dev))
    return dict(out=out, lse=lse, sel_idx=sel, chunk_w=w, lse_lmk=lse_lmk)


def decode_paged(q, k_pages, v_pages, page_table, lmk_k, N, topk, scale=None,
                 debug_checks=False):
    """One decode step over a paged cache (q [B,Hq,d]; pages [num_pages,Hkv,64,d];
    page_table [B, max_pages] int32; N tokens per sequence): returns
    dict(out, lse, sel_idx, chunk_w, lse_lmk)."""
    B, Hq, d = q.shape
    Hkv = k_pages.shape[1]
    p = make_params(B, Hq, Hkv, N, d, topk, 64, 64, scale, q.dtype, debug_checks)
    dev = q.device
    sel = torch.empty((B, Hq, topk), dtype=torch.int32, device=dev)
    w = torch.empty((B, Hq, topk), dtype=torch.float32, device=dev)
    lse_lmk = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    out = torch.empty_like(q)
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    hils_decode_fwd_paged(p, q, k_pages, v_pages, page_table, lmk_k, sel, w, lse_lmk, out, lse,
                          workspace(p, HILS_OP_DECODE, dev))
    return dict(out=out, lse=lse, sel_idx=sel, chunk_w=w, lse_lmk=lse_lmk)


def union(sel_idx, M=64, debug_checks=False):
    """Chunk union per group of M rows in CSR form: returns (u_off, u_idx)."""
    B, Hq, L, topk = sel_idx.shape
    p = make_params(B, Hq, Hq, L, 64, topk, M, 64, None, torch.bfloat16, debug_checks)
    cap = hils_union_capacity(p)
    G = B * Hq * ((L + M - 1) // M)
    u_off = torch.empty(G + 1, dtype=torch.int32, device=sel_idx.device)
    u_idx = torch.empty(max(cap, 4), dtype=torch.int32, device=sel_idx.device)
    hils_union(p, sel_idx, u_off, u_idx, workspace(p, HILS_OP_PREFILL, sel_idx.device))
    return u_off, u_idx[:int(u_off[-1].item())]
