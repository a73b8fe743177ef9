"""Activation-sparse FFN decoding on NVIDIA B200 — Python binding.

A thin ``ctypes`` layer over ``libspffn.so`` (C-ABI in ``include/spffn.h``):
it only marshals arguments.  Every step of the path — predictor, threshold,
compaction, FC1, FC2, reduction, chaining, profiling, row permutation — runs in
the library's CUDA kernels.  PyTorch is used only to own device memory and
streams.  There is no CPU fallback: if the library is missing and cannot be
built, importing the binding's functions raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

from . import build as _build

__all__ = ["SpffnError", "Layer", "AttnLayer", "attn_step_kernel_launches", "decode", "decode_tables", "decode_kernel_launches", "forward_noalloc",
           "reorder", "reorder_dealt", "permute_rows", "permute_vector", "set_trace", "trace_marks",
           "set_l2_hot_rows", "l2_hot_rows", "set_union_stack", "union_stack",
           "norm_quant", "quantize_rows", "Linear8", "Rope", "KvCache4", "rope_frequencies",
           "workspace_bytes", "library", "F16", "BF16"]

F16, BF16 = 0, 1
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE_CHECK, ERR_TIMEOUT = range(7)

EXPORTS = ("spffn_workspace_bytes", "spffn_create", "spffn_destroy", "spffn_predict", "spffn_forward",
           "spffn_step", "spffn_chain", "spffn_decode", "spffn_profile_counts", "spffn_reorder",
           "spffn_permute_rows", "spffn_permute_vector", "spffn_last_device_error", "spffn_status_string",
           "spffn_num_partials", "spffn_decode_kernel_launches", "spffn_set_trace", "spffn_trace_marks",
           "spffn_last_cuda_error_string", "spffn_reorder_dealt", "spffn_forward_noalloc",
           "spffn_decode_lookahead", "spffn_layer_table", "spffn_decode_tables", "spffn_set_wait_test", "spffn_set_l2_hot_rows", "spffn_l2_hot_rows",
           "spffn_set_union_stack", "spffn_union_stack",
           "spffn_attn_workspace_bytes", "spffn_attn_create", "spffn_attn_destroy", "spffn_attn_reset",
           "spffn_attn_step", "spffn_attn_cache", "spffn_attn_step_kernel_launches", "spffn_attn_last_device_error",
           "spffn_norm_quant", "spffn_quantize_rows", "spffn_mm8_workspace_bytes", "spffn_mm8_create",
           "spffn_mm8_destroy", "spffn_mm8_forward", "spffn_mm8_last_device_error", "spffn_rope_frequencies",
           "spffn_kv4_pool_bytes", "spffn_kv4_workspace_bytes", "spffn_kv4_create", "spffn_kv4_destroy",
           "spffn_kv4_append", "spffn_kv4_attend", "spffn_kv4_read", "spffn_kv4_last_device_error")


class SpffnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (what, _status_string(status), status))


class Config(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("n", ctypes.c_int32), ("H", ctypes.c_int32),
                ("max_batch", ctypes.c_int32), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class Weights(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("W1", "b1", "W2T", "b2", "Wp1", "bp1", "Wp2", "bp2")]


class AttnConfig(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("nh", ctypes.c_int32), ("dh", ctypes.c_int32), ("Ha", ctypes.c_int32),
                ("tmax", ctypes.c_int32), ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class AttnWeights(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("Wq", "bq", "Wk", "bk", "Wv", "bv", "WoT", "bo", "Wa1", "ba1",
                                                "Wa2", "ba2")]


class AttnCacheView(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("filled", ctypes.c_void_p), ("Y", ctypes.c_void_p),
                ("t", ctypes.c_void_p)]


class Mm8Config(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("N", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class Mm8Weights(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("W", "w_scale", "bias")]


class Kv4Config(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in ("pages", "page_size", "nh", "kvh", "dh", "max_seqs", "max_tokens", "dtype",
                                               "rope_dim", "rope_interleaved")] + [
        ("flags", ctypes.c_uint32), ("rope_amplitude", ctypes.c_double)]


_lib = None


def library(path: Optional[str] = None):
    """Load (building in-tree first if it is missing or stale) libspffn.so."""
    global _lib
    if _lib is not None:
        return _lib
    so = path or _build.SO
    if path is None and _build.stale():
        try:
            _build.build()
        except Exception as e:  # no nvcc here: the library must already exist
            if not os.path.exists(so):
                raise RuntimeError("libspffn.so is missing and could not be built: %s" % e) from e
    lib = ctypes.CDLL(so)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    i64, f32, f64 = ctypes.c_int64, ctypes.c_float, ctypes.c_double
    st = ctypes.c_int
    sig = {
        "spffn_workspace_bytes": (sz, [ctypes.POINTER(Config)]),
        "spffn_create": (st, [ctypes.POINTER(Config), ctypes.POINTER(Weights), vp, sz, ctypes.POINTER(vp)]),
        "spffn_destroy": (st, [vp]),
        "spffn_predict": (st, [vp, vp, i32, vp, vp, vp]),
        "spffn_forward": (st, [vp, vp, i32, vp, vp, vp, vp]),
        "spffn_step": (st, [vp, vp, i32, vp, vp, vp, vp]),
        "spffn_chain": (st, [vp, vp, vp, i32, vp, vp]),
        "spffn_decode": (st, [ctypes.POINTER(vp), i32, vp, i32, vp, vp, vp, vp]),
        "spffn_decode_lookahead": (st, [ctypes.POINTER(vp), i32, vp, i32, vp, vp, vp, vp]),
        "spffn_layer_table": (st, [vp, ctypes.POINTER(vp)]),
        "spffn_decode_tables": (st, [ctypes.POINTER(vp), i32, vp, i32, ctypes.POINTER(vp), vp, vp, vp, vp, vp]),
        "spffn_profile_counts": (st, [vp, vp, i32, vp, vp]),
        "spffn_reorder": (st, [vp, i32, vp]),
        "spffn_reorder_dealt": (st, [vp, i32, i32, vp]),
        "spffn_forward_noalloc": (st, [ctypes.POINTER(Config), ctypes.POINTER(Weights), vp, i32, vp, vp, vp, vp]),
        "spffn_permute_rows": (st, [vp, vp, i32, i32, vp, vp]),
        "spffn_permute_vector": (st, [vp, vp, i32, vp, vp]),
        "spffn_last_device_error": (st, [vp, ctypes.POINTER(ctypes.c_uint32), vp]),
        "spffn_status_string": (ctypes.c_char_p, [st]),
        "spffn_num_partials": (i32, [vp]),
        "spffn_decode_kernel_launches": (i32, [ctypes.POINTER(vp), i32, i32]),
        "spffn_set_trace": (st, [vp, sz]),
        "spffn_set_wait_test": (st, [ctypes.c_uint64, i32]),
        "spffn_set_l2_hot_rows": (st, [i32]),
        "spffn_set_union_stack": (st, [i32]),
        "spffn_union_stack": (i32, []),
        "spffn_l2_hot_rows": (i32, []),
        "spffn_trace_marks": (i32, []),
        "spffn_last_cuda_error_string": (ctypes.c_char_p, []),
        "spffn_attn_workspace_bytes": (sz, [ctypes.POINTER(AttnConfig)]),
        "spffn_attn_create": (st, [ctypes.POINTER(AttnConfig), ctypes.POINTER(AttnWeights), vp, sz, ctypes.POINTER(vp)]),
        "spffn_attn_destroy": (st, [vp]),
        "spffn_attn_reset": (st, [vp, vp]),
        "spffn_attn_step": (st, [vp, vp, vp, vp, vp, vp]),
        "spffn_attn_cache": (st, [vp, ctypes.POINTER(AttnCacheView)]),
        "spffn_attn_step_kernel_launches": (i32, []),
        "spffn_attn_last_device_error": (st, [vp, ctypes.POINTER(ctypes.c_uint32), vp]),
        "spffn_norm_quant": (st, [i32, i32, i32, vp, i64, vp, i64, i32, vp, f32, vp, i64, vp, i64, vp, vp]),
        "spffn_quantize_rows": (st, [i32, i32, i32, vp, i64, i32, vp, i64, vp, vp]),
        "spffn_mm8_workspace_bytes": (sz, [ctypes.POINTER(Mm8Config)]),
        "spffn_mm8_create": (st, [ctypes.POINTER(Mm8Config), ctypes.POINTER(Mm8Weights), vp, sz, ctypes.POINTER(vp)]),
        "spffn_mm8_destroy": (st, [vp]),
        "spffn_mm8_forward": (st, [vp, vp, i64, vp, i32, vp, i64, vp]),
        "spffn_mm8_last_device_error": (st, [vp, ctypes.POINTER(ctypes.c_uint32), vp]),
        "spffn_rope_frequencies": (st, [i32, f64, i32, f64, f64, ctypes.POINTER(f64), ctypes.POINTER(f64)]),
        "spffn_kv4_pool_bytes": (sz, [ctypes.POINTER(Kv4Config)]),
        "spffn_kv4_workspace_bytes": (sz, [ctypes.POINTER(Kv4Config)]),
        "spffn_kv4_create": (st, [ctypes.POINTER(Kv4Config), vp, sz, vp, vp, sz, ctypes.POINTER(vp)]),
        "spffn_kv4_destroy": (st, [vp]),
        "spffn_kv4_append": (st, [vp, vp, i64, vp, i64, vp, i64, i32, vp, i64, i32, vp, vp, i32, vp, i64, vp]),
        "spffn_kv4_attend": (st, [vp, vp, i64, i32, vp, i64, i32, vp, vp, i32, f32, vp, i64, vp]),
        "spffn_kv4_read": (st, [vp, vp, i32, vp, vp, vp]),
        "spffn_kv4_last_device_error": (st, [vp, ctypes.POINTER(ctypes.c_uint32), vp]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _status_string(s: int) -> str:
    try:
        return library().spffn_status_string(s).decode()
    except Exception:
        return "status"


def _check(status: int, what: str):
    if status != OK:
        if status == ERR_CUDA:
            what = "%s [%s]" % (what, library().spffn_last_cuda_error_string().decode())
        raise SpffnError(status, what)


def _p(t) -> Optional[int]:
    """Device pointer of a CUDA tensor (None stays NULL)."""
    if t is None:
        return None
    if not getattr(t, "is_cuda", False):
        raise TypeError("expected a CUDA tensor, got %r" % (type(t),))
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float16:
        return F16
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("storage dtype must be float16 or bfloat16, got %s" % t.dtype)


def workspace_bytes(d: int, n: int, H: int, max_batch: int, dtype: int = F16) -> int:
    cfg = Config(d, n, H, max_batch, dtype, 0)
    return int(library().spffn_workspace_bytes(ctypes.byref(cfg)))


class Layer:
    """One FFN layer bound to the library (wraps an ``spffn_ctx``).

    Weight tensors (CUDA, row-major, float16 or bfloat16): ``W1[n,d]``, ``b1[n]``,
    ``W2T[n,d]`` (neuron-major FC2), ``b2[d]`` or None, ``Wp1[H,d]``, ``bp1[H]``
    or None, ``Wp2[n,H]``, ``bp2[n]`` or None.  The workspace is a zero-filled
    uint8 CUDA tensor (allocated here when not given).
    """

    def __init__(self, W1, b1, W2T, b2, Wp1, bp1, Wp2, bp2, max_batch: int = 1, workspace=None):
        import torch
        n, d = W1.shape
        H = Wp1.shape[0]
        self.d, self.n, self.H, self.max_batch = int(d), int(n), int(H), int(max_batch)
        self.dtype = _dtype_code(W1)
        self.cfg = Config(self.d, self.n, self.H, self.max_batch, self.dtype, 0)
        self._keep = [W1, b1, W2T, b2, Wp1, bp1, Wp2, bp2]
        self.weights = Weights(_p(W1), _p(b1), _p(W2T), _p(b2), _p(Wp1), _p(bp1), _p(Wp2), _p(bp2))
        need = int(library().spffn_workspace_bytes(ctypes.byref(self.cfg)))
        if need == 0:
            raise SpffnError(ERR_INVALID_ARG, "spffn_workspace_bytes (bad shape)")
        if workspace is None:
            workspace = torch.zeros(need, dtype=torch.uint8, device=W1.device)
        self.workspace = workspace
        ctx = ctypes.c_void_p()
        _check(library().spffn_create(ctypes.byref(self.cfg), ctypes.byref(self.weights),
                                      _p(workspace), workspace.numel(), ctypes.byref(ctx)), "spffn_create")
        self.ctx = ctx

    @classmethod
    def from_device_layer(cls, L, max_batch: int = 1, workspace=None):
        return cls(L.W1, L.b1, L.W2T, L.b2, L.Wp1, L.bp1, L.Wp2, L.bp2, max_batch, workspace)

    def close(self):
        if getattr(self, "ctx", None):
            library().spffn_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def num_partials(self) -> int:
        return int(library().spffn_num_partials(self.ctx))

    def predict(self, x, idx, count, stream=None):
        _check(library().spffn_predict(self.ctx, _p(x), x.shape[0], _p(idx), _p(count), _stream(stream)),
               "spffn_predict")

    def forward(self, x, idx, count, y, stream=None):
        _check(library().spffn_forward(self.ctx, _p(x), x.shape[0], _p(idx), _p(count), _p(y),
                                       _stream(stream)), "spffn_forward")

    def step(self, x, idx, count, y, stream=None):
        _check(library().spffn_step(self.ctx, _p(x), x.shape[0], _p(idx), _p(count), _p(y), _stream(stream)),
               "spffn_step")

    def chain(self, x, y, x_next, stream=None):
        _check(library().spffn_chain(self.ctx, _p(x), _p(y), x.shape[0], _p(x_next), _stream(stream)),
               "spffn_chain")

    def profile_counts(self, X, counts, stream=None):
        _check(library().spffn_profile_counts(self.ctx, _p(X), X.shape[0], _p(counts), _stream(stream)),
               "spffn_profile_counts")

    def table(self, count: int):
        """The neuron table the last decode left in this layer's workspace: an
        int32 view of its first ``count`` entries (spffn_layer_table)."""
        import torch
        ptr = ctypes.c_void_p()
        _check(library().spffn_layer_table(self.ctx, ctypes.byref(ptr)), "spffn_layer_table")
        off = int(ptr.value) - self.workspace.data_ptr()
        return self.workspace[off:off + 4 * int(count)].view(torch.int32)

    def last_device_error(self, stream=None):
        code = ctypes.c_uint32(0)
        s = library().spffn_last_device_error(self.ctx, ctypes.byref(code), _stream(stream))
        return s, int(code.value)


class AttnLayer:
    """One attention layer with its head predictor (wraps an ``spffn_attn_ctx``).

    Weight tensors (CUDA, row-major, float16 or bfloat16): ``Wq, Wk, Wv[nh*dh, d]``,
    ``WoT[nh*dh, d]`` (output projection stored head-major), ``Wa1[Ha, d]``,
    ``Wa2[nh, Ha]``; biases ``bq, bk, bv[nh*dh]``, ``bo[d]``, ``ba1[Ha]``,
    ``ba2[nh]`` or None.  The workspace (cache included) is a zero-filled uint8
    CUDA tensor, allocated here when not given.
    """

    def __init__(self, Wq, Wk, Wv, WoT, Wa1, Wa2, nh: int, tmax: int, bq=None, bk=None, bv=None, bo=None,
                 ba1=None, ba2=None, workspace=None):
        import torch
        rows, d = Wq.shape
        self.d, self.nh, self.dh, self.Ha, self.tmax = int(d), int(nh), int(rows) // int(nh), int(Wa1.shape[0]), int(tmax)
        self.dtype = _dtype_code(Wq)
        self.cfg = AttnConfig(self.d, self.nh, self.dh, self.Ha, self.tmax, self.dtype, 0)
        self._keep = [Wq, bq, Wk, bk, Wv, bv, WoT, bo, Wa1, ba1, Wa2, ba2]
        self.weights = AttnWeights(*[_p(t) for t in self._keep])
        need = int(library().spffn_attn_workspace_bytes(ctypes.byref(self.cfg)))
        if need == 0:
            raise SpffnError(ERR_INVALID_ARG, "spffn_attn_workspace_bytes (bad shape)")
        if workspace is None:
            workspace = torch.zeros(need, dtype=torch.uint8, device=Wq.device)
        self.workspace = workspace
        ctx = ctypes.c_void_p()
        _check(library().spffn_attn_create(ctypes.byref(self.cfg), ctypes.byref(self.weights), _p(workspace),
                                           workspace.numel(), ctypes.byref(ctx)), "spffn_attn_create")
        self.ctx = ctx

    def close(self):
        if getattr(self, "ctx", None):
            library().spffn_attn_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def step(self, y, heads, count, out, stream=None):
        """One decode step: y [d] -> out [d] (fp32); heads [nh], count [1] (int32)."""
        _check(library().spffn_attn_step(self.ctx, _p(y), _p(heads), _p(count), _p(out), _stream(stream)),
               "spffn_attn_step")

    def reset(self, stream=None):
        _check(library().spffn_attn_reset(self.ctx, _stream(stream)), "spffn_attn_reset")

    def cache(self):
        """(K, V, filled, Y, t) views of the cache as torch tensors on the workspace."""
        import torch
        v = AttnCacheView()
        _check(library().spffn_attn_cache(self.ctx, ctypes.byref(v)), "spffn_attn_cache")
        base = self.workspace.data_ptr()
        dt = torch.bfloat16 if self.dtype == BF16 else torch.float16
        def view(ptr, nbytes):
            off = int(ptr) - base
            return self.workspace[off:off + nbytes]
        kv = self.nh * self.tmax * self.dh
        K = view(v.K, 2 * kv).view(dt).view(self.nh, self.tmax, self.dh)
        V = view(v.V, 2 * kv).view(dt).view(self.nh, self.tmax, self.dh)
        filled = view(v.filled, self.nh * self.tmax).view(self.nh, self.tmax)
        Y = view(v.Y, 2 * self.tmax * self.d).view(dt).view(self.tmax, self.d)
        t = view(v.t, 4).view(torch.int32)
        return K, V, filled, Y, t

    def last_device_error(self, stream=None):
        code = ctypes.c_uint32(0)
        s = library().spffn_attn_last_device_error(self.ctx, ctypes.byref(code), _stream(stream))
        return s, int(code.value)


def attn_step_kernel_launches() -> int:
    return int(library().spffn_attn_step_kernel_launches())


def forward_noalloc(layer: Layer, x, idx, count, y, stream=None):
    """spffn_forward for `layer`'s weights without its context or workspace
    (scratch in the library's fixed device array; see include/spffn.h)."""
    _check(library().spffn_forward_noalloc(ctypes.byref(layer.cfg), ctypes.byref(layer.weights), _p(x), x.shape[0],
                                           _p(idx), _p(count), _p(y), _stream(stream)), "spffn_forward_noalloc")


def decode(layers: Sequence[Layer], x_in, x_out, y, counts=None, stream=None, lookahead: bool = False):
    """One decode step through the stack (spffn_decode; with ``lookahead`` the
    set of layer l+1 is predicted from x_l, spffn_decode_lookahead)."""
    arr = (ctypes.c_void_p * len(layers))(*[l.ctx.value for l in layers])
    fn = library().spffn_decode_lookahead if lookahead else library().spffn_decode
    _check(fn(arr, len(layers), _p(x_in), x_in.shape[0], _p(x_out), _p(y), _p(counts), _stream(stream)),
           "spffn_decode_lookahead" if lookahead else "spffn_decode")


def decode_tables(layers: Sequence[Layer], x_in, tables, tab_counts, x_out, y, counts=None, stream=None):
    """One decode step on caller-supplied neuron tables, no predictor
    (spffn_decode_tables): ``tables`` is a sequence of L int32 CUDA tensors,
    ``tab_counts`` an int32 CUDA tensor [L] of their lengths."""
    arr = (ctypes.c_void_p * len(layers))(*[l.ctx.value for l in layers])
    tabs = (ctypes.c_void_p * len(tables))(*[_p(t) for t in tables])
    _check(library().spffn_decode_tables(arr, len(layers), _p(x_in), x_in.shape[0], tabs, _p(tab_counts),
                                         _p(x_out), _p(y), _p(counts), _stream(stream)), "spffn_decode_tables")


def decode_kernel_launches(layers: Sequence[Layer], B: int) -> int:
    arr = (ctypes.c_void_p * len(layers))(*[l.ctx.value for l in layers])
    return int(library().spffn_decode_kernel_launches(arr, len(layers), B))


def set_trace(buf=None):
    """Bind (or unbind with None) a uint64 CUDA tensor that whole-stack decode
    launches fill with per-(CTA, layer, mark) %globaltimer stamps."""
    if buf is None:
        _check(library().spffn_set_trace(None, 0), "spffn_set_trace")
    else:
        _check(library().spffn_set_trace(_p(buf), buf.numel() * buf.element_size()), "spffn_set_trace")


def trace_marks() -> int:
    return int(library().spffn_trace_marks())


def set_l2_hot_rows(rows_per_range: int):
    """Keep the first ``rows_per_range`` slots of every dealt range (the hottest
    neurons after the hot-first dealt placement) in L2 during small-batch decode
    (spffn_set_l2_hot_rows; 0 turns the cache hints off)."""
    _check(library().spffn_set_l2_hot_rows(int(rows_per_range)), "spffn_set_l2_hot_rows")


def l2_hot_rows() -> int:
    return int(library().spffn_l2_hot_rows())


UNION_PER_LAYER, UNION_STACK, UNION_AUTO = 0, 1, 2


def set_union_stack(mode: int):
    """How decode runs 3 <= B <= 128 (spffn_set_union_stack): UNION_STACK (one
    persistent launch), UNION_PER_LAYER, or UNION_AUTO (the default: the faster
    of the two on the measured shapes, per-layer launches at every batch)."""
    _check(library().spffn_set_union_stack(int(mode)), "spffn_set_union_stack")


def union_stack() -> int:
    return int(library().spffn_union_stack())


def reorder(counts: np.ndarray) -> np.ndarray:
    c = np.ascontiguousarray(counts, dtype=np.uint32)
    perm = np.empty(c.size, dtype=np.int32)
    _check(library().spffn_reorder(c.ctypes.data_as(ctypes.c_void_p), c.size,
                                   perm.ctypes.data_as(ctypes.c_void_p)), "spffn_reorder")
    return perm


def reorder_dealt(counts: np.ndarray, parts: int) -> np.ndarray:
    c = np.ascontiguousarray(counts, dtype=np.uint32)
    perm = np.empty(c.size, dtype=np.int32)
    _check(library().spffn_reorder_dealt(c.ctypes.data_as(ctypes.c_void_p), c.size, parts,
                                         perm.ctypes.data_as(ctypes.c_void_p)), "spffn_reorder_dealt")
    return perm


def permute_rows(src, dst, perm, stream=None):
    rows = src.shape[0]
    row_bytes = src[0].numel() * src.element_size()
    _check(library().spffn_permute_rows(_p(src), _p(dst), rows, row_bytes, _p(perm), _stream(stream)),
           "spffn_permute_rows")


def permute_vector(src, dst, perm, stream=None):
    _check(library().spffn_permute_vector(_p(src), _p(dst), src.numel(), _p(perm), _stream(stream)),
           "spffn_permute_vector")


# ---- the dense half of a batched decode block (include/spffn_block.h) -----------------------

_T = None            # torch, once a call of this part has needed it
_device_now = None   # the current device's index, and a device's current stream as an integer
_stream_now = None


def _torch():
    global _T, _device_now, _stream_now
    if _T is None:
        import torch
        # the index and the handle themselves where torch has them: the public calls build objects, and a decode
        # step makes several of these calls for kernels of a few microseconds
        _device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _stream_now = raw if raw is not None else lambda device: torch.cuda.current_stream(device).cuda_stream
        _T = torch
    return _T


def _on(device: int, *tensors):
    """Every tensor (None allowed) lives on CUDA device `device`."""
    if device < 0:
        raise TypeError("expected CUDA tensors")
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError("expected a CUDA tensor on device %d, got one on %s" % (device, t.device))


def _rows(t, what: str, dtype, T=None, d=None):
    """Row stride of a 2-D tensor whose rows are contiguous; checks its type and shape."""
    shape = t.shape
    if len(shape) != 2 or (T is not None and shape[0] != T) or (d is not None and shape[1] != d):
        raise ValueError("%s: expected shape [%s, %s], got %s" % (what, T, d, tuple(shape)))
    if t.dtype is not dtype:
        raise TypeError("%s: expected %s, got %s" % (what, dtype, t.dtype))
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError("%s: rows must be contiguous" % what)
    return ld if shape[0] > 1 else shape[1]


def _vector(t, what: str, dtype, n: int):
    if t.dtype is dtype and t.shape == (n,) and t.is_contiguous():
        return
    if t.dtype is not dtype:
        raise TypeError("%s: expected %s, got %s" % (what, dtype, t.dtype))
    raise ValueError("%s: expected a contiguous [%d], got %s" % (what, n, tuple(t.shape)))


def _made(device: int):
    """What a constructor has put on the current stream is done, so that its calls may go to any stream."""
    if not _T.cuda.is_current_stream_capturing():
        _T.cuda.current_stream(device).synchronize()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _status(device: int, stream, fn, *args):
    """fn(*args, stream) with `device` current; `stream` defaults to that device's current stream."""
    handle = _stream_now(device) if stream is None else getattr(stream, "cuda_stream", stream)
    if _device_now() == device:
        return fn(*args, handle)
    with _T.cuda.device(device):
        return fn(*args, handle)


def _call(device: int, stream, name: str, fn, *args):
    status = _status(device, stream, fn, *args)
    if status != OK:
        _check(status, name)


def norm_quant(x, y, g, x_out, q, scale, eps: float = 1e-6, stream=None):
    """Residual addition, RMS norm and 8-bit rows (spffn_norm_quant): ``u = x + y``, ``x_out = u`` in the
    storage type, ``q [T, d]`` int8 and ``scale [T]`` fp32 with ``q scale`` the normalised row times ``g``.
    ``x [T, d]`` float16 or bfloat16; ``y [T, d]`` of that type, float32 or None; ``g [d]`` or None; ``x_out``
    may be ``x`` (or ``y`` of the same type) or None."""
    torch = _torch()
    T, d = x.shape
    code, dev = _dtype_code(x), x.get_device()
    ldx = _rows(x, "x", x.dtype)
    y_f32 = y is not None and y.dtype == torch.float32
    ldy = 0 if y is None else _rows(y, "y", torch.float32 if y_f32 else x.dtype, T, d)
    ldo = 0 if x_out is None else _rows(x_out, "x_out", x.dtype, T, d)
    ldq = _rows(q, "q", torch.int8, T, d)
    _vector(scale, "scale", torch.float32, T)
    if g is not None:
        _vector(g, "g", x.dtype, d)
    _on(dev, x, y, g, x_out, q, scale)
    _call(dev, stream, "spffn_norm_quant", _lib.spffn_norm_quant if _lib is not None else library().spffn_norm_quant, T, d, code, x.data_ptr(), ldx, _ptr(y), ldy,
          y_f32, _ptr(g), eps, _ptr(x_out), ldo, q.data_ptr(), ldq, scale.data_ptr())


def quantize_rows(x, q, scale, stream=None):
    """8-bit rows with a scale each (spffn_quantize_rows): ``x [T, d]`` float16, bfloat16 or float32 to
    ``q [T, d]`` int8 and ``scale [T]`` fp32.  Weights ``[N, K]`` get their scales per channel this way."""
    torch = _torch()
    T, d = x.shape
    f32 = x.dtype == torch.float32
    code, dev = F16 if f32 else _dtype_code(x), x.get_device()
    ldx, ldq = _rows(x, "x", x.dtype), _rows(q, "q", torch.int8, T, d)
    _vector(scale, "scale", torch.float32, T)
    _on(dev, x, q, scale)
    _call(dev, stream, "spffn_quantize_rows", _lib.spffn_quantize_rows if _lib is not None else library().spffn_quantize_rows, T, d, code, x.data_ptr(), ldx, f32,
          q.data_ptr(), ldq, scale.data_ptr())


class Linear8:
    """A product with 8-bit weights (wraps an ``spffn_mm8_ctx``): ``y = round(scale[t] w_scale[n] sum_k q[t][k]
    W[n][k] + bias[n])`` with exact integer sums.

    ``W [N, K]`` int8 CUDA tensor, contiguous, K % 16 == 0; ``w_scale [N]`` fp32; ``bias [N]`` of ``dtype`` or
    None; ``dtype`` (torch.float16 or torch.bfloat16) is the output's type; ``max_tokens`` the most rows of a call.
    Keep the object until its calls have ended on the streams they were given (the workspace is its own).
    """

    def __init__(self, W, w_scale, bias=None, max_tokens: int = 256, dtype=None, workspace=None):
        torch = _torch()
        self.out_dtype = dtype if dtype is not None else bias.dtype if bias is not None else torch.float16
        self.N, self.K = (int(v) for v in W.shape)
        self.max_tokens = int(max_tokens)
        if _rows(W, "W", torch.int8) != self.K:
            raise ValueError("W must be contiguous")
        _vector(w_scale, "w_scale", torch.float32, self.N)
        if bias is not None:
            _vector(bias, "bias", self.out_dtype, self.N)
        self.device = W.get_device()
        code = {torch.float16: F16, torch.bfloat16: BF16}.get(self.out_dtype)
        if code is None:
            raise TypeError("dtype must be float16 or bfloat16, got %s" % self.out_dtype)
        _on(self.device, w_scale, bias, workspace)
        self.cfg = Mm8Config(self.K, self.N, self.max_tokens, code, 0)
        self._keep = [W, w_scale, bias]
        self.weights = Mm8Weights(_ptr(W), _ptr(w_scale), _ptr(bias))
        with torch.cuda.device(self.device):
            need = int(library().spffn_mm8_workspace_bytes(ctypes.byref(self.cfg)))
            if need == 0:
                raise SpffnError(ERR_INVALID_ARG, "spffn_mm8_workspace_bytes (bad shape)")
            if workspace is None:
                workspace = torch.zeros(need, dtype=torch.uint8, device=W.device)
            self.workspace = workspace
            ctx = ctypes.c_void_p()
            _check(library().spffn_mm8_create(ctypes.byref(self.cfg), ctypes.byref(self.weights), _p(workspace),
                                              workspace.numel(), ctypes.byref(ctx)), "spffn_mm8_create")
            _made(self.device)
        self.ctx = ctx

    def close(self):
        if getattr(self, "ctx", None):
            library().spffn_mm8_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, q, scale, y, stream=None):
        """``q [T, K]`` int8 and ``scale [T]`` fp32 (as norm_quant leaves them) to ``y [T, N]``."""
        torch = _torch()
        T = q.shape[0]
        ldq, ldy = _rows(q, "q", torch.int8, T, self.K), _rows(y, "y", self.out_dtype, T, self.N)
        _vector(scale, "scale", torch.float32, T)
        _on(self.device, q, scale, y)
        _call(self.device, stream, "spffn_mm8_forward", _lib.spffn_mm8_forward, self.ctx, q.data_ptr(), ldq,
              scale.data_ptr(), T, y.data_ptr(), ldy)

    def last_device_error(self, stream=None):
        code = ctypes.c_uint32(0)
        _torch()
        s = _status(self.device, stream, library().spffn_mm8_last_device_error, self.ctx, ctypes.byref(code))
        return s, int(code.value)


ROPE_SCALINGS = ("plain", "linear", "ntk", "parts")


def rope_frequencies(dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0, original_len: float = 0.0):
    """(radians per position of the dim / 2 rotated pairs as a float64 numpy array, amplitude) for the long-context
    scalings of spffn_rope_frequencies: "plain", "linear", "ntk", "parts"."""
    out, amp = np.empty(max(dim // 2, 1), dtype=np.float64), ctypes.c_double(1.0)
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % (ROPE_SCALINGS,))
    _check(library().spffn_rope_frequencies(int(dim), float(base), ROPE_SCALINGS.index(scaling), float(factor), float(original_len),
                                            out.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), ctypes.byref(amp)),
           "spffn_rope_frequencies")
    return out, float(amp.value)


class Rope:
    """Rotary positions of a cache: ``freqs`` (float64 CUDA tensor [dim / 2], radians per position, or a numpy array
    from rope_frequencies), pairs ``(2i, 2i + 1)`` if ``interleaved`` else ``(i, i + dim / 2)`` of the first dim dims."""

    def __init__(self, freqs, interleaved: bool = False, amplitude: float = 1.0):
        torch = _torch()
        self.freqs = torch.from_numpy(np.ascontiguousarray(freqs, dtype=np.float64)).cuda() if isinstance(freqs, np.ndarray) else freqs
        _vector(self.freqs, "freqs", torch.float64, self.freqs.numel())
        self.interleaved, self.amplitude = bool(interleaved), float(amplitude)


class KvCache4:
    """A paged cache of keys and values in 4 bits (wraps an ``spffn_kv4_ctx``): append with rotary positions, attend,
    read back.  The pool (uint8 CUDA tensor, allocated here when not given) has pages x page_size tokens of kvh heads of
    dh dims; ``max_seqs`` and ``max_tokens`` bound the sequences and new tokens of a call.  Keep the object until its
    calls have ended on the streams they were given (pool and workspace are its own).

    The batch of a call: ``table [B, width]`` int32 pages of each sequence, ``lens [B]`` int32 lengths with the new
    tokens included, ``start [B + 1]`` int32 first rows of the sequences' new tokens, or None for one token each.
    """

    def __init__(self, pages: int, page_size: int, nh: int, kvh: int, dh: int, dtype, max_seqs: int, max_tokens: int,
                 rope: Optional[Rope] = None, pool=None, workspace=None, device=None):
        torch = _torch()
        code = {torch.float16: F16, torch.bfloat16: BF16}.get(dtype)
        if code is None:
            raise TypeError("dtype must be float16 or bfloat16, got %s" % dtype)
        self.pages, self.page_size, self.nh, self.kvh, self.dh, self.dtype = int(pages), int(page_size), int(nh), int(kvh), int(dh), dtype
        self.rope = rope
        self.cfg = Kv4Config(self.pages, self.page_size, self.nh, self.kvh, self.dh, int(max_seqs), int(max_tokens), code,
                             0 if rope is None else 2 * rope.freqs.numel(), rope is not None and rope.interleaved,
                             0, 1.0 if rope is None else rope.amplitude)
        device = pool.device if pool is not None else torch.device("cuda" if device is None else device)
        with torch.cuda.device(device):
            size = int(library().spffn_kv4_pool_bytes(ctypes.byref(self.cfg)))
            need = int(library().spffn_kv4_workspace_bytes(ctypes.byref(self.cfg)))
            if size == 0 or need == 0:
                raise SpffnError(ERR_INVALID_ARG, "spffn_kv4_pool_bytes (bad shape)")
            if pool is None:
                pool = torch.zeros(size, dtype=torch.uint8, device=device)
            if workspace is None:
                workspace = torch.zeros(need, dtype=torch.uint8, device=device)
            self.device = pool.get_device()
            _on(self.device, pool, workspace, None if rope is None else rope.freqs)
            self.pool, self.workspace = pool, workspace
            ctx = ctypes.c_void_p()
            _check(library().spffn_kv4_create(ctypes.byref(self.cfg), _p(pool), pool.numel() * pool.element_size(),
                                              None if rope is None else rope.freqs.data_ptr(), _p(workspace),
                                              workspace.numel(), ctypes.byref(ctx)), "spffn_kv4_create")
            _made(self.device)
        self.ctx = ctx

    def close(self):
        if getattr(self, "ctx", None):
            library().spffn_kv4_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _heads(self, t, what: str, T: int, heads: int):
        """Row stride of [T, heads, dh] (or [T, heads * dh]) whose rows are contiguous."""
        if t is None:
            raise TypeError("%s: expected a tensor, got None" % what)
        if t.dim() == 3:
            ld, head, one = t.stride()
            if t.shape != (T, heads, self.dh) or one != 1 or (head != self.dh and heads > 1):
                raise ValueError("%s: expected [%d, %d, %d] with contiguous rows, got %s, strides %s" % (
                    what, T, heads, self.dh, tuple(t.shape), t.stride()))
            if t.dtype is not self.dtype:
                raise TypeError("%s: expected %s, got %s" % (what, self.dtype, t.dtype))
            return ld if T > 1 else heads * self.dh
        return _rows(t, what, self.dtype, T, heads * self.dh)

    def _batch(self, table, lens, start):
        torch = _torch()
        B = lens.shape[0]
        ldt = _rows(table, "table", torch.int32, B)
        _vector(lens, "lens", torch.int32, B)
        if start is not None:
            _vector(start, "start", torch.int32, B + 1)
        _on(self.device, table, lens, start)
        return table.data_ptr(), ldt, table.shape[1], lens.data_ptr(), _ptr(start), B

    def append(self, q, k, v, table, lens, start=None, q_out=None, stream=None):
        """Rotate ``q [T, nh, dh]`` into ``q_out`` (may be ``q``; both None to leave it out) and append ``k, v
        [T, kvh, dh]``, k rotated, at their sequences' positions."""
        _torch()
        T = k.shape[0]
        ldk, ldv = self._heads(k, "k", T, self.kvh), self._heads(v, "v", T, self.kvh)
        ldq, ldo = (0, 0) if q is None else (self._heads(q, "q", T, self.nh), 0)
        if q_out is not None:
            ldo = self._heads(q_out, "q_out", T, self.nh)
        batch = self._batch(table, lens, start)
        _on(self.device, q, k, v, q_out)
        _call(self.device, stream, "spffn_kv4_append", _lib.spffn_kv4_append, self.ctx, _ptr(q), ldq, k.data_ptr(),
              ldk, v.data_ptr(), ldv, T, *batch, _ptr(q_out), ldo)

    def attend(self, q, table, lens, start=None, out=None, scale: Optional[float] = None, stream=None):
        """Attention of the new tokens' ``q [T, nh, dh]`` over their sequences' cached positions up to their own, into
        ``out [T, nh, dh]``; ``scale`` defaults to 1 / sqrt(dh)."""
        _torch()
        T = q.shape[0]
        ldq, ldo = self._heads(q, "q", T, self.nh), self._heads(out, "out", T, self.nh)
        batch = self._batch(table, lens, start)
        _on(self.device, q, out)
        _call(self.device, stream, "spffn_kv4_attend", _lib.spffn_kv4_attend, self.ctx, q.data_ptr(), ldq, T, *batch,
              self.dh ** -0.5 if scale is None else scale, out.data_ptr(), ldo)

    def read(self, pages, K, V, stream=None):
        """The cached values of ``pages [n]`` (int32) into ``K, V [n, page_size, kvh, dh]``."""
        torch = _torch()
        n = pages.shape[0]
        _vector(pages, "pages", torch.int32, n)
        for t, what in ((K, "K"), (V, "V")):
            if t.shape != (n, self.page_size, self.kvh, self.dh) or not t.is_contiguous():
                raise ValueError("%s: expected a contiguous %s, got %s" % (what, (n, self.page_size, self.kvh, self.dh), tuple(t.shape)))
            if t.dtype != self.dtype:
                raise TypeError("%s: expected %s, got %s" % (what, self.dtype, t.dtype))
        _on(self.device, pages, K, V)
        _call(self.device, stream, "spffn_kv4_read", _lib.spffn_kv4_read, self.ctx, pages.data_ptr(), n, K.data_ptr(),
              V.data_ptr())

    def last_device_error(self, stream=None):
        code = ctypes.c_uint32(0)
        _torch()
        s = _status(self.device, stream, library().spffn_kv4_last_device_error, self.ctx, ctypes.byref(code))
        return s, int(code.value)
