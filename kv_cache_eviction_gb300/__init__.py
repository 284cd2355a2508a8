"""Python binding of libkvevict: head-adaptive KV-cache eviction and flat decode attention
on GB300 (sm_103a).

Every function here only marshals arguments (torch CUDA tensors to device
pointers, the current stream) and calls the C ABI declared in
``include/kvevict.h``; all computation runs in the library's CUDA kernels.
There is no CPU fallback: if ``libkvevict.so`` has not been built, or a tensor
is not on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import importlib
import os
from typing import Optional

from .rotary import kv_rotary_inv_freq

__all__ = [
    "KV_OK", "KV_ERR_INVALID_ARG", "KV_ERR_UNSUPPORTED", "KV_ERR_WORKSPACE", "KV_ERR_CAPACITY",
    "KV_ERR_CUDA", "KV_ERR_DEVICE_CHECK", "KV_BF16", "KV_F32", "KV_SCORE_ADA", "KV_SCORE_LAVA",
    "KV_SCORE_CRITICAL", "KV_GROUP_MEAN", "KV_GROUP_MAX", "KV_OP_SCORE", "KV_OP_ALLOCATE",
    "KV_OP_COMPACT", "KV_OP_DECODE", "KvShape", "KvError", "lib", "library_path",
    "kv_workspace_size", "kv_score", "kv_crit_norm", "kv_allocate", "kv_allocate_capped",
    "kv_compact", "kv_recompact", "kv_recompact_workspace_size", "kv_window_terms",
    "kv_proj_score", "kv_compact_kappa", "kv_compact_streaming", "KV_TERMS_MEAN_POOLED",
    "KV_TERMS_L2",
    "KV_PROJ_CRIT_GQA", "KV_PROJ_LAPROX",
    "flat_decode_attn", "kv_check_device_status", "kv_status_string", "kv_kernel_launches",
    "flat_decode_attn_noalloc",
    "KV_OP_PAGE_MAP", "KV_OP_PAGED_WRITE", "KV_OP_PAGED_DECODE", "KV_PAGE_MAP_MAX_TABLES",
    "KV_PAGED_DECODE_MAX_TABLES",
    "KvPagedShape", "kv_paged_workspace_size", "kv_page_map", "kv_paged_write",
    "paged_decode_attn",
    "KV_OP_QUANT_WRITE", "KV_OP_QUANT_READ", "KV_OP_QUANT_DECODE", "KV_E4M3", "KV_INT8",
    "KV_QUANT_BLOCK", "kv_quant_write", "kv_quant_read", "quant_decode_attn",
    "KV_ROTARY_HALF", "KV_ROTARY_INTERLEAVED", "KvRotaryShape", "kv_rotary", "kv_rotary_inv_freq",
]

KV_OK, KV_ERR_INVALID_ARG, KV_ERR_UNSUPPORTED, KV_ERR_WORKSPACE = 0, 1, 2, 3
KV_ERR_CAPACITY, KV_ERR_CUDA, KV_ERR_DEVICE_CHECK = 4, 5, 6
KV_BF16, KV_F32 = 0, 1
KV_SCORE_ADA, KV_SCORE_LAVA, KV_SCORE_CRITICAL = 0, 1, 2
KV_GROUP_MEAN, KV_GROUP_MAX = 0, 1
KV_OP_SCORE, KV_OP_ALLOCATE, KV_OP_COMPACT, KV_OP_DECODE = 0, 1, 2, 3
KV_OP_PAGE_MAP, KV_OP_PAGED_WRITE, KV_OP_PAGED_DECODE = 4, 5, 6
KV_OP_QUANT_WRITE, KV_OP_QUANT_READ, KV_OP_QUANT_DECODE = 16, 17, 18
KV_E4M3, KV_INT8 = 0, 1
KV_QUANT_BLOCK = 16
KV_ROTARY_HALF, KV_ROTARY_INTERLEAVED = 0, 1
KV_PAGE_MAP_MAX_TABLES = 16384
KV_PAGED_DECODE_MAX_TABLES = 1 << 20
KV_TERMS_MEAN_POOLED, KV_TERMS_L2 = 0, 1
KV_PROJ_CRIT_GQA, KV_PROJ_LAPROX = 0, 1

_HERE = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    return os.path.join(_HERE, "libkvevict.so")


class KvShape(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in
                ("batch", "layers", "hq", "hkv", "d", "n", "w", "pool", "dtype")]

    @classmethod
    def of(cls, batch, layers, hq, hkv, d, n, w, pool, dtype) -> "KvShape":
        if isinstance(dtype, str):
            dtype = KV_BF16 if dtype == "bf16" else KV_F32
        return cls(batch, layers, hq, hkv, d, n, w, pool, dtype)

    @classmethod
    def from_workload(cls, wl, batch: Optional[int] = None, layers: Optional[int] = None):
        return cls.of(wl.batch if batch is None else batch, wl.layers if layers is None else layers,
                      wl.hq, wl.hkv, wl.d, wl.n, wl.w, wl.pool, wl.dtype)


class KvPagedShape(ctypes.Structure):
    """Shape of a paged cache; ``page_stride`` (elements) 0 means dense pages."""
    _fields_ = [(f, ctypes.c_int32) for f in
                ("seqs", "hq", "hkv", "d", "tables", "page", "max_pages", "dtype")] + \
               [("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64)]

    @classmethod
    def of(cls, seqs, hq, hkv, d, tables, page, max_pages, dtype, num_pages,
           page_stride=0) -> "KvPagedShape":
        if isinstance(dtype, str):
            dtype = KV_BF16 if dtype == "bf16" else KV_F32
        return cls(seqs, hq, hkv, d, tables, page, max_pages, dtype, num_pages, page_stride)


class KvRotaryShape(ctypes.Structure):
    """Heads and pairs of ``kv_rotary``; ``magnitude`` goes with ``kv_rotary_inv_freq``."""
    _fields_ = [(f, ctypes.c_int32) for f in ("hq", "hkv", "d", "rot", "layout", "dtype")] + \
               [("magnitude", ctypes.c_float)]

    @classmethod
    def of(cls, hq, hkv, d, rot, layout, dtype, magnitude=1.0) -> "KvRotaryShape":
        if isinstance(dtype, str):
            dtype = KV_BF16 if dtype == "bf16" else KV_F32
        return cls(hq, hkv, d, rot, layout, dtype, magnitude)


class KvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__("%s: %s (status %d)" % (fn, kv_status_string(status), status))


_LIB = None
_vp, _sz, _i32, _u32, _f32, _i64 = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32,
                                     ctypes.c_uint32, ctypes.c_float, ctypes.c_int64)
_SIGS = {
    "kv_workspace_size": (_sz, [ctypes.c_int, ctypes.POINTER(KvShape)]),
    "kv_score": (ctypes.c_int, [ctypes.POINTER(KvShape), ctypes.c_int, ctypes.c_int, _vp, _vp, _vp,
                                _vp, _i32, _vp, _vp, _vp, _sz, _vp]),
    "kv_crit_norm": (ctypes.c_int, [ctypes.POINTER(KvShape), _vp, _vp, _i32, _vp, _vp, _sz, _vp]),
    "kv_window_terms": (ctypes.c_int, [ctypes.POINTER(KvShape), ctypes.c_int, _vp, _vp, _vp, _vp,
                                       _sz, _vp]),
    "kv_proj_score": (ctypes.c_int, [ctypes.POINTER(KvShape), ctypes.c_int, _vp, _vp, _i32, _vp,
                                     _f32, _vp, _vp, _sz, _vp]),
    "kv_compact_streaming": (ctypes.c_int, [ctypes.POINTER(KvShape), _vp, _vp, _i32, _vp, _i32,
                                            _vp, _vp, _vp, _vp, _vp, _i64, _vp, _sz, _vp]),
    "kv_compact_kappa": (ctypes.c_int, [ctypes.POINTER(KvShape), _vp, _vp, _vp, _vp, _u32, _u32,
                                        _vp, _i32, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _sz,
                                        _vp]),
    "kv_allocate_capped": (ctypes.c_int, [ctypes.POINTER(KvShape), _vp, _vp, _vp, _u32, _u32,
                                          _vp, _vp, _vp, _sz, _vp]),
    "kv_recompact_workspace_size": (_sz, [_i64]),
    "kv_recompact": (ctypes.c_int, [ctypes.POINTER(KvShape), _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                    _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _sz,
                                    _vp]),
    "kv_allocate": (ctypes.c_int, [ctypes.POINTER(KvShape), _vp, _vp, ctypes.c_int, _u32, _u32,
                                   _vp, _vp, _vp, _sz, _vp]),
    "kv_compact": (ctypes.c_int, [ctypes.POINTER(KvShape), _vp, _vp, _vp, _vp, _u32, _u32, _f32,
                                  _vp, _i32, _vp, _vp, _vp, _vp, _vp, _i64, _vp, _sz, _vp]),
    "flat_decode_attn": (ctypes.c_int, [ctypes.POINTER(KvShape), _vp, _vp, _vp, _vp, _vp, _vp,
                                        _vp, _i64, _f32, _vp, _vp, _sz, _vp]),
    "kv_check_device_status": (ctypes.c_int, [_vp, _vp, ctypes.POINTER(_u32)]),
    "kv_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kv_kernel_launches": (ctypes.c_uint64, []),
    "flat_decode_attn_noalloc": (ctypes.c_int, [ctypes.POINTER(KvShape), _vp, _vp, _vp, _vp, _vp,
                                                _vp, _vp, _i64, _f32, _vp, _vp]),
    "kv_paged_workspace_size": (_sz, [ctypes.c_int, ctypes.POINTER(KvPagedShape)]),
    "kv_page_map": (ctypes.c_int, [ctypes.POINTER(KvPagedShape), _vp, _vp, _vp, _vp, _i64, _vp,
                                   _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "kv_paged_write": (ctypes.c_int, [ctypes.POINTER(KvPagedShape), _vp, _vp, _i64, _vp, _i64,
                                      _vp, _vp, _vp, _vp, _sz, _vp]),
    "paged_decode_attn": (ctypes.c_int, [ctypes.POINTER(KvPagedShape), _vp, _vp, _vp, _vp, _vp,
                                         _i64, _vp, _vp, _vp, _vp, _f32, _vp, _vp, _sz, _vp]),
    "kv_quant_write": (ctypes.c_int, [ctypes.POINTER(KvPagedShape), ctypes.c_int, _vp, _vp, _i64,
                                      _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "kv_quant_read": (ctypes.c_int, [ctypes.POINTER(KvPagedShape), ctypes.c_int, _vp, _vp, _vp,
                                     _vp, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _sz, _vp]),
    "quant_decode_attn": (ctypes.c_int, [ctypes.POINTER(KvPagedShape), ctypes.c_int, _vp, _vp, _vp,
                                         _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _f32, _vp,
                                         _vp, _sz, _vp]),
    "kv_rotary": (ctypes.c_int, [ctypes.POINTER(KvRotaryShape), ctypes.c_int, _vp, _i64, _vp, _i64,
                                 _vp, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp]),
}


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError("libkvevict.so is not built: run __graft_entry__.build() "
                               "or python -m kv_cache_eviction_gb300._build")
        L = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _ptr(t) -> Optional[int]:
    """Device pointer of a CUDA tensor (None stays NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, st: int) -> None:
    if st != KV_OK:
        raise KvError(fn, st)


def kv_status_string(status: int) -> str:
    return lib().kv_status_string(status).decode()


def kv_workspace_size(op: int, shape: KvShape) -> int:
    return int(lib().kv_workspace_size(op, ctypes.byref(shape)))


def kv_score(shape: KvShape, mode: int, group: int, q_win, k, v, w_o, model_dim: int, scores,
             crit_norm, ws, stream=None) -> None:
    st = lib().kv_score(ctypes.byref(shape), mode, group, _ptr(q_win), _ptr(k), _ptr(v), _ptr(w_o),
                        model_dim, _ptr(scores), _ptr(crit_norm), _ptr(ws), _nbytes(ws),
                        _stream(stream))
    _check("kv_score", st)


def kv_crit_norm(shape: KvShape, v, w_o, model_dim: int, crit_norm, ws, stream=None) -> None:
    st = lib().kv_crit_norm(ctypes.byref(shape), _ptr(v), _ptr(w_o), model_dim, _ptr(crit_norm),
                            _ptr(ws), _nbytes(ws), _stream(stream))
    _check("kv_crit_norm", st)


def kv_allocate(shape: KvShape, scores, budget, layer_entropy_mode: int, alpha_num: int,
                alpha_den: int, layer_budget, head_budget, ws, stream=None) -> None:
    st = lib().kv_allocate(ctypes.byref(shape), _ptr(scores), _ptr(budget), layer_entropy_mode,
                           alpha_num, alpha_den, _ptr(layer_budget), _ptr(head_budget), _ptr(ws),
                           _nbytes(ws), _stream(stream))
    _check("kv_allocate", st)


def kv_window_terms(shape: KvShape, kind: int, q_win, k, terms, ws, stream=None) -> None:
    st = lib().kv_window_terms(ctypes.byref(shape), kind, _ptr(q_win), _ptr(k), _ptr(terms),
                               _ptr(ws), _nbytes(ws), _stream(stream))
    _check("kv_window_terms", st)


def kv_proj_score(shape: KvShape, kind: int, v, w_o, model_dim: int, terms, eps: float, out, ws,
                  stream=None) -> None:
    st = lib().kv_proj_score(ctypes.byref(shape), kind, _ptr(v), _ptr(w_o), model_dim,
                             _ptr(terms), eps, _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream))
    _check("kv_proj_score", st)


def kv_compact_streaming(shape: KvShape, k, v, sinks: int, head_budget, reserve: int, kept_idx,
                         cu_off, lens, k_flat, v_flat, flat_capacity_rows: int, ws,
                         stream=None) -> None:
    st = lib().kv_compact_streaming(ctypes.byref(shape), _ptr(k), _ptr(v), sinks,
                                    _ptr(head_budget), reserve, _ptr(kept_idx), _ptr(cu_off),
                                    _ptr(lens), _ptr(k_flat), _ptr(v_flat), flat_capacity_rows,
                                    _ptr(ws), _nbytes(ws), _stream(stream))
    _check("kv_compact_streaming", st)


def kv_compact_kappa(shape: KvShape, k, v, scores, kappa, crit_alpha_num: int,
                     crit_alpha_den: int, head_budget, reserve: int, kept_idx, cu_off, lens,
                     k_flat, v_flat, flat_capacity_rows: int, ws, stream=None) -> None:
    st = lib().kv_compact_kappa(ctypes.byref(shape), _ptr(k), _ptr(v), _ptr(scores), _ptr(kappa),
                                crit_alpha_num, crit_alpha_den, _ptr(head_budget), reserve,
                                _ptr(kept_idx), _ptr(cu_off), _ptr(lens), _ptr(k_flat),
                                _ptr(v_flat), flat_capacity_rows, _ptr(ws), _nbytes(ws),
                                _stream(stream))
    _check("kv_compact_kappa", st)


def kv_allocate_capped(shape: KvShape, scores, budget, layer_cap, alpha_num: int, alpha_den: int,
                       layer_budget, head_budget, ws, stream=None) -> None:
    st = lib().kv_allocate_capped(ctypes.byref(shape), _ptr(scores), _ptr(budget),
                                  _ptr(layer_cap), alpha_num, alpha_den, _ptr(layer_budget),
                                  _ptr(head_budget), _ptr(ws), _nbytes(ws), _stream(stream))
    _check("kv_allocate_capped", st)


def kv_recompact_workspace_size(src_capacity_rows: int) -> int:
    return int(lib().kv_recompact_workspace_size(src_capacity_rows))


def kv_recompact(shape: KvShape, scores, head_budget, src_kept, src_cu, src_lens, src_k, src_v,
                 reserve: int, row_base, kept_idx, cu_off, lens, k_flat, v_flat, ws,
                 stream=None, src_capacity_rows=None, flat_capacity_rows=None) -> None:
    """src_kept / src_cu / src_lens None: the source is the uncompacted K/V."""
    src_cap = src_k.shape[0] if src_capacity_rows is None else src_capacity_rows
    if src_kept is None:
        src_cap = 0
    cap = k_flat.shape[0] if flat_capacity_rows is None else flat_capacity_rows
    st = lib().kv_recompact(ctypes.byref(shape), _ptr(scores), _ptr(head_budget), _ptr(src_kept),
                            _ptr(src_cu), _ptr(src_lens), _ptr(src_k), _ptr(src_v), src_cap,
                            reserve, _ptr(row_base), _ptr(kept_idx), _ptr(cu_off), _ptr(lens),
                            _ptr(k_flat), _ptr(v_flat), cap, _ptr(ws), _nbytes(ws),
                            _stream(stream))
    _check("kv_recompact", st)


def kv_compact(shape: KvShape, k, v, scores, crit_norm, crit_alpha_num: int, crit_alpha_den: int,
               crit_eps: float, head_budget, reserve: int, kept_idx, cu_off, lens, k_flat, v_flat,
               flat_capacity_rows: int, ws, stream=None) -> None:
    st = lib().kv_compact(ctypes.byref(shape), _ptr(k), _ptr(v), _ptr(scores), _ptr(crit_norm),
                          crit_alpha_num, crit_alpha_den, crit_eps, _ptr(head_budget), reserve,
                          _ptr(kept_idx), _ptr(cu_off), _ptr(lens), _ptr(k_flat), _ptr(v_flat),
                          flat_capacity_rows, _ptr(ws), _nbytes(ws), _stream(stream))
    _check("kv_compact", st)


def flat_decode_attn(shape: KvShape, q, k_new, v_new, k_flat, v_flat, cu_off, lens,
                     softmax_scale: float, out, ws, stream=None, flat_capacity_rows=None) -> None:
    cap = k_flat.shape[0] if flat_capacity_rows is None else flat_capacity_rows
    st = lib().flat_decode_attn(ctypes.byref(shape), _ptr(q), _ptr(k_new), _ptr(v_new),
                                _ptr(k_flat), _ptr(v_flat), _ptr(cu_off), _ptr(lens), cap,
                                softmax_scale, _ptr(out), _ptr(ws), _nbytes(ws), _stream(stream))
    _check("flat_decode_attn", st)


def flat_decode_attn_noalloc(shape: KvShape, q, k_new, v_new, k_flat, v_flat, cu_off, lens,
                             softmax_scale: float, out, stream=None,
                             flat_capacity_rows=None) -> None:
    """flat_decode_attn without a workspace: the library's fixed device scratch is used."""
    cap = k_flat.shape[0] if flat_capacity_rows is None else flat_capacity_rows
    st = lib().flat_decode_attn_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k_new), _ptr(v_new),
                                        _ptr(k_flat), _ptr(v_flat), _ptr(cu_off), _ptr(lens), cap,
                                        softmax_scale, _ptr(out), _stream(stream))
    _check("flat_decode_attn_noalloc", st)


def kv_paged_workspace_size(op: int, shape: KvPagedShape) -> int:
    return int(lib().kv_paged_workspace_size(op, ctypes.byref(shape)))


# torch's dtypes and lookups for the paged calls, set when the first of them runs
_I32 = _I64 = _F32 = _F64 = _device_now = _stream_now = None
_ROWS = {}
_CODES = {}   # types that the codes of a format may come as


# csrc/binding.cpp as a module, once torch is there: it checks a call's tensors and calls the C
# function, or returns None for the code below to do it.  None: not built, or for another torch or
# Python than these; calls go through ctypes.
_quick = None
_FAST_CALLS = ("kv_quant_write", "kv_quant_read", "quant_decode_attn", "kv_rotary")


def _init_fast() -> None:
    global _quick
    from . import _build
    if not os.path.exists(_build.FAST):
        return
    why = ""
    # (it may load with another torch and read tensors at the wrong places, so this comes first)
    if _build.binding_built_for() != _build.binding_tag():
        why = "is not built for this torch and Python"
    else:
        try:
            fast = importlib.import_module("._fast", __package__)
        except ImportError as e:
            why = "does not load (%s)" % e
    if why:
        import warnings
        warnings.warn("kv_cache_eviction_gb300: _fast.so %s: build again" % why)
        return
    fast.bind(*(ctypes.cast(getattr(lib(), f), _vp).value for f in _FAST_CALLS))
    _quick = fast


def _init_torch() -> None:
    global _I32, _I64, _F32, _F64, _device_now, _stream_now
    import torch
    _I32, _I64, _F32, _F64 = torch.int32, torch.int64, torch.float32, torch.float64
    _ROWS.update({KV_BF16: torch.bfloat16, KV_F32: torch.float32})
    _CODES.update({KV_E4M3: (torch.float8_e4m3fn, torch.uint8), KV_INT8: (torch.int8,)})
    _stream_now = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    torch.cuda.init()   # (current_device() would ask for it on every call)
    _init_fast()
    _device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device(t, what: str) -> int:
    """The current device (a host tensor raises before CUDA is asked)."""
    if t is not None and not isinstance(t, int) and not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % what)
    if _device_now is None:
        _init_torch()
    return _device_now()


def _buf(t, dtype, count: int, dev: int, what: str) -> Optional[int]:
    """Device pointer of a contiguous tensor of the type and at least the entries that the call
    may touch, on the current device (None stays NULL, an int is a pointer already)."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.numel() >= count and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        if t is None or isinstance(t, int):
            return t
        raise
    if t.get_device() != dev:
        raise ValueError("%s must be on the current CUDA device" % what)
    if t.dtype is not dtype:
        raise ValueError("%s must be %s" % (what, dtype))
    if t.numel() < count:
        raise ValueError("%s has %d entries, needs %d" % (what, t.numel(), count))
    raise ValueError("%s must be contiguous" % what)


def _work(ws, dev: int):
    """Pointer and bytes of a workspace (of any type; None stays NULL)."""
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be contiguous on the current CUDA device")
    return ws.data_ptr(), ws.nbytes


def _rows_view(t, dtype, row: int, dev: int, what: str):
    """Pointer, count and stride (elements) of rows of `row` elements, [n][...]; a row is
    contiguous, rows may lie apart (parts of a fused projection)."""
    if t is None or t.get_device() != dev or t.dtype is not dtype:
        raise ValueError("%s must be %s on the current CUDA device" % (what, dtype))
    size = t.shape
    n = size[0]
    if len(size) < 2 or t.numel() != n * row:
        raise ValueError("%s must be rows of %d elements" % (what, row))
    stride = row
    if not t.is_contiguous():
        strides, step = t.stride(), 1
        for k in range(len(size) - 1, 0, -1):
            if size[k] > 1 and strides[k] != step:
                raise ValueError("the rows of %s must be contiguous" % what)
            step *= size[k]
        if n > 1:
            stride = strides[0]
            if stride < row:   # (0 would mean dense rows)
                raise ValueError("the rows of %s must not overlap" % what)
    return t.data_ptr(), n, stride


def _pool(t, dtype, inner: int, pages: int, page_stride: int, dev: int, what: str):
    """Pointer of a page pool: pages of `inner` elements, dense, ``page_stride`` apart."""
    try:
        if t.dtype is dtype and t.get_device() == dev:
            n = t.shape[0]
            if n >= pages and t.numel() == n * inner:
                if t.is_contiguous() and (page_stride == inner or pages == 1):
                    return t.data_ptr()
                size, strides, step, ok = t.shape, t.stride(), 1, True
                for k in range(len(size) - 1, 0, -1):
                    ok = ok and (size[k] == 1 or strides[k] == step)
                    step *= size[k]
                if ok and (pages == 1 or strides[0] == page_stride):
                    return t.data_ptr()
    except AttributeError:
        if t is None or isinstance(t, int):
            return t
        raise
    raise ValueError("%s must be [num_pages][heads][page][d] %s on the current CUDA device, pages "
                     "page_stride apart" % (what, dtype))


def _stream_on(stream, dev: int) -> Optional[int]:
    if stream is None:
        return _stream_now(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def kv_page_map(shape: KvPagedShape, lens, add, free_ring, free_state, block_table, lens_out,
                free_out, cu_add, slot_map, ws, stream=None) -> None:
    """Block tables, slots and lengths for the rows each table gains or loses.  ``lens_out`` may
    be ``lens`` and ``free_out`` may be ``free_state``; ``slot_map`` None: no table gains rows."""
    dev = _device(lens, "lens")
    i32, i64, n = _I32, _I64, shape.seqs * shape.tables
    wp, wn = _work(ws, dev)
    st = lib().kv_page_map(
        ctypes.byref(shape), _buf(lens, i32, n, dev, "lens"), _buf(add, i32, n, dev, "add"),
        _buf(free_ring, i32, shape.num_pages, dev, "free_ring"),
        _buf(free_state, i64, 2, dev, "free_state"), 0 if slot_map is None else slot_map.numel(),
        _buf(block_table, i32, n * shape.max_pages, dev, "block_table"),
        _buf(lens_out, i32, n, dev, "lens_out"), _buf(free_out, i64, 2, dev, "free_out"),
        _buf(cu_add, i64, n + 1, dev, "cu_add"), _buf(slot_map, i64, 0, dev, "slot_map"), wp, wn,
        _stream_on(stream, dev))
    if st:
        raise KvError("kv_page_map", st)


def kv_paged_write(shape: KvPagedShape, k, v, slot_map, n_rows, k_pages, v_pages, ws,
                   stream=None) -> None:
    """Rows of ``k`` and ``v`` ([n][heads per page][d], rows may lie apart) at their slots.
    ``n_rows`` (a device int64, or None): rows from there on are left out."""
    dev = _device(k, "k")
    el, row, pages = _ROWS.get(shape.dtype), shape.hkv // shape.tables * shape.d, shape.num_pages
    inner = row * shape.page
    apart = shape.page_stride or inner
    kp, n, ks = _rows_view(k, el, row, dev, "k")
    vp, nv, vs = _rows_view(v, el, row, dev, "v")
    if ks != vs or n != nv:
        raise ValueError("k and v must have the same rows and row stride")
    wp, wn = _work(ws, dev)
    st = lib().kv_paged_write(
        ctypes.byref(shape), kp, vp, ks, _buf(slot_map, _I64, n, dev, "slot_map"), n,
        _buf(n_rows, _I64, 1, dev, "n_rows"), _pool(k_pages, el, inner, pages, apart, dev, "k_pages"),
        _pool(v_pages, el, inner, pages, apart, dev, "v_pages"), wp, wn, _stream_on(stream, dev))
    if st:
        raise KvError("kv_paged_write", st)


def paged_decode_attn(shape: KvPagedShape, q, k_new, v_new, cu_add, slot_map, k_pages, v_pages,
                      block_table, lens, softmax_scale: float, out, ws, stream=None) -> None:
    """One decode step over the paged cache; ``k_new`` / ``v_new`` / ``cu_add`` / ``slot_map``
    None: no rows are stored."""
    dev = _device(q, "q")
    el, seqs, hkv, d, tables = _ROWS.get(shape.dtype), shape.seqs, shape.hkv, shape.d, shape.tables
    n, nq, nk, pages = seqs * tables, seqs * shape.hq * d, seqs * hkv * d, shape.num_pages
    inner = hkv // tables * shape.page * d
    apart = shape.page_stride or inner
    wp, wn = _work(ws, dev)
    st = lib().paged_decode_attn(
        ctypes.byref(shape), _buf(q, el, nq, dev, "q"), _buf(k_new, el, nk, dev, "k_new"),
        _buf(v_new, el, nk, dev, "v_new"), _buf(cu_add, _I64, n + 1, dev, "cu_add"),
        _buf(slot_map, _I64, 0, dev, "slot_map"), 0 if slot_map is None else slot_map.numel(),
        _pool(k_pages, el, inner, pages, apart, dev, "k_pages"),
        _pool(v_pages, el, inner, pages, apart, dev, "v_pages"),
        _buf(block_table, _I32, n * shape.max_pages, dev, "block_table"),
        _buf(lens, _I32, n, dev, "lens"), softmax_scale, _buf(out, el, nq, dev, "out"), wp, wn,
        _stream_on(stream, dev))
    if st:
        raise KvError("paged_decode_attn", st)


def _code_pool(t, format: int, inner: int, pages: int, page_stride: int, dev: int, what: str):
    """Pointer of a page pool of codes (one byte each)."""
    types = _CODES.get(format)
    if types is None:
        raise ValueError("format must be KV_E4M3 or KV_INT8")
    el = getattr(t, "dtype", None)
    return _pool(t, el if el in types else types[0], inner, pages, page_stride, dev, what)


def kv_quant_write(shape: KvPagedShape, format: int, k, v, slot_map, n_rows, k_pages, v_pages,
                   k_scale, v_scale, ws, stream=None) -> None:
    """``kv_paged_write`` into a cache in 8 bits: ``k_pages`` / ``v_pages`` hold codes (float8 e4m3
    or uint8 for KV_E4M3, int8 for KV_INT8), ``k_scale`` / ``v_scale`` [num_pages][heads per
    page][page / 16] float32 the scales of their blocks of 16 rows."""
    if _quick is not None:
        st = _quick.kv_quant_write(shape, format, k, v, slot_map, n_rows, k_pages, v_pages,
                                   k_scale, v_scale, ws, stream)
        if st == 0:
            return
        if st is not None:
            raise KvError("kv_quant_write", st)
    dev = _device(k, "k")
    heads, pages = shape.hkv // shape.tables, shape.num_pages
    el, row, inner = _ROWS.get(shape.dtype), heads * shape.d, heads * shape.d * shape.page
    apart, blocks = shape.page_stride or inner, pages * heads * (shape.page // 16)
    kp, n, ks = _rows_view(k, el, row, dev, "k")
    vp, nv, vs = _rows_view(v, el, row, dev, "v")
    if ks != vs or n != nv:
        raise ValueError("k and v must have the same rows and row stride")
    wp, wn = _work(ws, dev)
    st = lib().kv_quant_write(
        ctypes.byref(shape), format, kp, vp, ks, _buf(slot_map, _I64, n, dev, "slot_map"), n,
        _buf(n_rows, _I64, 1, dev, "n_rows"),
        _code_pool(k_pages, format, inner, pages, apart, dev, "k_pages"),
        _code_pool(v_pages, format, inner, pages, apart, dev, "v_pages"),
        _buf(k_scale, _F32, blocks, dev, "k_scale"), _buf(v_scale, _F32, blocks, dev, "v_scale"),
        wp, wn, _stream_on(stream, dev))
    if st:
        raise KvError("kv_quant_write", st)


def kv_quant_read(shape: KvPagedShape, format: int, k_pages, v_pages, k_scale, v_scale, slot_map,
                  n_rows, k, v, ws, stream=None) -> None:
    """Rows of a cache in 8 bits as values, into rows ``k`` and ``v`` ([n][heads per page][d], rows
    may lie apart).  ``n_rows`` (a device int64, or None): rows from there on are left out."""
    if _quick is not None:
        st = _quick.kv_quant_read(shape, format, k_pages, v_pages, k_scale, v_scale, slot_map,
                                  n_rows, k, v, ws, stream)
        if st == 0:
            return
        if st is not None:
            raise KvError("kv_quant_read", st)
    dev = _device(k, "k")
    heads, pages = shape.hkv // shape.tables, shape.num_pages
    el, row, inner = _ROWS.get(shape.dtype), heads * shape.d, heads * shape.d * shape.page
    apart, blocks = shape.page_stride or inner, pages * heads * (shape.page // 16)
    kp, n, ks = _rows_view(k, el, row, dev, "k")
    vp, nv, vs = _rows_view(v, el, row, dev, "v")
    if ks != vs or n != nv:
        raise ValueError("k and v must have the same rows and row stride")
    wp, wn = _work(ws, dev)
    st = lib().kv_quant_read(
        ctypes.byref(shape), format,
        _code_pool(k_pages, format, inner, pages, apart, dev, "k_pages"),
        _code_pool(v_pages, format, inner, pages, apart, dev, "v_pages"),
        _buf(k_scale, _F32, blocks, dev, "k_scale"), _buf(v_scale, _F32, blocks, dev, "v_scale"),
        _buf(slot_map, _I64, n, dev, "slot_map"), n, _buf(n_rows, _I64, 1, dev, "n_rows"), kp, vp,
        ks, wp, wn, _stream_on(stream, dev))
    if st:
        raise KvError("kv_quant_read", st)


def quant_decode_attn(shape: KvPagedShape, format: int, q, k_new, v_new, cu_add, slot_map, k_pages,
                      v_pages, k_scale, v_scale, block_table, lens, softmax_scale: float, out, ws,
                      stream=None) -> None:
    """``paged_decode_attn`` over a cache in 8 bits (``kv_quant_write`` has the pools)."""
    if _quick is not None:
        st = _quick.quant_decode_attn(shape, format, q, k_new, v_new, cu_add, slot_map, k_pages,
                                      v_pages, k_scale, v_scale, block_table, lens, softmax_scale,
                                      out, ws, stream)
        if st == 0:
            return
        if st is not None:
            raise KvError("quant_decode_attn", st)
    dev = _device(q, "q")
    el, seqs, hkv, d, tables = _ROWS.get(shape.dtype), shape.seqs, shape.hkv, shape.d, shape.tables
    n, nq, nk, pages = seqs * tables, seqs * shape.hq * d, seqs * hkv * d, shape.num_pages
    heads, page = hkv // tables, shape.page
    inner, blocks = heads * page * d, pages * heads * (page // 16)
    apart = shape.page_stride or inner
    wp, wn = _work(ws, dev)
    st = lib().quant_decode_attn(
        ctypes.byref(shape), format, _buf(q, el, nq, dev, "q"),
        _buf(k_new, el, nk, dev, "k_new"), _buf(v_new, el, nk, dev, "v_new"),
        _buf(cu_add, _I64, n + 1, dev, "cu_add"), _buf(slot_map, _I64, 0, dev, "slot_map"),
        0 if slot_map is None else slot_map.numel(),
        _code_pool(k_pages, format, inner, pages, apart, dev, "k_pages"),
        _code_pool(v_pages, format, inner, pages, apart, dev, "v_pages"),
        _buf(k_scale, _F32, blocks, dev, "k_scale"), _buf(v_scale, _F32, blocks, dev, "v_scale"),
        _buf(block_table, _I32, n * shape.max_pages, dev, "block_table"),
        _buf(lens, _I32, n, dev, "lens"), softmax_scale, _buf(out, el, nq, dev, "out"), wp, wn,
        _stream_on(stream, dev))
    if st:
        raise KvError("quant_decode_attn", st)


def kv_rotary(shape: KvRotaryShape, q, k, positions, inv_freq, q_out, k_out, n_rows=None,
              back: bool = False, stream=None) -> None:
    """Rotary positions of ``q`` ([n][hq][d]) and ``k`` ([n][hkv][d], None for 0 heads), rows may
    lie apart; in place where an output is its input.  ``positions`` int32 (rows below 0 are left
    alone), ``inv_freq`` [rot / 2] float64 on the device (``kv_rotary_inv_freq``).  ``back``:
    turned back, which is the gradient.  ``n_rows`` (a device int64, or None): rows from there on
    are left out."""
    if _quick is not None:
        st = _quick.kv_rotary(shape, q, k, positions, inv_freq, q_out, k_out, n_rows, back, stream)
        if st == 0:
            return
        if st is not None:
            raise KvError("kv_rotary", st)
    dev = _device(positions, "positions")
    el, n, sides = _ROWS.get(shape.dtype), None, []
    for heads, pair in ((shape.hq, ((q, "q"), (q_out, "q_out"))),
                        (shape.hkv, ((k, "k"), (k_out, "k_out")))):
        for t, what in pair:
            if heads == 0:
                sides += (None, 0)
                continue
            p, rows, stride = _rows_view(t, el, heads * shape.d, dev, what)
            if n is not None and rows != n:
                raise ValueError("%s has %d rows, others %d" % (what, rows, n))
            n = rows
            sides += (p, stride)
    n = n or 0
    qp, qs, qop, qos, kp, ks, kop, kos = sides
    st = lib().kv_rotary(
        ctypes.byref(shape), 1 if back else 0, qp, qs, kp, ks,
        _buf(positions, _I32, n, dev, "positions"),
        _buf(inv_freq, _F64, shape.rot // 2, dev, "inv_freq"), n,
        _buf(n_rows, _I64, 1, dev, "n_rows"), qop, qos, kop, kos, _stream_on(stream, dev))
    if st:
        raise KvError("kv_rotary", st)


def kv_check_device_status(ws, stream=None) -> int:
    """Returns 0, or the first device check code recorded in `ws` (and clears it)."""
    info = _u32(0)
    st = lib().kv_check_device_status(_ptr(ws), _stream(stream), ctypes.byref(info))
    if st == KV_ERR_DEVICE_CHECK:
        return int(info.value)
    _check("kv_check_device_status", st)
    return 0


def kv_kernel_launches() -> int:
    """Kernels launched by the library in this process so far."""
    return int(lib().kv_kernel_launches())
