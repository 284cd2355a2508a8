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
import os
from typing import Optional

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
    "KvPagedShape", "kv_paged_workspace_size", "kv_page_map", "kv_paged_write",
    "paged_decode_attn",
]

KV_OK, KV_ERR_INVALID_ARG, KV_ERR_UNSUPPORTED, KV_ERR_WORKSPACE = 0, 1, 2, 3
KV_ERR_CAPACITY, KV_ERR_CUDA, KV_ERR_DEVICE_CHECK = 4, 5, 6
KV_BF16, KV_F32 = 0, 1
KV_SCORE_ADA, KV_SCORE_LAVA, KV_SCORE_CRITICAL = 0, 1, 2
KV_GROUP_MEAN, KV_GROUP_MAX = 0, 1
KV_OP_SCORE, KV_OP_ALLOCATE, KV_OP_COMPACT, KV_OP_DECODE = 0, 1, 2, 3
KV_OP_PAGE_MAP, KV_OP_PAGED_WRITE, KV_OP_PAGED_DECODE = 4, 5, 6
KV_PAGE_MAP_MAX_TABLES = 16384
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


def _need(t, dtype: str, count: int, what: str) -> None:
    """A table's type and the entries the call may touch."""
    if t is not None and not isinstance(t, int):
        if str(t.dtype) != "torch." + dtype:
            raise ValueError("%s must be %s" % (what, dtype))
        if t.numel() < count:
            raise ValueError("%s has %d entries, needs %d" % (what, t.numel(), count))


def _rows_view(t, hp: int, d: int, what: str):
    """Pointer and row stride (elements) of rows [n][hp][d] or [n][hp * d]; a row is contiguous,
    rows may lie apart (parts of a fused projection)."""
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if t.dim() < 2 or t.numel() != t.shape[0] * hp * d:
        raise ValueError("%s must be rows of %d heads x %d" % (what, hp, d))
    step = 1
    for size, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if size > 1 and stride != step:
            raise ValueError("the rows of %s must be contiguous" % what)
        step *= size
    return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else hp * d)


def _pool(shape: KvPagedShape, t, what: str) -> Optional[int]:
    """Pointer of a page pool: its pages are dense, ``page_stride`` elements apart."""
    if t is None or isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if str(t.dtype) != ("torch.bfloat16" if shape.dtype == KV_BF16 else "torch.float32"):
        raise ValueError("%s is not of the shape's dtype" % what)
    inner = (shape.hkv // shape.tables) * shape.page * shape.d
    stride = shape.page_stride or inner
    if t.shape[0] < shape.num_pages or t[0].numel() != inner or not t[0].is_contiguous() or (
            shape.num_pages > 1 and t.stride(0) != stride):
        raise ValueError("%s must be [num_pages][heads][page][d], pages page_stride apart" % what)
    return t.data_ptr()


def kv_page_map(shape: KvPagedShape, lens, add, free_ring, free_state, block_table, lens_out,
                free_out, cu_add, slot_map, ws, stream=None) -> None:
    """Block tables, slots and lengths for the rows each table gains or loses.  ``lens_out`` may
    be ``lens`` and ``free_out`` may be ``free_state``."""
    n = shape.seqs * shape.tables
    _need(lens, "int32", n, "lens")
    _need(add, "int32", n, "add")
    _need(free_ring, "int32", shape.num_pages, "free_ring")
    _need(free_state, "int64", 2, "free_state")
    _need(block_table, "int32", n * shape.max_pages, "block_table")
    _need(lens_out, "int32", n, "lens_out")
    _need(free_out, "int64", 2, "free_out")
    _need(cu_add, "int64", n + 1, "cu_add")
    _need(slot_map, "int64", 0, "slot_map")
    st = lib().kv_page_map(ctypes.byref(shape), _ptr(lens), _ptr(add), _ptr(free_ring),
                           _ptr(free_state), slot_map.numel(), _ptr(block_table), _ptr(lens_out),
                           _ptr(free_out), _ptr(cu_add), _ptr(slot_map), _ptr(ws), _nbytes(ws),
                           _stream(stream))
    _check("kv_page_map", st)


def kv_paged_write(shape: KvPagedShape, k, v, slot_map, n_rows, k_pages, v_pages, ws,
                   stream=None) -> None:
    """Rows of ``k`` and ``v`` ([n][heads per page][d], rows may lie apart) at their slots.
    ``n_rows`` (a device int64, or None): rows from there on are left out."""
    hp = shape.hkv // shape.tables
    kp, ks = _rows_view(k, hp, shape.d, "k")
    vp, vs = _rows_view(v, hp, shape.d, "v")
    if k.dtype != k_pages.dtype or v.dtype != v_pages.dtype:
        raise ValueError("rows and pages must have one dtype")
    if ks != vs or k.shape[0] != v.shape[0]:
        raise ValueError("k and v must have the same rows and row stride")
    _need(slot_map, "int64", k.shape[0], "slot_map")
    _need(n_rows, "int64", 1, "n_rows")
    st = lib().kv_paged_write(ctypes.byref(shape), kp, vp, ks, _ptr(slot_map), k.shape[0],
                              _ptr(n_rows), _pool(shape, k_pages, "k_pages"),
                              _pool(shape, v_pages, "v_pages"), _ptr(ws), _nbytes(ws),
                              _stream(stream))
    _check("kv_paged_write", st)


def paged_decode_attn(shape: KvPagedShape, q, k_new, v_new, cu_add, slot_map, k_pages, v_pages,
                      block_table, lens, softmax_scale: float, out, ws, stream=None) -> None:
    """One decode step over the paged cache; ``k_new`` / ``v_new`` / ``cu_add`` / ``slot_map``
    None: no rows are stored."""
    n = shape.seqs * shape.tables
    _need(block_table, "int32", n * shape.max_pages, "block_table")
    _need(lens, "int32", n, "lens")
    _need(cu_add, "int64", n + 1, "cu_add")
    _need(slot_map, "int64", 0, "slot_map")
    el = "bfloat16" if shape.dtype == KV_BF16 else "float32"
    for t, heads, what in ((q, shape.hq, "q"), (out, shape.hq, "out"), (k_new, shape.hkv, "k_new"),
                           (v_new, shape.hkv, "v_new")):
        _need(t, el, shape.seqs * heads * shape.d, what)
    st = lib().paged_decode_attn(ctypes.byref(shape), _ptr(q), _ptr(k_new), _ptr(v_new),
                                 _ptr(cu_add), _ptr(slot_map),
                                 0 if slot_map is None else slot_map.numel(),
                                 _pool(shape, k_pages, "k_pages"),
                                 _pool(shape, v_pages, "v_pages"), _ptr(block_table), _ptr(lens),
                                 softmax_scale, _ptr(out), _ptr(ws), _nbytes(ws),
                                 _stream(stream))
    _check("paged_decode_attn", st)


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
