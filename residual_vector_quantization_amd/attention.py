"""Streaming attention on MI355X: binding of ``include/rvq_attention.h``.

The same thin layer as the package's quantizer functions: dtypes, devices and layouts are checked, outputs and
workspaces come from ``torch.empty``, raw pointers and the current HIP stream go to ``librvq.so``.

* ``rvq_window_attention(q, k, v, cu_q, cu_k=None, window=None, sinks=0, scale=None)`` -> ``(out, lse)``
* ``rvq_window_attention_backward(dout, q, k, v, out, lse, cu_q, cu_k=None, window=None, sinks=0, scale=None)``
  -> ``(dq, dk, dv)``
* ``rvq_cache_append(k, v, k_pool, v_pool, table, lens, cu=None)``
* ``rvq_cache_attention(q, k_pool, v_pool, table, lens, window=None, sinks=0, scale=None)`` -> ``out``
* ``rvq_cache_reserve(table, lens, new_lens, refs, page_size)`` -> ``(table, refs, missing)``
* ``rvq_cache_fork(table, lens, refs, parents, children, k_pool, v_pool)`` -> ``(table, lens, refs, missing)``
* ``rvq_cache_free(table, lens, refs, page_size, drop=None, window=None, sinks=0)`` -> ``(table, lens, refs)``
* ``rvq_cache_compact(table, refs, k_pool, v_pool)`` -> ``(table, refs, live)``
* ``rvq_cache_copy(src, dst, k_pool, v_pool)``

q, k, v are float32, float16 or bfloat16 [tokens, heads, dim] with dim 64 or 128; rows may be slices of a wider
tensor as long as they start at multiples of 16 bytes. A frame sees the last ``window`` frames up to itself
(``None``: all) and the clip's first ``sinks`` frames. ``scale`` is 1/sqrt(dim) unless given. Pools are
[pages, kv_heads, page_size, dim], or [layers, pages, ...] where pages are moved; they are changed in place,
while tables, lengths and reference counts are returned as new tensors.
"""

from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from . import RVQError, _check, _ptr, _require, _stream, load, rvq_status_string

EXPORTED_ATTENTION = ("rvq_window_attention", "rvq_window_attention_backward", "rvq_window_attention_backward_bytes",
                      "rvq_cache_append", "rvq_cache_attention", "rvq_cache_attention_bytes",
                      "rvq_cache_scratch_bytes", "rvq_cache_reserve", "rvq_cache_fork", "rvq_cache_free",
                      "rvq_cache_compact", "rvq_cache_copy")

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _AttentionShape(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_clips", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("dim", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("window", ctypes.c_int64), ("q_tokens", ctypes.c_int64), ("k_tokens", ctypes.c_int64),
                ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p), ("scale", ctypes.c_float)]


class _CacheShape(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_clips", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("table_ld", ctypes.c_int32)]


_ready = None


def _lib() -> ctypes.CDLL:
    global _ready
    if _ready is not None:
        return _ready
    lib = load()
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    heads, shape, cache = (ctypes.POINTER(t) for t in (_Heads, _AttentionShape, _CacheShape))
    for name, restype, argtypes in (
            ("rvq_window_attention", ctypes.c_int, [shape, heads, heads, heads, heads, vp, vp]),
            ("rvq_window_attention_backward_bytes", i64, [shape]),
            ("rvq_window_attention_backward", ctypes.c_int,
             [shape, heads, heads, heads, heads, heads, vp, heads, heads, heads, vp, i64, vp]),
            ("rvq_cache_append", ctypes.c_int, [cache, heads, heads, i64, vp, vp, vp, vp, vp, vp]),
            ("rvq_cache_attention_bytes", i64, [cache, i32]),
            ("rvq_cache_attention", ctypes.c_int,
             [cache, i32, heads, vp, vp, vp, vp, i64, i32, f32, heads, vp, i64, vp]),
            ("rvq_cache_scratch_bytes", i64, [i32, i32]),
            ("rvq_cache_reserve", ctypes.c_int, [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, i64, vp]),
            ("rvq_cache_fork", ctypes.c_int,
             [cache, i32, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, i64, vp]),
            ("rvq_cache_free", ctypes.c_int, [vp, vp, vp, vp, i32, i32, i32, i32, i64, i32, vp, vp, vp, vp]),
            ("rvq_cache_compact", ctypes.c_int, [cache, i32, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp]),
            ("rvq_cache_copy", ctypes.c_int, [cache, i32, vp, vp, i32, vp, vp, vp])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = restype, argtypes
    _ready = lib
    return lib


def _require_heads(t: torch.Tensor, name: str, dtype: torch.dtype, device, heads: Optional[int] = None,
                   dim: Optional[int] = None, tokens: Optional[int] = None) -> None:
    """A [tokens, heads, dim] tensor with contiguous rows; the C call checks strides and alignment."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim], got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    for what, have, want in (("tokens", t.shape[0], tokens), ("heads", t.shape[1], heads), ("dim", t.shape[2], dim)):
        if want is not None and have != want:
            raise ValueError(f"{name} {tuple(t.shape)} must have {want} {what}")


def _heads(t: torch.Tensor):
    # the stride of a dimension of one entry says nothing
    return ctypes.byref(_Heads(t.data_ptr(), t.stride(0) if t.shape[0] > 1 else 0, t.stride(1) if t.shape[1] > 1 else 0))


def _float_type(t: torch.Tensor, name: str) -> torch.dtype:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in DTYPES:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return t.dtype


def _offsets(cu: torch.Tensor, name: str, device, n_clips: Optional[int] = None) -> None:
    _require(cu, name, torch.int32, 1, device)
    if cu.shape[0] < 1 or (n_clips is not None and cu.shape[0] != n_clips + 1):
        raise ValueError(f"{name} must have one entry more than there are clips, got {cu.shape[0]}")


def _window(window: Optional[int]) -> int:
    if window is None:
        return -1
    if window < 0:
        raise ValueError(f"window={window} must not be negative (None: unbounded)")
    return int(window)


def _attention_shape(q, k, v, cu_q, cu_k, window, sinks, scale):
    dtype = _float_type(q, "q")
    dev = q.device
    _require_heads(q, "q", dtype, dev)
    dim = q.shape[2]
    _require_heads(k, "k", dtype, dev, dim=dim)
    _require_heads(v, "v", dtype, dev, heads=k.shape[1], dim=dim, tokens=k.shape[0])
    if k.shape[1] == 0 or q.shape[1] % k.shape[1] != 0:
        raise ValueError(f"q's heads ({q.shape[1]}) must be a multiple of k's ({k.shape[1]})")
    _offsets(cu_q, "cu_q", dev)
    if cu_k is None:
        if k.shape[0] != q.shape[0]:
            raise ValueError("cu_k is needed where k has other tokens than q")
        cu_k = cu_q
    _offsets(cu_k, "cu_k", dev, cu_q.shape[0] - 1)
    if sinks < 0:
        raise ValueError(f"sinks={sinks} must not be negative")
    return _AttentionShape(DTYPES[dtype], cu_q.shape[0] - 1, q.shape[1], k.shape[1], dim, sinks, _window(window),
                           q.shape[0], k.shape[0], cu_q.data_ptr(), cu_k.data_ptr(),
                           1.0 / math.sqrt(dim) if scale is None else scale)


def rvq_window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                         cu_k: Optional[torch.Tensor] = None, window: Optional[int] = None, sinks: int = 0,
                         scale: Optional[float] = None, out: Optional[torch.Tensor] = None):
    """Windowed attention of packed clips.

    ``q`` [Tq, Hq, D], ``k`` and ``v`` [Tk, Hk, D]; ``cu_q`` / ``cu_k`` int32 [clips + 1] are the clips' first rows
    (``cu_k`` None: the same). A clip's queries stand at the last positions of its keys. Returns
    ``(out [Tq, Hq, D], lse [Hq, Tq] float32)``; ``out`` may be preallocated. Rows outside every clip are not written.
    """
    shape = _attention_shape(q, k, v, cu_q, cu_k, window, sinks, scale)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    _require_heads(out, "out", q.dtype, q.device, q.shape[1], q.shape[2], q.shape[0])
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    st = _lib().rvq_window_attention(ctypes.byref(shape), _heads(q), _heads(k), _heads(v), _heads(out), _ptr(lse),
                                     _stream(q))
    _check("rvq_window_attention", st)
    return out, lse


def rvq_window_attention_backward_bytes(shape: _AttentionShape) -> int:
    """Workspace of the backward pass for a call's shape."""
    size = _lib().rvq_window_attention_backward_bytes(ctypes.byref(shape))
    if size < 0:
        raise RVQError("rvq_window_attention_backward_bytes", size, rvq_status_string(size))
    return size


def rvq_window_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                  out: torch.Tensor, lse: torch.Tensor, cu_q: torch.Tensor,
                                  cu_k: Optional[torch.Tensor] = None, window: Optional[int] = None, sinks: int = 0,
                                  scale: Optional[float] = None, grads=None):
    """Gradients ``(dq, dk, dv)`` of ``rvq_window_attention``; ``out`` and ``lse`` are its results, the other
    arguments as it had them. ``grads`` may pass the three outputs preallocated (for example slices of one tensor)."""
    shape = _attention_shape(q, k, v, cu_q, cu_k, window, sinks, scale)
    for t, name in ((dout, "dout"), (out, "out")):
        _require_heads(t, name, q.dtype, q.device, q.shape[1], q.shape[2], q.shape[0])
    _require(lse, "lse", torch.float32, 2, q.device)
    if tuple(lse.shape) != (q.shape[1], q.shape[0]):
        raise ValueError(f"lse must be [{q.shape[1]}, {q.shape[0]}], got {tuple(lse.shape)}")
    if grads is None:
        grads = tuple(torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
    dq, dk, dv = grads
    for t, name, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
        _require_heads(t, name, q.dtype, q.device, like.shape[1], like.shape[2], like.shape[0])
    work = torch.empty(rvq_window_attention_backward_bytes(shape), dtype=torch.uint8, device=q.device)
    st = _lib().rvq_window_attention_backward(
        ctypes.byref(shape), _heads(dout), _heads(q), _heads(k), _heads(v), _heads(out), _ptr(lse), _heads(dq),
        _heads(dk), _heads(dv), _ptr(work), work.numel(), _stream(q))
    _check("rvq_window_attention_backward", st)
    return dq, dk, dv


def _require_pools(k_pool: torch.Tensor, v_pool: torch.Tensor, dims) -> None:
    _require(k_pool, "k_pool", _float_type(k_pool, "k_pool"), k_pool.dim())
    if k_pool.dim() not in dims:
        raise ValueError(f"k_pool must have {' or '.join(map(str, dims))} dims, got shape {tuple(k_pool.shape)}")
    _require(v_pool, "v_pool", k_pool.dtype, k_pool.dim(), k_pool.device)
    if v_pool.shape != k_pool.shape:
        raise ValueError(f"v_pool {tuple(v_pool.shape)} must match k_pool {tuple(k_pool.shape)}")


def _require_table(table: torch.Tensor, lens: Optional[torch.Tensor], device, refs: Optional[torch.Tensor] = None,
                   n_pages: Optional[int] = None) -> None:
    _require(table, "table", torch.int32, 2, device)
    if lens is not None:
        _require(lens, "lens", torch.int32, 1, device)
        if lens.shape[0] != table.shape[0]:
            raise ValueError(f"lens must have one entry per clip ({table.shape[0]}), got {lens.shape[0]}")
    if refs is not None:
        _require(refs, "refs", torch.int32, 1, device)
        if n_pages is not None and refs.shape[0] != n_pages:
            raise ValueError(f"refs must have one entry per page ({n_pages}), got {refs.shape[0]}")


def _cache_shape(pool: torch.Tensor, table: torch.Tensor) -> _CacheShape:
    pages, heads, size, dim = pool.shape[-4:]
    return _CacheShape(DTYPES[pool.dtype], table.shape[0], heads, dim, size, pages, table.shape[1])


def rvq_cache_append(k: torch.Tensor, v: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                     table: torch.Tensor, lens: torch.Tensor, cu: Optional[torch.Tensor] = None) -> None:
    """Writes new frames ``k``, ``v`` [T, Hk, D] into the pools [P, Hk, page, D]: frame i of clip b (rows ``cu[b]``
    and on; None: one frame a clip) goes to position ``lens[b] + i``. Frames without a page are dropped."""
    _require_pools(k_pool, v_pool, (4,))
    dev = k_pool.device
    _require_heads(k, "k", k_pool.dtype, dev, k_pool.shape[1], k_pool.shape[3])
    _require_heads(v, "v", k_pool.dtype, dev, k_pool.shape[1], k_pool.shape[3], k.shape[0])
    _require_table(table, lens, dev)
    if cu is not None:
        _offsets(cu, "cu", dev, table.shape[0])
    elif k.shape[0] != table.shape[0]:
        raise ValueError("without cu, k must have one frame per clip")
    st = _lib().rvq_cache_append(ctypes.byref(_cache_shape(k_pool, table)), _heads(k), _heads(v), k.shape[0], _ptr(cu),
                                 _ptr(table), _ptr(lens), _ptr(k_pool), _ptr(v_pool), _stream(k_pool))
    _check("rvq_cache_append", st)


def _cache_attention_bytes(shape: _CacheShape, q_heads: int) -> int:
    size = _lib().rvq_cache_attention_bytes(ctypes.byref(shape), q_heads)
    if size < 0:
        raise RVQError("rvq_cache_attention_bytes", size, rvq_status_string(size))
    return size


def rvq_cache_attention_bytes(k_pool: torch.Tensor, table: torch.Tensor, q_heads: int) -> int:
    """Workspace of ``rvq_cache_attention`` for these pools, this table and ``q_heads`` query heads."""
    _require_pools(k_pool, k_pool, (4,))
    _require(table, "table", torch.int32, 2, k_pool.device)
    return _cache_attention_bytes(_cache_shape(k_pool, table), q_heads)


def rvq_cache_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, table: torch.Tensor,
                        lens: torch.Tensor, window: Optional[int] = None, sinks: int = 0,
                        scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of every clip's newest frame ``q`` [clips, Hq, D] over its cache; ``lens`` counts that frame, whose
    key and value have been appended. ``out`` and ``workspace`` (uint8, ``rvq_cache_attention_bytes``) may be
    preallocated."""
    _require_pools(k_pool, v_pool, (4,))
    dev = k_pool.device
    _require_table(table, lens, dev)
    _require_heads(q, "q", k_pool.dtype, dev, dim=k_pool.shape[3], tokens=table.shape[0])
    if k_pool.shape[1] == 0 or q.shape[1] % k_pool.shape[1] != 0:
        raise ValueError(f"q's heads ({q.shape[1]}) must be a multiple of the pools' ({k_pool.shape[1]})")
    if sinks < 0:
        raise ValueError(f"sinks={sinks} must not be negative")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    _require_heads(out, "out", q.dtype, dev, q.shape[1], q.shape[2], q.shape[0])
    shape = _cache_shape(k_pool, table)
    size = _cache_attention_bytes(shape, q.shape[1])
    if workspace is None:
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    _require(workspace, "workspace", torch.uint8, 1, dev)
    st = _lib().rvq_cache_attention(ctypes.byref(shape), q.shape[1], _heads(q), _ptr(k_pool), _ptr(v_pool),
                                    _ptr(table), _ptr(lens), _window(window), sinks,
                                    1.0 / math.sqrt(q.shape[2]) if scale is None else scale, _heads(out),
                                    _ptr(workspace), workspace.numel(), _stream(k_pool))
    _check("rvq_cache_attention", st)
    return out


def rvq_cache_scratch_bytes(n_clips: int, n_pages: int) -> int:
    """Workspace of reserve, fork and compact."""
    size = _lib().rvq_cache_scratch_bytes(n_clips, n_pages)
    if size < 0:
        raise RVQError("rvq_cache_scratch_bytes", size, rvq_status_string(size))
    return size


def _scratch(table: torch.Tensor, refs: torch.Tensor) -> torch.Tensor:
    return torch.empty(rvq_cache_scratch_bytes(table.shape[0], refs.shape[0]), dtype=torch.uint8, device=table.device)


def rvq_cache_reserve(table: torch.Tensor, lens: torch.Tensor, new_lens: torch.Tensor, refs: torch.Tensor,
                      page_size: int):
    """Gives every clip the pages for positions ``lens[b]`` .. ``new_lens[b] - 1``, lowest free pages first.

    ``table`` [clips, E], ``lens``, ``new_lens`` [clips], ``refs`` [pages], all int32. Returns ``(table, refs,
    missing [1])``; ``missing`` counts the pages that were not there (their entries stay -1).
    """
    _require_table(table, lens, table.device, refs)
    _require(new_lens, "new_lens", torch.int32, 1, table.device)
    if new_lens.shape != lens.shape:
        raise ValueError("new_lens must match lens")
    table_out, refs_out = torch.empty_like(table), torch.empty_like(refs)
    missing, work = torch.empty(1, dtype=torch.int32, device=table.device), _scratch(table, refs)
    st = _lib().rvq_cache_reserve(_ptr(table), _ptr(lens), _ptr(new_lens), _ptr(refs), table.shape[0], table.shape[1],
                                  page_size, refs.shape[0], _ptr(table_out), _ptr(refs_out), _ptr(missing),
                                  _ptr(work), work.numel(), _stream(table))
    _check("rvq_cache_reserve", st)
    return table_out, refs_out, missing


def _layers(pool: torch.Tensor) -> int:
    return pool.shape[0] if pool.dim() == 5 else 1


def rvq_cache_fork(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, parents: torch.Tensor,
                   children: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor):
    """Lets clips ``children[c]`` go on from clips ``parents[c]`` (int32, children distinct): full pages are shared,
    a partial page is copied into a free one in the pools [(layers,) pages, Hk, page, D].

    Returns ``(table, lens, refs, missing [1])``.
    """
    _require_pools(k_pool, v_pool, (4, 5))
    dev = k_pool.device
    _require_table(table, lens, dev, refs, k_pool.shape[-4])
    _require(parents, "parents", torch.int32, 1, dev)
    _require(children, "children", torch.int32, 1, dev)
    if parents.shape != children.shape or children.shape[0] > table.shape[0]:
        raise ValueError("parents and children must match and be no more than there are clips")
    table_out, lens_out, refs_out = torch.empty_like(table), torch.empty_like(lens), torch.empty_like(refs)
    missing, work = torch.empty(1, dtype=torch.int32, device=dev), _scratch(table, refs)
    st = _lib().rvq_cache_fork(ctypes.byref(_cache_shape(k_pool, table)), _layers(k_pool), _ptr(table), _ptr(lens),
                               _ptr(refs), _ptr(parents), _ptr(children), children.shape[0], _ptr(k_pool),
                               _ptr(v_pool), _ptr(table_out), _ptr(lens_out), _ptr(refs_out), _ptr(missing),
                               _ptr(work), work.numel(), _stream(k_pool))
    _check("rvq_cache_fork", st)
    return table_out, lens_out, refs_out, missing


def rvq_cache_free(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_size: int,
                   drop: Optional[torch.Tensor] = None, window: Optional[int] = None, sinks: int = 0):
    """Lets go of all pages of the clips with ``drop`` [clips] int32 not 0, and with a ``window`` of the other clips'
    pages that no later frame sees. Returns ``(table, lens, refs)``."""
    _require_table(table, lens, table.device, refs)
    if drop is not None:
        _require(drop, "drop", torch.int32, 1, table.device)
        if drop.shape != lens.shape:
            raise ValueError("drop must match lens")
    if sinks < 0:
        raise ValueError(f"sinks={sinks} must not be negative")
    table_out, lens_out, refs_out = torch.empty_like(table), torch.empty_like(lens), torch.empty_like(refs)
    st = _lib().rvq_cache_free(_ptr(table), _ptr(lens), _ptr(refs), _ptr(drop), table.shape[0], table.shape[1],
                               page_size, refs.shape[0], _window(window), sinks, _ptr(table_out), _ptr(lens_out),
                               _ptr(refs_out), _stream(table))
    _check("rvq_cache_free", st)
    return table_out, lens_out, refs_out


def rvq_cache_compact(table: torch.Tensor, refs: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor):
    """Moves the pages in use to the numbers 0 .. live - 1. Returns ``(table, refs, live [1])``."""
    _require_pools(k_pool, v_pool, (4, 5))
    dev = k_pool.device
    _require_table(table, None, dev, refs, k_pool.shape[-4])
    table_out, refs_out = torch.empty_like(table), torch.empty_like(refs)
    live, work = torch.empty(1, dtype=torch.int32, device=dev), _scratch(table, refs)
    st = _lib().rvq_cache_compact(ctypes.byref(_cache_shape(k_pool, table)), _layers(k_pool), _ptr(table), _ptr(refs),
                                  _ptr(k_pool), _ptr(v_pool), _ptr(table_out), _ptr(refs_out), _ptr(live),
                                  _ptr(work), work.numel(), _stream(k_pool))
    _check("rvq_cache_compact", st)
    return table_out, refs_out, live


def rvq_cache_copy(src: torch.Tensor, dst: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor) -> None:
    """Copies page ``src[i]`` to page ``dst[i]`` (int32) in every layer of both pools."""
    _require_pools(k_pool, v_pool, (4, 5))
    _require(src, "src", torch.int32, 1, k_pool.device)
    _require(dst, "dst", torch.int32, 1, k_pool.device)
    if src.shape != dst.shape:
        raise ValueError("src and dst must match")
    shape = _cache_shape(k_pool, dst[:, None])
    shape.n_clips, shape.table_ld = 0, 0
    st = _lib().rvq_cache_copy(ctypes.byref(shape), _layers(k_pool), _ptr(src), _ptr(dst), src.shape[0], _ptr(k_pool),
                               _ptr(v_pool), _stream(k_pool))
    _check("rvq_cache_copy", st)
