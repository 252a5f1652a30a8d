"""Streaming attention on MI355X: binding of ``include/rvq_attention.h``.

The same thin layer as the package's quantizer functions: dtypes, devices and layouts are checked, outputs and
workspaces come from ``torch.empty``, raw pointers and the current HIP stream go to ``librvq.so``.

* ``rvq_window_attention(q, k, v, cu_q, cu_k=None, window=None, sinks=0, scale=None)`` -> ``(out, lse)``
* ``rvq_window_attention_backward(dout, q, k, v, out, lse, cu_q, cu_k=None, window=None, sinks=0, scale=None)``
  -> ``(dq, dk, dv)``
* ``rvq_cross_attention(q, k, v, cu_q, cu_k, scale=None)`` -> ``(out, lse)``
* ``rvq_cross_attention_backward(dout, q, k, v, out, lse, cu_q, cu_k, scale=None)`` -> ``(dq, dk, dv)``
* ``rvq_cache_append(k, v, k_pool, v_pool, table, lens, cu=None)``
* ``rvq_cache_attention(q, k_pool, v_pool, table, lens, window=None, sinks=0, scale=None)`` -> ``out``
* ``rvq_cache_chunk_attention(q, k_pool, v_pool, table, lens, cu=None, window=None, sinks=0, scale=None)``
  -> ``(out, lse)``
* ``rvq_rotary_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, context=0, slow=1.0, fast=32.0)``
  -> float64 CPU tensor
* ``rvq_rotary(q, k, frequencies, cu=None, first=None, positions=None, interleaved=False, amplitude=1.0,
  inverse=False)`` -> ``(q, k)``
* ``rvq_rotary_append(q, k, v, frequencies, k_pool, v_pool, table, lens, cu=None, interleaved=False, amplitude=1.0)``
  -> ``q``
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
import struct
from typing import Optional

import torch

from . import RVQError, _check, _ptr, _require, load, rvq_status_string

EXPORTED_ATTENTION = ("rvq_window_attention", "rvq_window_attention_backward", "rvq_window_attention_backward_bytes",
                      "rvq_cache_append", "rvq_cache_attention", "rvq_cache_attention_bytes",
                      "rvq_cache_scratch_bytes", "rvq_cache_reserve", "rvq_cache_fork", "rvq_cache_free",
                      "rvq_cache_compact", "rvq_cache_copy", "rvq_rotary_frequencies", "rvq_rotary",
                      "rvq_rotary_append", "rvq_cache_chunk_attention", "rvq_cache_chunk_attention_bytes",
                      "rvq_cross_attention", "rvq_cross_attention_bytes", "rvq_cross_attention_backward",
                      "rvq_cross_attention_backward_bytes")

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
SCALINGS = {None: 0, "linear": 1, "base": 2, "ramp": 3}


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


class _Rotation(ctypes.Structure):
    _fields_ = [("frequencies", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("inverse", ctypes.c_int32), ("amplitude", ctypes.c_float)]


# The same structures packed by hand: a tenth of the time of a ctypes.Structure, which counts where a call takes 10 us.
_pack_heads = struct.Struct("=Qqq").pack
_pack_attention = struct.Struct("=6i3qQQf4x").pack
_pack_cache = struct.Struct("=7i").pack
_pack_rotation = struct.Struct("=Q3if").pack

_ready = None


def _lib() -> ctypes.CDLL:
    global _ready
    if _ready is not None:
        return _ready
    lib = load()
    vp, i32, i64, f32, f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double
    heads = shape = cache = vp      # packed bytes or a pointer to the structure
    for name, restype, argtypes in (
            ("rvq_window_attention", ctypes.c_int, [shape, heads, heads, heads, heads, vp, vp]),
            ("rvq_window_attention_backward_bytes", i64, [shape]),
            ("rvq_window_attention_backward", ctypes.c_int,
             [shape, heads, heads, heads, heads, heads, vp, heads, heads, heads, vp, i64, vp]),
            ("rvq_cross_attention_bytes", i64, [shape]),
            ("rvq_cross_attention", ctypes.c_int, [shape, heads, heads, heads, heads, vp, vp, i64, vp]),
            ("rvq_cross_attention_backward_bytes", i64, [shape]),
            ("rvq_cross_attention_backward", ctypes.c_int,
             [shape, heads, heads, heads, heads, heads, vp, heads, heads, heads, vp, i64, vp]),
            ("rvq_cache_append", ctypes.c_int, [cache, heads, heads, i64, vp, vp, vp, vp, vp, vp]),
            ("rvq_cache_attention_bytes", i64, [cache, i32]),
            ("rvq_cache_attention", ctypes.c_int,
             [cache, i32, heads, vp, vp, vp, vp, i64, i32, f32, heads, vp, i64, vp]),
            ("rvq_cache_chunk_attention_bytes", i64, [cache, i32, i64]),
            ("rvq_cache_chunk_attention", ctypes.c_int,
             [cache, i32, i64, vp, heads, vp, vp, vp, vp, i64, i32, f32, heads, vp, vp, i64, vp]),
            ("rvq_rotary_frequencies", ctypes.c_int, [i32, f64, i32, f64, f64, f64, f64, vp]),
            ("rvq_rotary", ctypes.c_int,
             [vp, i32, i64, i32, i32, i32, i32, vp, vp, vp, heads, heads, heads, heads, vp]),
            ("rvq_rotary_append", ctypes.c_int,
             [cache, vp, i32, heads, heads, heads, i64, vp, vp, vp, heads, vp, vp, vp]),
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


def _stream(t: torch.Tensor) -> int:
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _launch(name: str, device: torch.device, *args) -> None:
    """The call on the tensors' own device: a default stream is that of the device that is current."""
    if torch._C._cuda_getDevice() == device.index:
        st = getattr(_ready or _lib(), name)(*args)
    else:
        with torch.cuda.device(device):
            st = getattr(_ready or _lib(), name)(*args)
    if st:
        _check(name, st)


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _new_heads(like: torch.Tensor, tokens: int, heads: int, dim: int):
    """A new [tokens, heads, dim] tensor, and it as the C structure."""
    t = like.new_empty((tokens, heads, dim))
    return t, _pack_heads(t.data_ptr(), heads * dim if tokens > 1 else 0, dim if heads > 1 else 0)


def _require_heads(t: torch.Tensor, name: str, dtype: torch.dtype, device, heads: Optional[int] = None,
                   dim: Optional[int] = None, tokens: Optional[int] = None) -> bytes:
    """A [tokens, heads, dim] tensor with contiguous rows, as the C structure; the C call checks strides and
    alignment."""
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
    (n, h, d), (n_stride, h_stride, d_stride) = t.shape, t.stride()
    if d_stride != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if (heads is not None and h != heads) or (dim is not None and d != dim) or (tokens is not None and n != tokens):
        want = ", ".join("*" if x is None else str(x) for x in (tokens, heads, dim))
        raise ValueError(f"{name} must be [{want}], got {tuple(t.shape)}")
    # the stride of a dimension of one entry says nothing
    return _pack_heads(t.data_ptr(), n_stride if n > 1 else 0, h_stride if h > 1 else 0)


def _float_type(t: torch.Tensor, name: str) -> torch.dtype:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in DTYPES:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return t.dtype


def _offsets(cu: torch.Tensor, name: str, device, n_clips: Optional[int] = None) -> int:
    _require(cu, name, torch.int32, 1, device)
    n = cu.shape[0] - 1
    if n < 0 or (n_clips is not None and n != n_clips):
        raise ValueError(f"{name} must have one entry more than there are clips, got {n + 1}")
    return n


def _window(window: Optional[int]) -> int:
    if window is None:
        return -1
    if window < 0:
        raise ValueError(f"window={window} must not be negative (None: unbounded)")
    return int(window)


def _attention_args(q, k, v, cu_q, cu_k, window, sinks, scale):
    """The checked call: (shape, q, k, v) as C structures, and q's sizes."""
    dtype, dev = _float_type(q, "q"), q.device
    q_heads = _require_heads(q, "q", dtype, dev)
    tq, hq, dim = q.shape
    k_heads = _require_heads(k, "k", dtype, dev, dim=dim)
    tk, hk, _ = k.shape
    v_heads = _require_heads(v, "v", dtype, dev, hk, dim, tk)
    if hk == 0 or hq % hk != 0:
        raise ValueError(f"q's heads ({hq}) must be a multiple of k's ({hk})")
    n = _offsets(cu_q, "cu_q", dev)
    if cu_k is None:
        if tk != tq:
            raise ValueError("cu_k is needed where k has other tokens than q")
        cu_k = cu_q
    elif cu_k is not cu_q:
        _offsets(cu_k, "cu_k", dev, n)
    if sinks < 0:
        raise ValueError(f"sinks={sinks} must not be negative")
    shape = _pack_attention(DTYPES[dtype], n, hq, hk, dim, sinks, _window(window), tq, tk, cu_q.data_ptr(),
                            cu_k.data_ptr(), 1.0 / math.sqrt(dim) if scale is None else scale)
    return shape, q_heads, k_heads, v_heads, (tq, hq, dim)


def rvq_window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                         cu_k: Optional[torch.Tensor] = None, window: Optional[int] = None, sinks: int = 0,
                         scale: Optional[float] = None, out: Optional[torch.Tensor] = None):
    """Windowed attention of packed clips.

    ``q`` [Tq, Hq, D], ``k`` and ``v`` [Tk, Hk, D]; ``cu_q`` / ``cu_k`` int32 [clips + 1] are the clips' first rows
    (``cu_k`` None: the same). A clip's queries stand at the last positions of its keys. Returns
    ``(out [Tq, Hq, D], lse [Hq, Tq] float32)``; ``out`` may be preallocated. Rows outside every clip are not written.
    """
    shape, q_heads, k_heads, v_heads, size = _attention_args(q, k, v, cu_q, cu_k, window, sinks, scale)
    if out is None:
        out = q.new_empty(size)
    out_heads = _require_heads(out, "out", q.dtype, q.device, size[1], size[2], size[0])
    lse = q.new_empty((size[1], size[0]), dtype=torch.float32)
    _launch("rvq_window_attention", q.device, shape, q_heads, k_heads, v_heads, out_heads, lse.data_ptr(), _stream(q))
    return out, lse


def _size(name: str, *args) -> int:
    size = getattr(_lib(), name)(*args)
    if size < 0:
        raise RVQError(name, size, rvq_status_string(size))
    return size


def rvq_window_attention_backward_bytes(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                                        cu_k: Optional[torch.Tensor] = None, window: Optional[int] = None,
                                        sinks: int = 0) -> int:
    """Workspace of ``rvq_window_attention_backward`` for these arguments."""
    return _size("rvq_window_attention_backward_bytes", _attention_args(q, k, v, cu_q, cu_k, window, sinks, None)[0])


def rvq_window_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                  out: torch.Tensor, lse: torch.Tensor, cu_q: torch.Tensor,
                                  cu_k: Optional[torch.Tensor] = None, window: Optional[int] = None, sinks: int = 0,
                                  scale: Optional[float] = None, grads=None,
                                  workspace: Optional[torch.Tensor] = None):
    """Gradients ``(dq, dk, dv)`` of ``rvq_window_attention``; ``out`` and ``lse`` are its results, the other
    arguments as it had them. ``grads`` may pass the three outputs preallocated (for example slices of one tensor),
    ``workspace`` a uint8 tensor of ``rvq_window_attention_backward_bytes``."""
    shape, q_heads, k_heads, v_heads, _ = _attention_args(q, k, v, cu_q, cu_k, window, sinks, scale)
    return _backward("rvq_window_attention_backward", shape, dout, (q, k, v), (q_heads, k_heads, v_heads), out, lse, grads,
                     workspace)


def _backward(name, shape, dout, inputs, input_heads, out, lse, grads, workspace):
    (q, k, v), (q_heads, k_heads, v_heads) = inputs, input_heads
    tq, hq, dim = q.shape
    dtype, dev = q.dtype, q.device
    dout_heads = _require_heads(dout, "dout", dtype, dev, hq, dim, tq)
    out_heads = _require_heads(out, "out", dtype, dev, hq, dim, tq)
    _require(lse, "lse", torch.float32, 2, dev)
    if lse.shape != (hq, tq):
        raise ValueError(f"lse must be [{hq}, {tq}], got {tuple(lse.shape)}")
    if grads is None:
        grads = tuple(t.new_empty(t.shape) for t in (q, k, v))
    dq, dk, dv = grads
    tk, hk, _ = k.shape
    dq_heads = _require_heads(dq, "dq", dtype, dev, hq, dim, tq)
    dk_heads = _require_heads(dk, "dk", dtype, dev, hk, dim, tk)
    dv_heads = _require_heads(dv, "dv", dtype, dev, hk, dim, tk)
    if workspace is None:
        workspace = q.new_empty(_size(name + "_bytes", shape), dtype=torch.uint8)
    _require(workspace, "workspace", torch.uint8, 1, dev)
    _launch(name, dev, shape, dout_heads, q_heads, k_heads, v_heads, out_heads, lse.data_ptr(), dq_heads, dk_heads,
            dv_heads, workspace.data_ptr(), workspace.numel(), _stream(q))
    return dq, dk, dv


def _workspace(given: Optional[torch.Tensor], like: torch.Tensor, name: str, *args):
    """The workspace that was given, or a new one where the operator needs any; and its size."""
    if given is not None:
        _require(given, "workspace", torch.uint8, 1, like.device)
        return given, given.numel()
    size = _size(name, *args)
    return (like.new_empty(size, dtype=torch.uint8) if size else None), size


def _cross_args(q, k, v, cu_q, cu_k, scale):
    """The checked call: (shape, q, k, v) as C structures, and q's sizes."""
    dtype, dev = _float_type(q, "q"), q.device
    q_heads = _require_heads(q, "q", dtype, dev)
    tq, hq, dim = q.shape
    k_heads = _require_heads(k, "k", dtype, dev, dim=dim)
    tk, hk, _ = k.shape
    v_heads = _require_heads(v, "v", dtype, dev, hk, dim, tk)
    if hk == 0 or hq % hk != 0:
        raise ValueError(f"q's heads ({hq}) must be a multiple of k's ({hk})")
    n = _offsets(cu_k, "cu_k", dev)
    if cu_q is not None:
        _offsets(cu_q, "cu_q", dev, n)
    elif tq != n:
        raise ValueError("without cu_q, q must have one row per clip")
    shape = _pack_attention(DTYPES[dtype], n, hq, hk, dim, 0, -1, tq, tk, 0 if cu_q is None else cu_q.data_ptr(),
                            cu_k.data_ptr(), 1.0 / math.sqrt(dim) if scale is None else scale)
    return shape, q_heads, k_heads, v_heads, (tq, hq, dim)


def rvq_cross_attention_bytes(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: Optional[torch.Tensor],
                              cu_k: torch.Tensor) -> int:
    """Workspace of ``rvq_cross_attention`` for these arguments."""
    return _size("rvq_cross_attention_bytes", _cross_args(q, k, v, cu_q, cu_k, None)[0])


def rvq_cross_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: Optional[torch.Tensor],
                        cu_k: torch.Tensor, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None):
    """Attention of packed clips' queries to all of their clips' keys.

    ``q`` [Tq, Hq, D], ``k`` and ``v`` [Tk, Hk, D]; ``cu_q`` / ``cu_k`` int32 [clips + 1] are the clips' first rows
    (``cu_q`` None: one query a clip). Returns ``(out [Tq, Hq, D], lse [Hq, Tq] float32)``, 0 and -inf for a clip
    without keys. ``out`` and ``workspace`` (uint8, ``rvq_cross_attention_bytes``) may be preallocated. Rows outside
    every clip are not written.
    """
    shape, q_heads, k_heads, v_heads, size = _cross_args(q, k, v, cu_q, cu_k, scale)
    dev = q.device
    if out is None:
        out, out_heads = _new_heads(q, *size)
    else:
        out_heads = _require_heads(out, "out", q.dtype, dev, size[1], size[2], size[0])
    lse = q.new_empty((size[1], size[0]), dtype=torch.float32)
    work, work_bytes = _workspace(workspace, q, "rvq_cross_attention_bytes", shape)
    _launch("rvq_cross_attention", dev, shape, q_heads, k_heads, v_heads, out_heads, lse.data_ptr(), _at(work), work_bytes,
            _stream(q))
    return out, lse


def rvq_cross_attention_backward_bytes(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                                       cu_k: torch.Tensor) -> int:
    """Workspace of ``rvq_cross_attention_backward`` for these arguments."""
    return _size("rvq_cross_attention_backward_bytes", _cross_args(q, k, v, cu_q, cu_k, None)[0])


def rvq_cross_attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                 out: torch.Tensor, lse: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
                                 scale: Optional[float] = None, grads=None, workspace: Optional[torch.Tensor] = None):
    """Gradients ``(dq, dk, dv)`` of ``rvq_cross_attention``, as ``rvq_window_attention_backward``; ``cu_q`` must be
    given (``torch.arange(clips + 1)`` for one query a clip)."""
    if cu_q is None:
        raise ValueError("the gradient needs cu_q")
    shape, q_heads, k_heads, v_heads, _ = _cross_args(q, k, v, cu_q, cu_k, scale)
    return _backward("rvq_cross_attention_backward", shape, dout, (q, k, v), (q_heads, k_heads, v_heads), out, lse, grads,
                     workspace)


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


def _cache_shape(pool: torch.Tensor, n_clips: int, table_ld: int) -> bytes:
    pages, heads, size, dim = pool.shape[-4:]
    return _pack_cache(DTYPES[pool.dtype], n_clips, heads, dim, size, pages, table_ld)


def rvq_cache_append(k: torch.Tensor, v: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                     table: torch.Tensor, lens: torch.Tensor, cu: Optional[torch.Tensor] = None) -> None:
    """Writes new frames ``k``, ``v`` [T, Hk, D] into the pools [P, Hk, page, D]: frame i of clip b (rows ``cu[b]``
    and on; None: one frame a clip) goes to position ``lens[b] + i``. Frames without a page are dropped."""
    _require_pools(k_pool, v_pool, (4,))
    dev = k_pool.device
    _, heads, _, dim = k_pool.shape
    k_heads = _require_heads(k, "k", k_pool.dtype, dev, heads, dim)
    n = k.shape[0]
    v_heads = _require_heads(v, "v", k_pool.dtype, dev, heads, dim, n)
    _require_table(table, lens, dev)
    clips, cols = table.shape
    if cu is not None:
        _offsets(cu, "cu", dev, clips)
    elif n != clips:
        raise ValueError("without cu, k must have one frame per clip")
    _launch("rvq_cache_append", dev, _cache_shape(k_pool, clips, cols), k_heads, v_heads, n, _ptr(cu),
            table.data_ptr(), lens.data_ptr(), k_pool.data_ptr(), v_pool.data_ptr(), _stream(k_pool))


def _cache_attention_bytes(shape: bytes, q_heads: int) -> int:
    size = _lib().rvq_cache_attention_bytes(shape, q_heads)
    if size < 0:
        raise RVQError("rvq_cache_attention_bytes", size, rvq_status_string(size))
    return size


def rvq_cache_attention_bytes(k_pool: torch.Tensor, table: torch.Tensor, q_heads: int) -> int:
    """Workspace of ``rvq_cache_attention`` for these pools, this table and ``q_heads`` query heads."""
    _require_pools(k_pool, k_pool, (4,))
    _require(table, "table", torch.int32, 2, k_pool.device)
    return _cache_attention_bytes(_cache_shape(k_pool, *table.shape), q_heads)


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
    clips, cols = table.shape
    _, heads, _, dim = k_pool.shape
    q_heads = _require_heads(q, "q", k_pool.dtype, dev, dim=dim, tokens=clips)
    hq = q.shape[1]
    if heads == 0 or hq % heads != 0:
        raise ValueError(f"q's heads ({hq}) must be a multiple of the pools' ({heads})")
    if sinks < 0:
        raise ValueError(f"sinks={sinks} must not be negative")
    if out is None:
        out = q.new_empty((clips, hq, dim))
    out_heads = _require_heads(out, "out", q.dtype, dev, hq, dim, clips)
    shape = _cache_shape(k_pool, clips, cols)
    if workspace is None:
        workspace = q.new_empty(_cache_attention_bytes(shape, hq), dtype=torch.uint8)
    _require(workspace, "workspace", torch.uint8, 1, dev)
    _launch("rvq_cache_attention", dev, shape, hq, q_heads, k_pool.data_ptr(), v_pool.data_ptr(), table.data_ptr(),
            lens.data_ptr(), _window(window), sinks, 1.0 / math.sqrt(dim) if scale is None else scale, out_heads,
            workspace.data_ptr(), workspace.numel(), _stream(k_pool))
    return out


def rvq_cache_chunk_attention_bytes(k_pool: torch.Tensor, table: torch.Tensor, q_heads: int, tokens: int) -> int:
    """Workspace of ``rvq_cache_chunk_attention`` for these pools, this table and ``tokens`` rows of ``q_heads`` heads."""
    _require_pools(k_pool, k_pool, (4,))
    _require(table, "table", torch.int32, 2, k_pool.device)
    return _size("rvq_cache_chunk_attention_bytes", _cache_shape(k_pool, *table.shape), q_heads, tokens)


def rvq_cache_chunk_attention(q: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor, table: torch.Tensor,
                              lens: torch.Tensor, cu: Optional[torch.Tensor] = None, window: Optional[int] = None,
                              sinks: int = 0, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None):
    """Attention of every clip's newest frames ``q`` [T, Hq, D] over its cache.

    Clip b's queries are rows ``cu[b]`` and on (int32 [clips + 1]; None: one a clip), the last ones of the ``lens[b]``
    frames that its cache holds; their keys and values have been appended. Returns ``(out [T, Hq, D],
    lse [Hq, T] float32)``. ``out`` and ``workspace`` (uint8, ``rvq_cache_chunk_attention_bytes``) may be preallocated.
    Rows outside every clip are not written.
    """
    _require_pools(k_pool, v_pool, (4,))
    dev = k_pool.device
    _require_table(table, lens, dev)
    clips, cols = table.shape
    _, heads, _, dim = k_pool.shape
    q_heads = _require_heads(q, "q", k_pool.dtype, dev, dim=dim)
    n, hq, _ = q.shape
    if cu is not None:
        _offsets(cu, "cu", dev, clips)
    elif n != clips:
        raise ValueError("without cu, q must have one frame per clip")
    if heads == 0 or hq % heads != 0:
        raise ValueError(f"q's heads ({hq}) must be a multiple of the pools' ({heads})")
    if sinks < 0:
        raise ValueError(f"sinks={sinks} must not be negative")
    if out is None:
        out, out_heads = _new_heads(q, n, hq, dim)
    else:
        out_heads = _require_heads(out, "out", q.dtype, dev, hq, dim, n)
    lse = q.new_empty((hq, n), dtype=torch.float32)
    shape = _cache_shape(k_pool, clips, cols)
    work, work_bytes = _workspace(workspace, q, "rvq_cache_chunk_attention_bytes", shape, hq, n)
    _launch("rvq_cache_chunk_attention", dev, shape, hq, n, _at(cu), q_heads, k_pool.data_ptr(), v_pool.data_ptr(),
            table.data_ptr(), lens.data_ptr(), _window(window), sinks, 1.0 / math.sqrt(dim) if scale is None else scale,
            out_heads, lse.data_ptr(), _at(work), work_bytes, _stream(k_pool))
    return out, lse


def rvq_rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                           context: float = 0.0, slow: float = 1.0, fast: float = 32.0) -> torch.Tensor:
    """Radians a position of the ``rot_dim / 2`` pairs, float64 on the CPU: ``base^(-2 i / rot_dim)``.

    ``scaling`` stretches them for clips ``factor`` times longer: "linear" divides all by ``factor``; "base" raises
    the base so that the slowest one is divided by it; "ramp" keeps those that turn ``fast`` times or more within
    ``context`` positions and divides those that turn ``slow`` times or less.
    """
    if scaling not in SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(map(repr, SCALINGS))}, got {scaling!r}")
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim={rot_dim} must be even and at least 2")
    out = torch.empty(rot_dim // 2, dtype=torch.float64)
    st = _lib().rvq_rotary_frequencies(rot_dim, base, SCALINGS[scaling], factor, context, slow, fast, out.data_ptr())
    _check("rvq_rotary_frequencies", st)
    return out


def _rotation(frequencies: torch.Tensor, interleaved: bool, inverse: bool, amplitude: float, device, dim: int) -> bytes:
    _require(frequencies, "frequencies", torch.float64, 1, device)
    n = frequencies.shape[0]
    if not 0 < 2 * n <= dim:
        raise ValueError(f"frequencies must have 1 to {dim // 2} entries, got {n}")
    return _pack_rotation(frequencies.data_ptr(), 2 * n, interleaved, inverse, amplitude)


def rvq_rotary(q: Optional[torch.Tensor], k: Optional[torch.Tensor], frequencies: torch.Tensor,
               cu: Optional[torch.Tensor] = None, first: Optional[torch.Tensor] = None,
               positions: Optional[torch.Tensor] = None, interleaved: bool = False, amplitude: float = 1.0,
               inverse: bool = False, out=None):
    """Rotary positions of packed queries ``q`` [T, Hq, D] and keys ``k`` [T, Hk, D] (either may be None).

    ``frequencies`` float64 [n]: the first 2 n values of every head turn, in pairs of (i, n + i), or of neighbours
    where ``interleaved``; turned values are scaled by ``amplitude``. Positions are ``positions`` int32 [T], or
    ``first[b] + i`` for frame i of clip b (``cu`` int32 [clips + 1]; ``first`` int32 [clips], None: 0); rows outside
    every clip are not written. ``inverse`` turns backwards: gradients of the results give those of ``q`` and ``k``.
    ``out`` may pass the two outputs preallocated; they may be ``q`` and ``k`` themselves. Returns ``(q_out, k_out)``.
    """
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k must be given")
    dtype, dev = _float_type(x, "q" if q is not None else "k"), x.device
    x_heads = _require_heads(x, "q" if q is not None else "k", dtype, dev)
    tokens, _, dim = x.shape
    if q is not None and k is not None:
        k_heads = _require_heads(k, "k", dtype, dev, dim=dim, tokens=tokens)
    else:
        k_heads = x_heads
    rotation = _rotation(frequencies, interleaved, inverse, amplitude, dev, dim)
    clips = 0
    if positions is not None:
        if cu is not None or first is not None:
            raise ValueError("positions, or cu and first")
        _require(positions, "positions", torch.int32, 1, dev)
        if positions.shape[0] != tokens:
            raise ValueError(f"positions must have one entry per row ({tokens}), got {positions.shape[0]}")
    else:
        if cu is None:
            raise ValueError("positions or cu must be given")
        clips = _offsets(cu, "cu", dev)
        if first is not None:
            _require(first, "first", torch.int32, 1, dev)
            if first.shape[0] != clips:
                raise ValueError(f"first must have one entry per clip ({clips}), got {first.shape[0]}")
    q_out, k_out = (None, None) if out is None else out
    hq = hk = 0
    q_to = k_to = None
    if q is not None:
        hq = q.shape[1]
        if q_out is None:
            q_out, q_to = _new_heads(q, tokens, hq, dim)
        else:
            q_to = x_heads if q_out is q else _require_heads(q_out, "q_out", dtype, dev, hq, dim, tokens)
    if k is not None:
        hk = k.shape[1]
        if k_out is None:
            k_out, k_to = _new_heads(k, tokens, hk, dim)
        else:
            k_to = k_heads if k_out is k else _require_heads(k_out, "k_out", dtype, dev, hk, dim, tokens)
    _launch("rvq_rotary", dev, rotation, DTYPES[dtype], tokens, hq, hk, dim, clips, _at(cu), _at(first),
            _at(positions), x_heads if hq else None, k_heads if hk else None, q_to, k_to, _stream(x))
    return (None if q is None else q_out), (None if k is None else k_out)


def rvq_rotary_append(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, frequencies: torch.Tensor,
                      k_pool: torch.Tensor, v_pool: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                      cu: Optional[torch.Tensor] = None, interleaved: bool = False, amplitude: float = 1.0,
                      out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """``rvq_cache_append`` with rotary positions: new frame i of clip b is at position ``lens[b] + i``. Keys turn on
    their way into the pages, values go there as they are, and the queries ``q`` [T, Hq, D] (None: there are none) are
    returned turned, in ``out`` where given (which may be ``q``)."""
    _require_pools(k_pool, v_pool, (4,))
    dtype, dev = k_pool.dtype, k_pool.device
    _, heads, _, dim = k_pool.shape
    k_heads = _require_heads(k, "k", dtype, dev, heads, dim)
    n = k.shape[0]
    v_heads = _require_heads(v, "v", dtype, dev, heads, dim, n)
    _require_table(table, lens, dev)
    clips, cols = table.shape
    if cu is not None:
        _offsets(cu, "cu", dev, clips)
    elif n != clips:
        raise ValueError("without cu, k must have one frame per clip")
    rotation = _rotation(frequencies, interleaved, False, amplitude, dev, dim)
    hq, q_heads, to = 0, None, None
    if q is not None:
        q_heads = _require_heads(q, "q", dtype, dev, dim=dim, tokens=n)
        hq = q.shape[1]
        if out is None:
            out, to = _new_heads(q, n, hq, dim)
        else:
            to = q_heads if out is q else _require_heads(out, "out", dtype, dev, hq, dim, n)
    elif out is not None:
        raise ValueError("out needs q")
    _launch("rvq_rotary_append", dev, _cache_shape(k_pool, clips, cols), rotation, hq, q_heads, k_heads, v_heads, n,
            _at(cu), table.data_ptr(), lens.data_ptr(), to, k_pool.data_ptr(), v_pool.data_ptr(), _stream(k_pool))
    return out


def rvq_cache_scratch_bytes(n_clips: int, n_pages: int) -> int:
    """Workspace of reserve, fork and compact."""
    size = _lib().rvq_cache_scratch_bytes(n_clips, n_pages)
    if size < 0:
        raise RVQError("rvq_cache_scratch_bytes", size, rvq_status_string(size))
    return size


def _scratch(table: torch.Tensor, refs: torch.Tensor) -> torch.Tensor:
    return table.new_empty(rvq_cache_scratch_bytes(table.shape[0], refs.shape[0]), dtype=torch.uint8)


def rvq_cache_reserve(table: torch.Tensor, lens: torch.Tensor, new_lens: torch.Tensor, refs: torch.Tensor,
                      page_size: int):
    """Gives every clip pages for positions ``lens[b]`` .. ``new_lens[b] - 1``, lowest free pages first; pages that it
    was given for them before (reserved ahead) stay.

    ``table`` [clips, E], ``lens``, ``new_lens`` [clips], ``refs`` [pages], all int32. Returns ``(table, refs,
    missing [1])``; ``missing`` counts the pages that were not there (their entries stay as they were).
    """
    _require_table(table, lens, table.device, refs)
    _require(new_lens, "new_lens", torch.int32, 1, table.device)
    if new_lens.shape != lens.shape:
        raise ValueError("new_lens must match lens")
    table_out, refs_out = torch.empty_like(table), torch.empty_like(refs)
    missing, work = table.new_empty(1), _scratch(table, refs)
    _launch("rvq_cache_reserve", table.device, _ptr(table), _ptr(lens), _ptr(new_lens), _ptr(refs), table.shape[0],
            table.shape[1], page_size, refs.shape[0], _ptr(table_out), _ptr(refs_out), _ptr(missing), _ptr(work),
            work.numel(), _stream(table))
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
    missing, work = table.new_empty(1), _scratch(table, refs)
    _launch("rvq_cache_fork", dev, _cache_shape(k_pool, *table.shape), _layers(k_pool), _ptr(table), _ptr(lens),
            _ptr(refs), _ptr(parents), _ptr(children), children.shape[0], _ptr(k_pool), _ptr(v_pool), _ptr(table_out),
            _ptr(lens_out), _ptr(refs_out), _ptr(missing), _ptr(work), work.numel(), _stream(k_pool))
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
    _launch("rvq_cache_free", table.device, _ptr(table), _ptr(lens), _ptr(refs), _ptr(drop), table.shape[0],
            table.shape[1], page_size, refs.shape[0], _window(window), sinks, _ptr(table_out), _ptr(lens_out),
            _ptr(refs_out), _stream(table))
    return table_out, lens_out, refs_out


def rvq_cache_compact(table: torch.Tensor, refs: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor):
    """Moves the pages in use to the numbers 0 .. live - 1. Returns ``(table, refs, live [1])``."""
    _require_pools(k_pool, v_pool, (4, 5))
    dev = k_pool.device
    _require_table(table, None, dev, refs, k_pool.shape[-4])
    table_out, refs_out = torch.empty_like(table), torch.empty_like(refs)
    live, work = table.new_empty(1), _scratch(table, refs)
    _launch("rvq_cache_compact", dev, _cache_shape(k_pool, *table.shape), _layers(k_pool), _ptr(table), _ptr(refs),
            _ptr(k_pool), _ptr(v_pool), _ptr(table_out), _ptr(refs_out), _ptr(live), _ptr(work), work.numel(),
            _stream(k_pool))
    return table_out, refs_out, live


def rvq_cache_copy(src: torch.Tensor, dst: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor) -> None:
    """Copies page ``src[i]`` to page ``dst[i]`` (int32) in every layer of both pools."""
    _require_pools(k_pool, v_pool, (4, 5))
    _require(src, "src", torch.int32, 1, k_pool.device)
    _require(dst, "dst", torch.int32, 1, k_pool.device)
    if src.shape != dst.shape:
        raise ValueError("src and dst must match")
    _launch("rvq_cache_copy", k_pool.device, _cache_shape(k_pool, 0, 0), _layers(k_pool), _ptr(src), _ptr(dst),
            src.shape[0], _ptr(k_pool), _ptr(v_pool), _stream(k_pool))
