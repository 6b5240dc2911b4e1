"""Paged key/value cache on MI355X (gfx950): Python binding of ``libkm_cache.so``.

A thin ctypes layer over ``include/kmeans_cache.h``, in the manner of the
K-Means binding: it checks tensors, passes pointers, strides and the current
HIP stream, and never computes anything itself.  Key/value-cache compression
is one of the uses that the page "Flash-KMeans: Fast and Memory-Efficient
Exact K-Means" (gist.science summary of paper 2603.09229) names for K-Means as
an online primitive (tech §1, §5); the cache here takes a request's clustered
keys beside its exact ones.

Entry points (all tensors on one ROCm device):
  tables(ctx_lens, new_lens, block_table, free_pages, page_size, total)   page and slot tables of a serving step
  append(q, k, v, k_cache, v_cache, slots, ...)    norm, rotation and cache write of new tokens
  attend(q, k_cache, v_cache, block_table, query_start, seq_lens, ...)    attention of new tokens over the cache

Caches are 4-d tensors [pages, page_size, heads, dim] of any strides with
adjacent row elements (a transposed [pages, heads, page_size, dim] tensor too).
There is no backward pass: while gradients are recorded, tensors that require
them are refused.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading
from typing import NamedTuple

import torch

from . import KM_BF16, KM_F16, KM_F32, KMeansError, Workspace

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkm_cache.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "kmeans_cache.h")

__all__ = ["KVCache", "Tables", "Workspace", "append", "attend", "tables"]

_DT = {torch.bfloat16: KM_BF16, torch.float16: KM_F16, torch.float32: KM_F32}
KM_ERR_WORKSPACE = 3
_lock = threading.Lock()
_lib = None


class KVCache(ctypes.Structure):
    """km_kv_cache of include/kmeans_cache.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [
        (n, ctypes.c_int64) for n in ("pages", "page_size", "heads", "dim", "k_page", "k_slot", "k_head", "v_page",
                                      "v_slot", "v_head")]


class Tables(NamedTuple):
    """What ``tables`` writes: see kmeans_kv_tables."""
    seq_lens: torch.Tensor
    query_start: torch.Tensor
    page_start: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor


def lib():
    """The loaded HIP library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                                   "(python -m means_clustering_amd.build)")
            L = ctypes.CDLL(LIB_PATH)
            i64, vp, c_int, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            cache, f = ctypes.POINTER(KVCache), ctypes.c_float
            sig = {
                "kmeans_kv_tables": (c_int, [vp, vp, vp, i64, i64, vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, vp,
                                             vp]),
                "kmeans_kv_append": (c_int, [cache, c_int, i64, vp, i64, i64, i64, vp, i64, i64, vp, i64, i64, vp, vp,
                                             f, vp, vp, i64, i64, c_int, vp, vp, i64, i64, vp]),
                "kmeans_kv_attend_workspace": (sz, [cache, i64, i64, i64, i64]),
                "kmeans_kv_attend": (c_int, [cache, c_int, vp, i64, i64, i64, i64, vp, i64, i64, i64, vp, vp, vp, i64,
                                             i64, f, i64, i64, vp, i64, i64, vp, vp, sz, vp]),
                "kmeans_kv_last_error": (ctypes.c_char_p, []),
            }
            for name, (res, args) in sig.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
        return _lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/kmeans_cache.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:[\w\s\*]+?)\b(kmeans_kv_\w+)\s*\(", text, re.M)))


def _check(status: int):
    if status != 0:
        raise KMeansError(status, lib().kmeans_kv_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


# The checks run in every call, which for a decode step costs as much host time as the step takes on the GPU: they
# compare before they format anything.

def _ints(t, name: str, index: int, n: int):
    if t.dtype is not torch.int32 or t.shape != (n,) or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 vector of {n} entries on cuda:{index}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows(t, name: str, index: int, dtype, shape):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {shape} on cuda:{index}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    s = t.stride()
    if s[2] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return s


def _floats(t, name: str, index: int, shape):
    if t.dtype is not torch.float32 or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {shape} on cuda:{index}")
    return t.data_ptr()


def _cache(k_cache, v_cache):
    shape = k_cache.shape
    if len(shape) != 4 or not k_cache.is_cuda:
        raise ValueError("k_cache must be a [pages, page_size, heads, dim] device tensor")
    if k_cache.dtype not in _DT:
        raise TypeError(f"the cache must be bfloat16 or float16, got {k_cache.dtype}")
    a = k_cache.stride()
    b, v = (0, 0, 0, 1), None
    if v_cache is not None:
        if v_cache.shape != shape or v_cache.dtype is not k_cache.dtype or (
                v_cache.get_device() != k_cache.get_device()):
            raise ValueError("v_cache must match k_cache")
        b, v = v_cache.stride(), v_cache.data_ptr()
    if a[3] != 1 or b[3] != 1:
        raise ValueError("the last dimension of the caches must be contiguous")
    return KVCache(k_cache.data_ptr(), v, *shape, a[0], a[1], a[2], b[0], b[1], b[2])


def _no_backward():
    raise ValueError("the cache's calls have no backward pass, and a tensor requires gradients: call them under "
                     "torch.no_grad()")


def _table(t, index: int):
    if t.dtype is not torch.int32 or t.dim() != 2 or t.get_device() != index:
        raise ValueError(f"block_table must be an int32 matrix on cuda:{index}")
    R, width = t.shape
    stride, one = t.stride()
    if one != 1 and width > 1:
        raise ValueError("the rows of block_table must be contiguous")
    if stride < width:
        if R > 1:
            raise ValueError(f"the rows of block_table must not overlap (row stride {stride}, {width} columns)")
        stride = width
    return R, width, stride


# The handle of a device's current stream (torch.cuda.current_stream would make a Stream object of it).
_stream = torch._C._cuda_getCurrentRawStream
_device = torch._C._cuda_getDevice
_capturing = torch._C._cuda_isCurrentStreamCapturing
_recording = torch.is_grad_enabled


def _on(dev: int, fn):
    """fn with the tensors' device as the current one, to whose streams a launch belongs."""
    if _device() == dev:
        return fn

    def there(*args):
        with torch.cuda.device(dev):
            return fn(*args)
    return there


def tables(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
           page_size: int, total: int, pos_offset: torch.Tensor | None = None) -> Tables:
    """Page and slot tables of one serving step, from the requests' lengths (kmeans_kv_tables).

    ``block_table`` [R, width] is updated in place: the pages that the ``new_lens`` tokens need beyond those of
    ``ctx_lens`` are taken from ``free_pages`` in order.  ``total`` is the number of new tokens (the capacity of
    ``positions`` and ``slots``).  ``pos_offset`` is added to positions.
    """
    dev = ctx_lens.get_device()
    if dev < 0:
        raise ValueError("ctx_lens must be a device tensor")
    R, width, stride = _table(block_table, dev)
    c, n = _ints(ctx_lens, "ctx_lens", dev, R), _ints(new_lens, "new_lens", dev, R)
    f = _ints(free_pages, "free_pages", dev, free_pages.numel())
    o = None if pos_offset is None else _ints(pos_offset, "pos_offset", dev, R)
    if total < 0:
        raise ValueError("total must not be negative")
    # one allocation, five views: seq_lens, query_start, page_start, positions, slots
    seq, qs, ps, pos, slots = ctx_lens.new_empty(3 * R + 2 + 2 * total).split_with_sizes(
        (R, R + 1, R + 1, total, total))
    _check(_on(dev, lib().kmeans_kv_tables)(
        c, n, o, R, page_size, block_table.data_ptr(), width, stride, f, free_pages.shape[0], total, seq.data_ptr(),
        qs.data_ptr(), ps.data_ptr(), pos.data_ptr(), slots.data_ptr(), _stream(dev)))
    return Tables(seq, qs, ps, pos, slots)


def append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor | None, k_cache: torch.Tensor,
           v_cache: torch.Tensor | None, slots: torch.Tensor | None, positions: torch.Tensor | None = None,
           rope: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
           k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
           out: torch.Tensor | None = None):
    """Norm and rotation of new queries and keys, and the write of keys and values into the cache (kmeans_kv_append).

    q [T, q_heads, dim], k and v [T, heads, dim] may be views of one packed projection.  ``q_weight`` and
    ``k_weight`` (fp32 [dim]) turn the RMS norm on, ``rope`` (fp32 [max_pos, rot]: cosines, then sines) with
    ``positions`` the rotation.  Token t goes to slot ``slots[t]`` (None: slot t; out of range: padding).  Returns
    the queries (``out``, or a new tensor; ``out`` may be q).
    """
    if _recording():
        for t in (q, k, v, k_cache, v_cache, q_weight, k_weight, rope, out):
            if t is not None and t.requires_grad:
                _no_backward()
    cache = _cache(k_cache, v_cache if v is not None else None)
    dev, dt = k_cache.get_device(), k_cache.dtype
    T, heads, dim = k.shape[0] if k.dim() else 0, cache.heads, cache.dim
    ks = _rows(k, "k", dev, dt, (T, heads, dim))
    if v is not None and v_cache is None:
        raise ValueError("v needs a v_cache")
    vs = _rows(v, "v", dev, dt, (T, heads, dim)) if v is not None else (0, 0)
    hq, qs, os_ = 0, (0, 0), (0, 0)
    if q is not None:
        hq = q.shape[1] if q.dim() == 3 else 0
        qs = _rows(q, "q", dev, dt, (T, hq, dim))
        if out is None:
            out = k.new_empty((T, hq, dim))
        os_ = _rows(out, "out", dev, dt, (T, hq, dim))
    if (rope is None) != (positions is None):
        raise ValueError("rope and positions go together")
    max_pos = rot = 0
    rope_at = pos_at = slots_at = qw_at = kw_at = None
    if rope is not None:
        if rope.dim() != 2:
            raise ValueError("rope must be [max_pos, rot]")
        max_pos, rot = rope.shape
        rope_at = _floats(rope, "rope", dev, (max_pos, rot))
        pos_at = _ints(positions, "positions", dev, T)
    if slots is not None:
        slots_at = _ints(slots, "slots", dev, T)
    if q_weight is not None:
        qw_at = _floats(q_weight, "q_weight", dev, (dim,))
    if k_weight is not None:
        kw_at = _floats(k_weight, "k_weight", dev, (dim,))
    _check(_on(dev, lib().kmeans_kv_append)(
        cache, _DT[dt], T, _ptr(q), hq, qs[0], qs[1], k.data_ptr(), ks[0], ks[1], _ptr(v), vs[0], vs[1], qw_at, kw_at,
        eps, pos_at, rope_at, max_pos, rot, bool(interleaved), slots_at, _ptr(out) if hq else None, os_[0], os_[1],
        _stream(dev)))
    return out


def attend(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
           query_start: torch.Tensor, seq_lens: torch.Tensor, scale: float | None = None, window: int = 0,
           log_weight: torch.Tensor | None = None, max_new: int | None = None, out: torch.Tensor | None = None,
           lse: bool | torch.Tensor = False, ws: Workspace | None = None):
    """Attention of each request's new tokens over its cached keys and values (kmeans_kv_attend).

    Request r's queries are rows query_start[r] .. query_start[r+1]-1 of q [T, q_heads, dim] and stand at its last
    slots; each sees the slots up to its own, with ``window`` > 0 only the last ``window`` of them.  ``log_weight``
    (fp32 [pages, heads, page_size]) is added to the scores: the logarithm of the number of keys that a centroid
    stands for, 0 for a token, -inf for none.  ``scale`` defaults to dim ** -0.5.  ``max_new`` bounds the new tokens
    of any request (1 in a decode step; left out, it is T, and the kernel for chunks is launched as well).  ``lse``
    True or an fp32 [T, q_heads] tensor also gives the logarithm of each row's sum.  Returns out, or (out, lse).

    Without ``ws`` each call takes its workspace from torch's allocator, so calls of several threads and calls that a
    graph captures share nothing.  A ``ws`` serves one stream of calls at a time; graphs that captured it have to be
    gone before it is.
    """
    if _recording() and (q.requires_grad or k_cache.requires_grad or v_cache.requires_grad or (
            out is not None and out.requires_grad) or (log_weight is not None and log_weight.requires_grad) or (
            isinstance(lse, torch.Tensor) and lse.requires_grad)):
        _no_backward()
    cache = _cache(k_cache, v_cache)
    dev, dt, dim = k_cache.get_device(), k_cache.dtype, cache.dim
    shape = q.shape
    T, hq = (shape[0], shape[1]) if len(shape) == 3 else (0, 0)  # (of another number of dimensions _rows refuses it)
    qs = _rows(q, "q", dev, dt, (T, hq, dim))
    if out is None:
        out = q.new_empty((T, hq, dim))
    os_ = _rows(out, "out", dev, dt, (T, hq, dim))
    R, width, tstride = _table(block_table, dev)
    starts, lens = _ints(query_start, "query_start", dev, R + 1), _ints(seq_lens, "seq_lens", dev, R)
    lw_page = lw_head = 0
    if log_weight is not None:
        if log_weight.shape != (cache.pages, cache.heads, cache.page_size) or (
                log_weight.dtype is not torch.float32 or log_weight.get_device() != dev or log_weight.stride(2) != 1):
            raise ValueError(f"log_weight must be float32 [{cache.pages}, {cache.heads}, {cache.page_size}] on "
                             f"cuda:{dev} with contiguous rows")
        lw_page, lw_head = log_weight.stride(0), log_weight.stride(1)
    if lse is True:
        lse = q.new_empty((T, hq), dtype=torch.float32)
    elif lse is False:
        lse = None
    l = None if lse is None else _floats(lse, "lse", dev, (T, hq))
    if max_new is None:
        max_new = T
    L, stream = lib(), _stream(dev)
    if ws is None:
        # (freed at the end: the allocator gives it to later work of this stream only, a graph's stays the graph's)
        buf = q.new_empty(L.kmeans_kv_attend_workspace(cache, T, hq, R, max_new), dtype=torch.uint8)
    else:
        buf = ws.buf
        if buf is not None:
            if buf.get_device() != dev:
                buf = None
            elif _capturing():
                ws.hold()
    for _ in range(2):
        status = _on(dev, L.kmeans_kv_attend)(
            cache, _DT[dt], q.data_ptr(), T, hq, qs[0], qs[1], block_table.data_ptr(), R, width, tstride, starts, lens,
            _ptr(log_weight), lw_page, lw_head, dim ** -0.5 if scale is None else scale, window, max_new,
            out.data_ptr(), os_[0], os_[1], l, _ptr(buf), 0 if buf is None else buf.numel(), stream)
        if status != KM_ERR_WORKSPACE or ws is None:
            break
        # the first call, or a larger one than before (the workspace is the last argument to be refused)
        buf = ws.get(L.kmeans_kv_attend_workspace(cache, T, hq, R, max_new), q.device)
    _check(status)
    return out if lse is None else (out, lse)
