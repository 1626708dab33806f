"""Binding of the paged key/value cache's entry points (declared in ``include/fa.h``).

A serving step on a small batch runs for a few microseconds on the GPU, so the way to the
library is kept short here: every argument is checked once, addresses and strides go
straight into the call.
"""
from __future__ import annotations

import ctypes
import struct
from functools import lru_cache

import torch

from . import FA_BF16, FA_FP16, FAError, _scale, load_library

TREE_MAX = 512  # FA_TREE_MAX: tokens of a drafted tree


class KVCacheDesc(ctypes.Structure):
    """fa_kv_cache of include/fa.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("H_kv", ctypes.c_int), ("d", ctypes.c_int),
                ("page_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong),
                ("row_stride", ctypes.c_longlong)]


class RowsDesc(ctypes.Structure):
    """fa_rows of include/fa.h."""
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong)]


_CACHE, _ROWS, _THREE = struct.Struct("@QQ5iqqq"), struct.Struct("@Qqq"), struct.Struct("@qqq")  # the same, packed
assert _CACHE.size == ctypes.sizeof(KVCacheDesc) and _ROWS.size == ctypes.sizeof(RowsDesc)
_CODES = {torch.float16: FA_FP16, torch.bfloat16: FA_BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(fn, where, dev, stream, *args):
    """Entry point ``fn`` with ``args`` and the stream, on the tensors' device."""
    if dev != _current():
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    else:
        status = fn(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        raise FAError(status, where)


def _addresses(dev, dtype, *tensors):
    """Addresses of contiguous tensors of one type on device ``dev``."""
    out = []
    for t in tensors:
        if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"expected contiguous {dtype} tensors on cuda:{dev}, got {t.dtype} {tuple(t.shape)} with "
                             f"strides {t.stride()} on {t.device}")
        out.append(t.data_ptr())
    return out


def _strides(t):
    """Element strides of all but the last dimension (a dimension of size 1 has none of its own)."""
    shape, st = t.shape, t.stride()
    d = shape[-1]
    if st[-1] != 1 and d > 1:
        raise ValueError("the head dimension must be contiguous")
    if 1 in shape:
        return tuple([d if n == 1 else s for n, s in zip(shape[:-1], st)])
    return st[:-1]


def _cache_desc(k, v):
    shape, dtype = k.shape, k.dtype
    if len(shape) != 4 or shape != v.shape or dtype is not v.dtype or not k.is_cuda or k.get_device() != v.get_device():
        raise ValueError("expected two CUDA caches of one type and shape [pages, H_kv, page_size, d]")
    st = _strides(k)
    if st != _strides(v):
        raise ValueError("the caches of K and V must have the same strides")
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}; expected float16 or bfloat16")
    return _CACHE.pack(k.data_ptr(), v.data_ptr(), code, shape[0], shape[2], shape[1], shape[3], *st)


def _rows_desc(t, like, heads, T):
    """Packed rows [T, heads, d] of the cache's type."""
    if tuple(t.shape) != (T, heads, like.shape[3]) or t.dtype is not like.dtype or t.get_device() != like.get_device():
        raise ValueError(f"expected packed rows [{T}, {heads}, {like.shape[3]}] of the cache's type and device, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    return _ROWS.pack(t.data_ptr(), *_strides(t))


def fa_cache_plan(ctx_len, cu_new, block_table, n_pages, free_list, free_count, seq_len, slot, position, page_size: int,
                  max_new: int, parent=None, tree_mask=None, stream=None) -> None:
    """Pages, slot map, positions and (with ``parent``) tree masks of a step from the
    requests' lengths, on the GPU. int32 tensors: ``ctx_len``, ``n_pages``, ``seq_len`` [B],
    ``cu_new`` [B+1], ``block_table`` [B, max_pages], ``free_list`` [num_pages],
    ``free_count`` [1], ``slot``, ``position``, ``parent`` [rows]; ``tree_mask`` int64
    [rows, ceil(max_new/64)]. See include/fa.h for what is read, written and refused."""
    dev = ctx_len.get_device()
    if dev < 0 or block_table.dim() != 2:
        raise ValueError("expected CUDA tensors and a two-dimensional block table")
    B, rows = ctx_len.numel(), slot.numel()
    table_rows, max_pages = block_table.shape
    if (cu_new.numel() != B + 1 or table_rows != B or n_pages.numel() != B or seq_len.numel() != B
            or position.numel() != rows or free_count.numel() != 1):
        raise ValueError("lengths do not fit: cu_new [B+1]; block_table, n_pages, seq_len [B]; position [rows]")
    c, cu, table, held, free, count, seq, sl, pos = _addresses(
        dev, torch.int32, ctx_len, cu_new, block_table, n_pages, free_list, free_count, seq_len, slot, position)
    up = words = None
    if (parent is None) != (tree_mask is None):
        raise ValueError("parent and tree_mask go together")
    if parent is not None:
        if parent.numel() != rows or tuple(tree_mask.shape) != (rows, -(-max_new // 64)):
            raise ValueError("expected parent [rows] and tree_mask [rows, ceil(max_new/64)]")
        up, = _addresses(dev, torch.int32, parent)
        words, = _addresses(dev, torch.int64, tree_mask)
    _call(load_library().fa_cache_plan, "fa_cache_plan", dev, stream, B, rows, max_new, page_size, free_list.numel(),
          max_pages, c, cu, up, table, held, free, count, seq, sl, pos, words)


def _rope_tables(dev, positions, inv_freq, axis):
    if positions.dtype is not torch.int32 or positions.get_device() != dev or (positions.shape[-1] > 1
                                                                               and positions.stride(-1) != 1):
        raise ValueError("positions: expected int32 on the same device, contiguous along the tokens")
    pairs = inv_freq.numel()
    if pairs != axis.numel():
        raise ValueError("inv_freq and axis hold one entry for each rotated pair")
    f, = _addresses(dev, torch.float32, inv_freq)
    a, = _addresses(dev, torch.uint8, axis)
    return f, a, 2 * pairs


def fa_rope(x, out, positions, inv_freq, axis, inverse: bool = False, pairs: bool = False, stream=None) -> None:
    """Rotary positions over several axes: ``x`` [B, H, N, d] -> ``out`` (``x`` itself is
    fine). ``positions`` int32 [axes, B, N] or [axes, N]; ``inv_freq`` fp32 and ``axis`` uint8,
    one entry for each rotated pair (:func:`rope_tables`). ``inverse`` turns back, which is
    the gradient. Strided views are taken as they are."""
    dev = x.get_device()
    if x.dim() != 4 or out.shape != x.shape or out.dtype is not x.dtype or dev < 0 or out.get_device() != dev:
        raise ValueError("x and out must be CUDA tensors [B, H, N, d] of one shape and type")
    code = _CODES.get(x.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {x.dtype}; expected float16 or bfloat16")
    B, H, N, d = x.shape
    shape, st = tuple(positions.shape), positions.stride()
    if shape[1:] == (N,) and len(shape) == 2:
        per_b = 0
    elif len(shape) == 3 and shape[1:] == (B, N):
        per_b = st[1]
    else:
        raise ValueError("expected positions [axes, B, N] or [axes, N]")
    f, a, rot = _rope_tables(dev, positions, inv_freq, axis)
    _call(load_library().fa_rope, "fa_rope", dev, stream, code, x.data_ptr(), out.data_ptr(), B, H, N, d,
          _THREE.pack(*_strides(x)), _THREE.pack(*_strides(out)), positions.data_ptr(), st[0], per_b, shape[0], f, a, rot,
          1 if inverse else 0, 1 if pairs else 0)


def fa_rope_append(q, k, v, q_out, cache_k, cache_v, slot, positions=None, inv_freq=None, axis=None,
                   pairs: bool = False, stream=None) -> None:
    """A step's new rows: ``q`` [T, Hq, d] rotated into ``q_out``, ``k`` [T, H_kv, d] rotated and
    ``v`` as it is written to rows ``slot`` [T] of the caches [pages, H_kv, page_size, d].
    ``positions`` int32 [axes, T]; without it nothing is rotated. ``q`` and ``q_out`` may be None."""
    desc = _cache_desc(cache_k, cache_v)
    T, H_kv, dev = k.shape[0], cache_k.shape[1], cache_k.get_device()
    rk, rv = _rows_desc(k, cache_k, H_kv, T), _rows_desc(v, cache_k, H_kv, T)
    if slot.numel() != T or (q is None) != (q_out is None):
        raise ValueError("k, v and slot hold the same rows; q and q_out go together")
    rq = ro = None
    heads = 0
    if q is not None:
        heads = q.shape[1]
        rq, ro = _rows_desc(q, cache_k, heads, T), _rows_desc(q_out, cache_k, heads, T)
    s, = _addresses(dev, torch.int32, slot)
    p = f = a = None
    rot = axes = stride = 0
    if positions is not None:
        if positions.dim() != 2 or positions.shape[1] != T:
            raise ValueError("expected positions [axes, T]")
        f, a, rot = _rope_tables(dev, positions, inv_freq, axis)
        p, stride, axes = positions.data_ptr(), positions.stride(0), positions.shape[0]
    _call(load_library().fa_rope_append, "fa_rope_append", dev, stream, desc, T, heads, rq, rk, rv, ro, s, p, stride,
          axes, f, a, rot, 1 if pairs else 0)


@lru_cache(maxsize=1024)
def fa_tree_fwd_workspace_size(B: int, rows: int, max_q: int, Hq: int, H_kv: int, d: int) -> int:
    return int(load_library().fa_tree_fwd_workspace_size(B, rows, max_q, Hq, H_kv, d))


def fa_tree_fwd(q, cache_k, cache_v, block_table, seq_len, cu_q, o, lse, workspace, max_q: int, tree_mask=None,
                scale: float | None = None, stream=None) -> None:
    """Attention of packed rows ``q`` [T, Hq, d] (request b's are ``cu_q[b]`` .. ``cu_q[b+1]-1``,
    at most ``max_q``) over the first ``seq_len[b]`` rows of its pages; writes ``o`` and ``lse``
    [T, Hq]. ``tree_mask`` int64 [T, ceil(max_q/64)] as :func:`fa_cache_plan` builds it; None
    is a chain (decoding, prompt chunks). See include/fa.h."""
    desc = _cache_desc(cache_k, cache_v)
    T, Hq, d = q.shape
    dev, B = cache_k.get_device(), seq_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B or cu_q.numel() != B + 1:
        raise ValueError("expected block_table [B, max_pages], seq_len [B], cu_q [B+1]")
    rq, ro = _rows_desc(q, cache_k, Hq, T), _rows_desc(o, cache_k, Hq, T)
    if tuple(lse.shape) != (T, Hq) or not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("expected lse [T, Hq] and a contiguous workspace on the same device")
    if workspace.nbytes < fa_tree_fwd_workspace_size(B, T, max_q, Hq, cache_k.shape[1], d):
        raise ValueError("workspace is smaller than fa_tree_fwd_workspace_size")
    table, lens, cu = _addresses(dev, torch.int32, block_table, seq_len, cu_q)
    out, = _addresses(dev, torch.float32, lse)
    words = None
    if tree_mask is not None:
        if tuple(tree_mask.shape) != (T, -(-max_q // 64)):
            raise ValueError("expected tree_mask [T, ceil(max_q/64)]")
        words, = _addresses(dev, torch.int64, tree_mask)
    _call(load_library().fa_tree_fwd, "fa_tree_fwd", dev, stream, desc, rq, ro, out, B, T, max_q, Hq,
          block_table.shape[1], table, cu, lens, words, _scale(scale, d), workspace.data_ptr())


def fa_cache_commit(cache_k, cache_v, block_table, ctx_len, accepted, n_accepted, new_len, stream=None) -> None:
    """Move the accepted path of each request's draft to the front of its new rows:
    ``accepted`` int32 [B, max_accept] request-local indices, strictly increasing, the first
    ``n_accepted[b]`` of them; ``new_len[b]`` (may be ``ctx_len``) = rows then kept."""
    desc = _cache_desc(cache_k, cache_v)
    B, dev = ctx_len.numel(), cache_k.get_device()
    if (block_table.dim() != 2 or accepted.dim() != 2 or block_table.shape[0] != B or accepted.shape[0] != B
            or n_accepted.numel() != B or new_len.numel() != B):
        raise ValueError("expected block_table [B, max_pages], accepted [B, max_accept], n_accepted and new_len [B]")
    table, ctx, acc, count, out = _addresses(dev, torch.int32, block_table, ctx_len, accepted, n_accepted, new_len)
    _call(load_library().fa_cache_commit, "fa_cache_commit", dev, stream, desc, B, block_table.shape[1],
          accepted.shape[1], table, ctx, acc, count, out)
