"""Binding of the paged key/value cache's entry points (declared in ``include/fa.h``).

The arguments are read and checked in ``_paged.so`` (``csrc/paged_binding.cpp``), which
calls the library: a serving step on a small batch runs for a few microseconds on the GPU,
less than Python needs to look at its tensors. Mismatched tensors raise ``ValueError`` or
``TypeError``, a refusal by the library ``FAError``.
"""
from __future__ import annotations

import ctypes

import torch  # noqa: F401  (its libraries are loaded before the binding's)

from . import FAError, load_library
from .build import binding_stamp

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


def _load_binding():
    missing = ("the binding _paged.so is missing or was built for another torch; run "
               "`python -m io_aware_exact_19_b200.build`")
    try:
        from . import _paged
    except ImportError as e:
        raise FileNotFoundError(missing) from e
    if getattr(_paged, "built_for", None) != binding_stamp():
        raise FileNotFoundError(missing)
    lib = load_library()
    _paged.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in
                  ("fa_cache_plan", "fa_rope", "fa_rope_append", "fa_tree_fwd", "fa_tree_fwd_workspace_size",
                   "fa_cache_commit")))
    return _paged


_binding = _load_binding()
_plan, _rope, _append, _tree, _commit = (_binding.plan, _binding.rope, _binding.append, _binding.tree, _binding.commit)


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status:
        raise FAError(status, where)


def fa_cache_plan(ctx_len, cu_new, block_table, n_pages, free_list, free_count, seq_len, slot, position, page_size: int,
                  max_new: int, parent=None, tree_mask=None, stream=None) -> None:
    """Pages, slot map, positions and (with ``parent``) tree masks of a step from the
    requests' lengths, on the GPU. int32 tensors: ``ctx_len``, ``n_pages``, ``seq_len`` [B],
    ``cu_new`` [B+1], ``block_table`` [B, max_pages], ``free_list`` [num_pages],
    ``free_count`` [1], ``slot``, ``position``, ``parent`` [rows]; ``tree_mask`` int64
    [rows, ceil(max_new/64)]. See include/fa.h for what is read, written and refused."""
    _check(_plan(ctx_len, cu_new, block_table, n_pages, free_list, free_count, seq_len, slot, position, page_size, max_new,
                 parent, tree_mask, _handle(stream)), "fa_cache_plan")


def fa_rope(x, out, positions, inv_freq, axis, inverse: bool = False, pairs: bool = False, stream=None) -> None:
    """Rotary positions over several axes: ``x`` [B, H, N, d] -> ``out`` (``x`` itself is
    fine). ``positions`` int32 [axes, B, N] or [axes, N]; ``inv_freq`` fp32 and ``axis`` uint8,
    one entry for each rotated pair (:func:`rope_tables`). ``inverse`` turns back, which is
    the gradient. Strided views are taken as they are."""
    _check(_rope(x, out, positions, inv_freq, axis, inverse, pairs, _handle(stream)), "fa_rope")


def fa_rope_append(q, k, v, q_out, cache_k, cache_v, slot, positions=None, inv_freq=None, axis=None,
                   pairs: bool = False, stream=None) -> None:
    """A step's new rows: ``q`` [T, Hq, d] rotated into ``q_out``, ``k`` [T, H_kv, d] rotated and
    ``v`` as it is written to rows ``slot`` [T] of the caches [pages, H_kv, page_size, d].
    ``positions`` int32 [axes, T]; without it nothing is rotated. ``q`` and ``q_out`` may be None."""
    _check(_append(q, k, v, q_out, cache_k, cache_v, slot, positions, inv_freq, axis, pairs, _handle(stream)),
           "fa_rope_append")


def fa_tree_fwd_workspace_size(B: int, rows: int, max_q: int, Hq: int, H_kv: int, d: int) -> int:
    return int(load_library().fa_tree_fwd_workspace_size(B, rows, max_q, Hq, H_kv, d))


def fa_tree_fwd(q, cache_k, cache_v, block_table, seq_len, cu_q, o, lse, workspace, max_q: int, tree_mask=None,
                scale: float | None = None, stream=None) -> None:
    """Attention of packed rows ``q`` [T, Hq, d] (request b's are ``cu_q[b]`` .. ``cu_q[b+1]-1``,
    at most ``max_q``) over the first ``seq_len[b]`` rows of its pages; writes ``o`` and ``lse``
    [T, Hq]. ``tree_mask`` int64 [T, ceil(max_q/64)] as :func:`fa_cache_plan` builds it; None
    is a chain (decoding, prompt chunks). See include/fa.h."""
    _check(_tree(q, cache_k, cache_v, block_table, seq_len, cu_q, o, lse, workspace, max_q, tree_mask,
                 q.shape[-1] ** -0.5 if scale is None else scale, _handle(stream)), "fa_tree_fwd")


def fa_cache_commit(cache_k, cache_v, block_table, ctx_len, accepted, n_accepted, new_len, stream=None) -> None:
    """Move the accepted path of each request's draft to the front of its new rows:
    ``accepted`` int32 [B, max_accept] request-local indices, strictly increasing, the first
    ``n_accepted[b]`` of them; ``new_len[b]`` (may be ``ctx_len``) = rows then kept."""
    _check(_commit(cache_k, cache_v, block_table, ctx_len, accepted, n_accepted, new_len, _handle(stream)),
           "fa_cache_commit")
