"""Python binding of libfa.so, the B200 (sm_100a) exact fused attention library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/fa.h``. PyTorch supplies device
memory and streams. There is no fallback: if ``libfa.so`` is missing or no CUDA
device is present, the calls raise.

Functions keep the C names: :func:`fa_fwd`, :func:`fa_bwd`,
:func:`fa_blocksparse_fwd`, :func:`fa_blocksparse_bwd`, :func:`fa_fwd_qk`,
:func:`fa_bwd_qk` (N_q query rows, N_k key rows), :func:`fa_bwd_workspace_size`,
plus debug entry points for tile traces and the device status word. Serving over a
paged key/value cache: :func:`fa_cache_plan`, :func:`fa_rope_append`,
:func:`fa_tree_fwd`, :func:`fa_cache_commit`, and :class:`PagedCache`, which keeps
the buffers they share; :func:`fa_rope` rotates q and k for training.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfa.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)
FA_FP16, FA_BF16 = 0, 1

EXPORTED = (
    "fa_status_string", "fa_fwd", "fa_bwd", "fa_blocksparse_fwd", "fa_blocksparse_bwd",
    "fa_bwd_workspace_size", "fa_fwd_trace_size", "fa_bwd_trace_size", "fa_bwd_row_tile",
    "fa_debug_fwd_trace", "fa_debug_bwd_trace", "fa_debug_bwd_phase", "fa_device_status",
    "fa_debug_timeout_probe", "fa_bwd_noalloc", "fa_fwd_qk", "fa_bwd_qk", "fa_debug_fwd_withhold",
    "fa_fwd_splitkv", "fa_fwd_splitkv_workspace_size", "fa_fwd_splitkv_splits", "fa_debug_bwd_withhold",
    "fa_fwd_dropout", "fa_bwd_dropout", "fa_debug_dropout_draws", "fa_fwd_fp8",
    "fa_cache_plan", "fa_rope", "fa_rope_append", "fa_tree_fwd", "fa_tree_fwd_workspace_size", "fa_cache_commit",
)

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


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfa.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is not built; run `python -m io_aware_exact_19_b200.build`")
    lib = ctypes.CDLL(path)
    vp, i, f, sz, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
    fwd_args = [i, vp, vp, vp, vp, vp, i, i, i, i, f, i]
    bwd_args = [i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i]
    sigs = {
        "fa_status_string": ([i], ctypes.c_char_p),
        "fa_fwd": (fwd_args + [vp], i),
        "fa_blocksparse_fwd": (fwd_args + [vp, vp], i),
        "fa_debug_fwd_trace": (fwd_args + [vp, vp, vp], i),
        "fa_bwd": (bwd_args + [vp], i),
        "fa_blocksparse_bwd": (bwd_args + [vp, vp], i),
        "fa_debug_bwd_trace": (bwd_args + [vp, vp, vp], i),
        "fa_debug_bwd_phase": ([i] + bwd_args + [vp, vp], i),
        "fa_bwd_workspace_size": ([i, i, i, i], sz),
        "fa_fwd_trace_size": ([i, i, i], sz),
        "fa_bwd_trace_size": ([i, i, i, i], sz),
        "fa_bwd_row_tile": ([i], i),
        "fa_device_status": ([vp], i),
        "fa_debug_timeout_probe": ([i, vp], i),
        "fa_debug_fwd_withhold": (fwd_args + [i, vp], i),
        "fa_debug_bwd_withhold": (bwd_args + [i, vp], i),
        "fa_bwd_noalloc": (bwd_args[:10] + bwd_args[11:] + [vp], i),
        # N_q, N_k in place of N
        "fa_fwd_qk": (fwd_args[:8] + [i] + fwd_args[8:] + [vp, vp], i),
        "fa_bwd_qk": (bwd_args[:13] + [i] + bwd_args[13:] + [vp, vp], i),
        "fa_fwd_splitkv": (fwd_args[:8] + [i] + fwd_args[8:] + [vp, i, vp, vp], i),
        "fa_fwd_splitkv_workspace_size": ([i, i, i, i, i], sz),
        "fa_fwd_splitkv_splits": ([i, i, i, i], i),
        "fa_fwd_dropout": (fwd_args[:8] + [i] + fwd_args[8:] + [vp, f, ctypes.c_ulonglong, vp], i),
        "fa_bwd_dropout": (bwd_args[:13] + [i] + bwd_args[13:] + [vp, f, ctypes.c_ulonglong, vp], i),
        "fa_debug_dropout_draws": ([i, i, i, i, ctypes.c_ulonglong, vp, vp, vp], i),
        "fa_fwd_fp8": ([vp, vp, vp, f, f, f, vp, vp, i, i, i, i, i, f, i, vp, vp], i),
        "fa_cache_plan": ([i] * 6 + [vp] * 12, i),
        "fa_rope": ([i, vp, vp, i, i, i, i, vp, vp, vp, ll, ll, i, vp, vp, i, i, i, vp], i),
        "fa_rope_append": ([vp, i, i, vp, vp, vp, vp, vp, vp, ll, i, vp, vp, i, i, vp], i),
        "fa_tree_fwd_workspace_size": ([i] * 6, sz),
        "fa_tree_fwd": ([vp, vp, vp, vp, i, i, i, i, i, vp, vp, vp, vp, f, vp, vp], i),
        "fa_cache_commit": ([vp, i, i, i, vp, vp, vp, vp, vp, vp], i),
    }
    for name, (argtypes, restype) in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = restype
    _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load_library().fa_status_string(int(status)).decode()
    except FileNotFoundError:
        return f"status {status}"


def _check(status: int, where: str) -> None:
    if status != FA_OK:
        raise FAError(status, where)


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float16:
        return FA_FP16
    raise TypeError(f"unsupported dtype {t.dtype}; expected float16 or bfloat16")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _shape(q):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    return tuple(int(x) for x in q.shape)


def _check_tensors(ref, *ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")


def _scale(scale, d):
    return float(scale) if scale is not None else 1.0 / (d ** 0.5)


def fa_fwd(q, k, v, o, lse, causal: bool = False, scale: float | None = None, stream=None) -> None:
    """Forward: writes ``o`` [B,H,N,d] and ``lse`` [B,H,N] fp32 (see include/fa.h)."""
    B, H, N, d = _shape(q)
    _check_tensors(q, k, v, o, lse)
    st = load_library().fa_fwd(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                               _scale(scale, d), int(bool(causal)), _stream(stream))
    _check(st, "fa_fwd")


def fa_blocksparse_fwd(q, k, v, o, lse, block_mask, causal: bool = False, scale: float | None = None,
                       stream=None) -> None:
    """Block-sparse forward; ``block_mask`` is a uint8 CUDA tensor [N/128, N/128]."""
    B, H, N, d = _shape(q)
    _check_tensors(q, k, v, o, lse, block_mask)
    st = load_library().fa_blocksparse_fwd(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H,
                                           N, d, _scale(scale, d), int(bool(causal)), _ptr(block_mask),
                                           _stream(stream))
    _check(st, "fa_blocksparse_fwd")


def fa_bwd_workspace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load_library().fa_bwd_workspace_size(B, H, N, d))


def fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, causal: bool = False, scale: float | None = None,
           stream=None) -> None:
    """Backward: writes ``dq``, ``dk``, ``dv``; ``workspace`` is a CUDA uint8 tensor of
    at least :func:`fa_bwd_workspace_size` bytes."""
    B, H, N, d = _shape(q)
    _check_tensors(q, k, v, o, lse, dout, dq, dk, dv, workspace)
    st = load_library().fa_bwd(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                               _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), B, H, N, d, _scale(scale, d),
                               int(bool(causal)), _stream(stream))
    _check(st, "fa_bwd")


def fa_bwd_noalloc(q, k, v, o, lse, dout, dq, dk, dv, causal: bool = False, scale: float | None = None,
                   stream=None) -> None:
    """Backward without a workspace argument, for callers that cannot allocate device
    memory: the scratch lives in a fixed static device array inside the library (see
    include/fa.h for the size limit and the rule that overlapping calls race)."""
    B, H, N, d = _shape(q)
    _check_tensors(q, k, v, o, lse, dout, dq, dk, dv)
    st = load_library().fa_bwd_noalloc(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                       _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, _scale(scale, d),
                                       int(bool(causal)), _stream(stream))
    _check(st, "fa_bwd_noalloc")


def fa_blocksparse_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, block_mask, causal: bool = False,
                       scale: float | None = None, stream=None) -> None:
    B, H, N, d = _shape(q)
    _check_tensors(q, k, v, o, lse, dout, dq, dk, dv, workspace, block_mask)
    st = load_library().fa_blocksparse_bwd(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                           _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), B, H, N, d,
                                           _scale(scale, d), int(bool(causal)), _ptr(block_mask),
                                           _stream(stream))
    _check(st, "fa_blocksparse_bwd")


def fa_fwd_trace_size(B: int, H: int, N: int) -> int:
    return int(load_library().fa_fwd_trace_size(B, H, N))


def fa_bwd_trace_size(B: int, H: int, N: int, d: int) -> int:
    return int(load_library().fa_bwd_trace_size(B, H, N, d))


def fa_bwd_row_tile(d: int) -> int:
    return int(load_library().fa_bwd_row_tile(d))


def fa_debug_fwd_trace(q, k, v, o, lse, trace, causal: bool = False, block_mask=None, scale=None,
                       stream=None) -> None:
    B, H, N, d = _shape(q)
    st = load_library().fa_debug_fwd_trace(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H,
                                           N, d, _scale(scale, d), int(bool(causal)), _ptr(block_mask),
                                           _ptr(trace), _stream(stream))
    _check(st, "fa_debug_fwd_trace")


def fa_debug_bwd_trace(q, k, v, o, lse, dout, dq, dk, dv, workspace, trace, causal: bool = False,
                       block_mask=None, scale=None, stream=None) -> None:
    B, H, N, d = _shape(q)
    st = load_library().fa_debug_bwd_trace(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                           _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), B, H, N, d,
                                           _scale(scale, d), int(bool(causal)), _ptr(block_mask), _ptr(trace),
                                           _stream(stream))
    _check(st, "fa_debug_bwd_trace")


def fa_debug_bwd_phase(phase: int, q, k, v, o, lse, dout, dq, dk, dv, workspace, causal: bool = False,
                       block_mask=None, scale=None, stream=None) -> None:
    """One of the backward's two launches (0 prep, 1 main); see include/fa.h."""
    B, H, N, d = _shape(q)
    st = load_library().fa_debug_bwd_phase(int(phase), _dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                           _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
                                           B, H, N, d, _scale(scale, d), int(bool(causal)), _ptr(block_mask),
                                           _stream(stream))
    _check(st, "fa_debug_bwd_phase")


def fa_device_status(stream=None) -> int:
    """Synchronise the stream, return and clear the device status word."""
    return int(load_library().fa_device_status(_stream(stream)))


def fa_debug_fwd_withhold(q, k, v, o, lse, timeout_ms: int, causal: bool = False, scale=None, stream=None) -> None:
    """The forward kernel with a producer that issues no load: its waits run out after
    ``timeout_ms`` and record FA_ERR_TIMEOUT (see include/fa.h)."""
    B, H, N, d = _shape(q)
    st = load_library().fa_debug_fwd_withhold(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H,
                                              N, d, _scale(scale, d), int(bool(causal)), int(timeout_ms),
                                              _stream(stream))
    _check(st, "fa_debug_fwd_withhold")


def fa_debug_bwd_withhold(q, k, v, o, lse, dout, dq, dk, dv, workspace, timeout_ms: int, causal: bool = False,
                          scale=None, stream=None) -> None:
    """The backward with main-kernel producers that issue no load: the waits run out
    after ``timeout_ms`` and record FA_ERR_TIMEOUT (see include/fa.h)."""
    B, H, N, d = _shape(q)
    st = load_library().fa_debug_bwd_withhold(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                              _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), B, H, N, d,
                                              _scale(scale, d), int(bool(causal)), int(timeout_ms), _stream(stream))
    _check(st, "fa_debug_bwd_withhold")


def fa_debug_timeout_probe(timeout_ms: int, stream=None) -> None:
    _check(load_library().fa_debug_timeout_probe(int(timeout_ms), _stream(stream)), "fa_debug_timeout_probe")


# ----------------------------------------------------------------------------- conveniences

def fa_fwd_qk(q, k, v, o, lse, causal: bool = False, block_mask=None, scale: float | None = None,
              stream=None) -> None:
    """Forward with q, o [B, H, N_q, d] and k, v [B, H, N_k, d]; the causal mask is
    bottom-right aligned (query i sees key j <= i + N_k - N_q)."""
    B, H, Nq, d = _shape(q)
    Nk = _shape(k)[2]
    _check_tensors(q, k, v, o, lse, block_mask)
    st = load_library().fa_fwd_qk(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk, d,
                                  _scale(scale, d), int(bool(causal)),
                                  _ptr(block_mask) if block_mask is not None else None, _stream(stream))
    _check(st, "fa_fwd_qk")


def fa_bwd_qk(q, k, v, o, lse, dout, dq, dk, dv, workspace, causal: bool = False, block_mask=None,
              scale: float | None = None, stream=None) -> None:
    """Backward of :func:`fa_fwd_qk`; ``workspace`` holds at least
    ``fa_bwd_workspace_size(B, H, N_q, d)`` bytes."""
    B, H, Nq, d = _shape(q)
    Nk = _shape(k)[2]
    _check_tensors(q, k, v, o, lse, dout, dq, dk, dv, workspace, block_mask)
    st = load_library().fa_bwd_qk(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                  _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), B, H, Nq, Nk, d,
                                  _scale(scale, d), int(bool(causal)),
                                  _ptr(block_mask) if block_mask is not None else None, _stream(stream))
    _check(st, "fa_bwd_qk")


def fa_fwd_splitkv_workspace_size(B: int, H: int, Nq: int, d: int, n_splits: int) -> int:
    return int(load_library().fa_fwd_splitkv_workspace_size(B, H, Nq, d, n_splits))


def fa_fwd_splitkv_splits(B: int, H: int, Nq: int, Nk: int) -> int:
    return int(load_library().fa_fwd_splitkv_splits(B, H, Nq, Nk))


def fa_fwd_splitkv(q, k, v, o, lse, n_splits: int, workspace, causal: bool = False, block_mask=None,
                   scale: float | None = None, stream=None) -> None:
    """Split-KV forward: ``n_splits`` key ranges computed apart, then merged; the
    partials stay in ``workspace`` (see include/fa.h for its layout)."""
    B, H, Nq, d = _shape(q)
    Nk = _shape(k)[2]
    _check_tensors(q, k, v, o, lse, workspace, block_mask)
    st = load_library().fa_fwd_splitkv(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk,
                                       d, _scale(scale, d), int(bool(causal)),
                                       _ptr(block_mask) if block_mask is not None else None, int(n_splits),
                                       _ptr(workspace), _stream(stream))
    _check(st, "fa_fwd_splitkv")


def fa_fwd_dropout(q, k, v, o, lse, p_drop: float, seed: int, causal: bool = False, block_mask=None,
                   scale: float | None = None, stream=None) -> None:
    """Forward with dropout on P (keep decisions from Philox4x32-10; see include/fa.h)."""
    B, H, Nq, d = _shape(q)
    Nk = _shape(k)[2]
    _check_tensors(q, k, v, o, lse, block_mask)
    st = load_library().fa_fwd_dropout(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Nq, Nk,
                                       d, _scale(scale, d), int(bool(causal)),
                                       _ptr(block_mask) if block_mask is not None else None, float(p_drop),
                                       ctypes.c_ulonglong(int(seed)), _stream(stream))
    _check(st, "fa_fwd_dropout")


def fa_bwd_dropout(q, k, v, o, lse, dout, dq, dk, dv, workspace, p_drop: float, seed: int, causal: bool = False,
                   block_mask=None, scale: float | None = None, stream=None) -> None:
    """Backward of :func:`fa_fwd_dropout` (same p_drop and seed)."""
    B, H, Nq, d = _shape(q)
    Nk = _shape(k)[2]
    _check_tensors(q, k, v, o, lse, dout, dq, dk, dv, workspace, block_mask)
    st = load_library().fa_bwd_dropout(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dout),
                                       _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace), B, H, Nq, Nk, d,
                                       _scale(scale, d), int(bool(causal)),
                                       _ptr(block_mask) if block_mask is not None else None, float(p_drop),
                                       ctypes.c_ulonglong(int(seed)), _stream(stream))
    _check(st, "fa_bwd_dropout")


def fa_fwd_fp8(q8, k8, v8, q_scale: float, k_scale: float, v_scale: float, o, lse, causal: bool = False,
               block_mask=None, scale: float | None = None, stream=None) -> None:
    """8-bit forward: ``q8``, ``k8``, ``v8`` are uint8 CUDA tensors of e4m3 values
    [B, H, N, 128] with per-tensor scales; ``o`` is bf16 (see include/fa.h)."""
    B, H, Nq, d = _shape(q8)
    Nk = _shape(k8)[2]
    _check_tensors(q8, k8, v8, o, lse, block_mask)
    st = load_library().fa_fwd_fp8(_ptr(q8), _ptr(k8), _ptr(v8), float(q_scale), float(k_scale), float(v_scale),
                                   _ptr(o), _ptr(lse), B, H, Nq, Nk, d, _scale(scale, d), int(bool(causal)),
                                   _ptr(block_mask) if block_mask is not None else None, _stream(stream))
    _check(st, "fa_fwd_fp8")


def fa_debug_dropout_draws(B: int, H: int, Nq: int, Nk: int, seed: int, row_major, col_major, stream=None) -> None:
    """The dropout draws through both device generator paths (uint8 [B*H, Nq, Nk] each)."""
    st = load_library().fa_debug_dropout_draws(B, H, Nq, Nk, ctypes.c_ulonglong(int(seed)), _ptr(row_major),
                                               _ptr(col_major), _stream(stream))
    _check(st, "fa_debug_dropout_draws")


# ----------------------------------------------------------------------------- paged cache

def _call(where: str, device, stream, *args) -> None:
    """Call entry point ``where`` with the stream behind ``args``, on ``device``."""
    import torch
    lib = _lib or load_library()
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(where, device, stream, *args)
    handle = torch.cuda.current_stream().cuda_stream if stream is None else stream.cuda_stream
    _check(getattr(lib, where)(*args, handle), where)


def _ints(device, dtype, **tensors):
    """Contiguous integer tensors of one type on ``device``; the addresses in order."""
    out = []
    for name, t in tensors.items():
        if t.dtype != dtype or not t.is_contiguous() or t.device != device:
            raise ValueError(f"{name}: expected a contiguous {dtype} tensor on {device}, got {t.dtype} on {t.device}")
        out.append(t.data_ptr())
    return out


def _strides(t):
    """Element strides of all but the last dimension (a dimension of size 1 has none of its own)."""
    d = t.shape[-1]
    if d > 1 and t.stride(-1) != 1:
        raise ValueError("the head dimension must be contiguous")
    return [d if n == 1 else st for n, st in zip(t.shape[:-1], t.stride()[:-1])]


def _cache_desc(k, v):
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device or not k.is_cuda:
        raise ValueError("expected two CUDA caches of one type and shape [pages, H_kv, page_size, d]")
    st = _strides(k)
    if st != _strides(v):
        raise ValueError("the caches of K and V must have the same strides")
    pages, heads, page_size, d = k.shape
    return KVCacheDesc(k.data_ptr(), v.data_ptr(), _dtype_code(k), pages, page_size, heads, d, *st)


def _rows_desc(t, like, heads=None):
    """Packed rows [T, H, d] of the cache's type."""
    if t.dim() != 3 or t.dtype != like.dtype or t.device != like.device or t.shape[2] != like.shape[3]:
        raise ValueError("expected packed rows [T, H, d] of the cache's type, device and head dimension")
    if heads is not None and t.shape[1] != heads:
        raise ValueError(f"expected {heads} heads, got {t.shape[1]}")
    return RowsDesc(t.data_ptr(), *_strides(t))


def fa_cache_plan(ctx_len, cu_new, block_table, n_pages, free_list, free_count, seq_len, slot, position, page_size: int,
                  max_new: int, parent=None, tree_mask=None, stream=None) -> None:
    """Pages, slot map, positions and (with ``parent``) tree masks of a step from the
    requests' lengths, on the GPU. int32 tensors: ``ctx_len``, ``n_pages``, ``seq_len`` [B],
    ``cu_new`` [B+1], ``block_table`` [B, max_pages], ``free_list`` [num_pages],
    ``free_count`` [1], ``slot``, ``position``, ``parent`` [rows]; ``tree_mask`` int64
    [rows, ceil(max_new/64)]. See include/fa.h for what is read, written and refused."""
    import torch
    dev = ctx_len.device
    if not ctx_len.is_cuda or block_table.dim() != 2:
        raise ValueError("expected CUDA tensors and a two-dimensional block table")
    B, rows = ctx_len.numel(), slot.numel()
    if (cu_new.numel() != B + 1 or block_table.shape[0] != B or n_pages.numel() != B or seq_len.numel() != B
            or position.numel() != rows or free_count.numel() != 1):
        raise ValueError("lengths do not fit: cu_new [B+1]; block_table, n_pages, seq_len [B]; position [rows]")
    a = _ints(dev, torch.int32, ctx_len=ctx_len, cu_new=cu_new)
    c = _ints(dev, torch.int32, block_table=block_table, n_pages=n_pages, free_list=free_list, free_count=free_count,
              seq_len=seq_len, slot=slot, position=position)
    up = words = None
    if (parent is None) != (tree_mask is None):
        raise ValueError("parent and tree_mask go together")
    if parent is not None:
        if parent.numel() != rows or tuple(tree_mask.shape) != (rows, -(-max_new // 64)):
            raise ValueError("expected parent [rows] and tree_mask [rows, ceil(max_new/64)]")
        up, = _ints(dev, torch.int32, parent=parent)
        words, = _ints(dev, torch.int64, tree_mask=tree_mask)
    _call("fa_cache_plan", dev, stream, B, rows, max_new, page_size, free_list.numel(), block_table.shape[1], *a, up, *c,
          words)


def _rope_tables_ptr(dev, positions, inv_freq, axis):
    import torch
    if positions.dtype != torch.int32 or positions.device != dev or (positions.shape[-1] > 1
                                                                     and positions.stride(-1) != 1):
        raise ValueError("positions: expected int32 on the same device, contiguous along the tokens")
    if inv_freq.numel() != axis.numel():
        raise ValueError("inv_freq and axis hold one entry for each rotated pair")
    f, = _ints(dev, torch.float32, inv_freq=inv_freq)
    a, = _ints(dev, torch.uint8, axis=axis)
    return f, a, 2 * inv_freq.numel()


def fa_rope(x, out, positions, inv_freq, axis, inverse: bool = False, pairs: bool = False, stream=None) -> None:
    """Rotary positions over several axes: ``x`` [B, H, N, d] -> ``out`` (``x`` itself is
    fine). ``positions`` int32 [axes, B, N] or [axes, N]; ``inv_freq`` fp32 and ``axis`` uint8,
    one entry for each rotated pair (:func:`rope_tables`). ``inverse`` turns back, which is
    the gradient. Strided views are taken as they are."""
    B, H, N, d = _shape(x)
    if out.shape != x.shape or out.dtype != x.dtype or out.device != x.device or not x.is_cuda:
        raise ValueError("x and out must be CUDA tensors of one shape and type")
    if positions.dim() == 2:
        positions = positions[:, None]
    if positions.dim() != 3 or positions.shape[1] not in (1, B) or positions.shape[2] != N:
        raise ValueError("expected positions [axes, B, N] or [axes, N]")
    f, a, rot = _rope_tables_ptr(x.device, positions, inv_freq, axis)
    three = ctypes.c_longlong * 3
    _call("fa_rope", x.device, stream, _dtype_code(x), x.data_ptr(), out.data_ptr(), B, H, N, d, three(*_strides(x)),
          three(*_strides(out)), positions.data_ptr(), positions.stride(0),
          positions.stride(1) if positions.shape[1] == B else 0, positions.shape[0], f, a, rot, int(bool(inverse)),
          int(bool(pairs)))


def fa_rope_append(q, k, v, q_out, cache_k, cache_v, slot, positions=None, inv_freq=None, axis=None,
                   pairs: bool = False, stream=None) -> None:
    """A step's new rows: ``q`` [T, Hq, d] rotated into ``q_out``, ``k`` [T, H_kv, d] rotated and
    ``v`` as it is written to rows ``slot`` [T] of the caches [pages, H_kv, page_size, d].
    ``positions`` int32 [axes, T]; without it nothing is rotated. ``q`` and ``q_out`` may be None."""
    import torch
    desc = _cache_desc(cache_k, cache_v)
    T, H_kv, dev = k.shape[0], cache_k.shape[1], cache_k.device
    rk, rv = _rows_desc(k, cache_k, H_kv), _rows_desc(v, cache_k, H_kv)
    if v.shape[0] != T or slot.numel() != T or (q is None) != (q_out is None):
        raise ValueError("k, v and slot hold the same rows; q and q_out go together")
    rq = ro = None
    if q is not None:
        if q.shape != q_out.shape or q.shape[0] != T:
            raise ValueError("q and q_out hold the same rows as k")
        rq, ro = _rows_desc(q, cache_k), _rows_desc(q_out, cache_k)
        rq, ro, heads = ctypes.byref(rq), ctypes.byref(ro), q.shape[1]
    else:
        heads = 0
    s, = _ints(dev, torch.int32, slot=slot)
    p = f = a = None
    rot = axes = stride = 0
    if positions is not None:
        if positions.dim() != 2 or positions.shape[1] != T:
            raise ValueError("expected positions [axes, T]")
        f, a, rot = _rope_tables_ptr(dev, positions, inv_freq, axis)
        p, stride, axes = positions.data_ptr(), positions.stride(0), positions.shape[0]
    _call("fa_rope_append", dev, stream, ctypes.byref(desc), T, heads, rq, ctypes.byref(rk), ctypes.byref(rv), ro, s, p,
          stride, axes, f, a, rot, int(bool(pairs)))


def fa_tree_fwd_workspace_size(B: int, rows: int, max_q: int, Hq: int, H_kv: int, d: int) -> int:
    return int(load_library().fa_tree_fwd_workspace_size(B, rows, max_q, Hq, H_kv, d))


def fa_tree_fwd(q, cache_k, cache_v, block_table, seq_len, cu_q, o, lse, workspace, max_q: int, tree_mask=None,
                scale: float | None = None, stream=None) -> None:
    """Attention of packed rows ``q`` [T, Hq, d] (request b's are ``cu_q[b]`` .. ``cu_q[b+1]-1``,
    at most ``max_q``) over the first ``seq_len[b]`` rows of its pages; writes ``o`` and ``lse``
    [T, Hq]. ``tree_mask`` int64 [T, ceil(max_q/64)] as :func:`fa_cache_plan` builds it; None
    is a chain (decoding, prompt chunks). See include/fa.h."""
    import torch
    desc = _cache_desc(cache_k, cache_v)
    T, Hq, d = q.shape
    dev, B = cache_k.device, seq_len.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B or cu_q.numel() != B + 1:
        raise ValueError("expected block_table [B, max_pages], seq_len [B], cu_q [B+1]")
    rq, ro = _rows_desc(q, cache_k), _rows_desc(o, cache_k, Hq)
    if o.shape[0] != T or tuple(lse.shape) != (T, Hq) or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError("expected o like q, lse [T, Hq] and a contiguous workspace on the same device")
    if workspace.numel() * workspace.element_size() < fa_tree_fwd_workspace_size(B, T, max_q, Hq, cache_k.shape[1], d):
        raise ValueError("workspace is smaller than fa_tree_fwd_workspace_size")
    table, lens, cu = _ints(dev, torch.int32, block_table=block_table, seq_len=seq_len, cu_q=cu_q)
    out, = _ints(dev, torch.float32, lse=lse)
    words = None
    if tree_mask is not None:
        if tuple(tree_mask.shape) != (T, -(-max_q // 64)):
            raise ValueError("expected tree_mask [T, ceil(max_q/64)]")
        words, = _ints(dev, torch.int64, tree_mask=tree_mask)
    _call("fa_tree_fwd", dev, stream, ctypes.byref(desc), ctypes.byref(rq), ctypes.byref(ro), out, B, T, max_q, Hq,
          block_table.shape[1], table, cu, lens, words, _scale(scale, d), workspace.data_ptr())


def fa_cache_commit(cache_k, cache_v, block_table, ctx_len, accepted, n_accepted, new_len, stream=None) -> None:
    """Move the accepted path of each request's draft to the front of its new rows:
    ``accepted`` int32 [B, max_accept] request-local indices, strictly increasing, the first
    ``n_accepted[b]`` of them; ``new_len[b]`` (may be ``ctx_len``) = rows then kept."""
    import torch
    desc = _cache_desc(cache_k, cache_v)
    B, dev = ctx_len.numel(), cache_k.device
    if (block_table.dim() != 2 or accepted.dim() != 2 or block_table.shape[0] != B or accepted.shape[0] != B
            or n_accepted.numel() != B or new_len.numel() != B):
        raise ValueError("expected block_table [B, max_pages], accepted [B, max_accept], n_accepted and new_len [B]")
    a = _ints(dev, torch.int32, block_table=block_table, ctx_len=ctx_len, accepted=accepted, n_accepted=n_accepted,
              new_len=new_len)
    _call("fa_cache_commit", dev, stream, ctypes.byref(desc), B, block_table.shape[1], accepted.shape[1], *a)


def attention_forward(q, k, v, causal: bool = False, block_mask=None, scale=None, stream=None):
    """Allocate O and lse with torch and run the forward; returns (o, lse)."""
    import torch
    B, H, N, d = _shape(q)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if block_mask is None:
        fa_fwd(q, k, v, o, lse, causal, scale, stream)
    else:
        fa_blocksparse_fwd(q, k, v, o, lse, block_mask, causal, scale, stream)
    return o, lse


def attention_backward(q, k, v, o, lse, dout, causal: bool = False, block_mask=None, scale=None,
                       workspace=None, stream=None):
    """Allocate dQ, dK, dV (and the workspace if none is given) and run the backward."""
    import torch
    B, H, N, d = _shape(q)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if workspace is None:
        workspace = torch.empty(fa_bwd_workspace_size(B, H, N, d), dtype=torch.uint8, device=q.device)
    if block_mask is None:
        fa_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, causal, scale, stream)
    else:
        fa_blocksparse_bwd(q, k, v, o, lse, dout, dq, dk, dv, workspace, block_mask, causal, scale, stream)
    return dq, dk, dv
