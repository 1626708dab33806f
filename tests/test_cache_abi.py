"""Refusals of the paged-cache entry points: arguments are checked on the host before any
CUDA call (the addresses here are never read)."""
import ctypes

import pytest

import io_aware_exact_19_b200 as fa
from io_aware_exact_19_b200 import build as fa_build

INVALID, UNSUPPORTED = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED
P = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.load_library()


def cache(**kw):
    c = dict(k=4096, v=4096, dtype=1, num_pages=10, page_size=16, H_kv=2, d=64, page_stride=2048, head_stride=1024,
             row_stride=64)
    c.update(kw)
    return fa.KVCacheDesc(*c.values())


def rows(data=4096, row=256, head=64):
    return fa.RowsDesc(data, row, head)


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=4104), INVALID), (dict(dtype=2), INVALID), (dict(num_pages=0), INVALID),
    (dict(page_size=4), INVALID), (dict(page_size=24), INVALID), (dict(page_size=2048), INVALID), (dict(H_kv=0), INVALID),
    (dict(d=0), INVALID), (dict(d=80), UNSUPPORTED), (dict(d=512), UNSUPPORTED), (dict(row_stride=60), INVALID),
    (dict(page_stride=0), INVALID), (dict(head_stride=-64), INVALID),
    (dict(num_pages=2 ** 27, page_size=16), UNSUPPORTED),
]


def plan(lib, B=2, rows=4, max_new=8, page=16, pages=10, width=3, ctx=P, cu=P, parent=None, table=P, held=P, free=P,
         count=P, seq=P, slot=P, pos=P, mask=None):
    return lib.fa_cache_plan(B, rows, max_new, page, pages, width, ctx, cu, parent, table, held, free, count, seq, slot,
                             pos, mask, None)


def test_plan_refusals(lib):
    for kw in (dict(B=0), dict(rows=-1), dict(max_new=0), dict(page=12), dict(page=4), dict(pages=0), dict(width=0),
               dict(ctx=None), dict(cu=ctypes.c_void_p(4098)), dict(table=None), dict(held=None), dict(free=None),
               dict(count=None), dict(seq=None), dict(slot=None), dict(pos=None), dict(parent=P), dict(mask=P),
               dict(parent=P, mask=ctypes.c_void_p(4100))):
        assert plan(lib, **kw) == INVALID, kw
    for kw in (dict(B=4097), dict(parent=P, mask=P, max_new=513), dict(pages=2 ** 27, page=16),
               dict(B=4096, width=2 ** 20)):
        assert plan(lib, **kw) == UNSUPPORTED, kw


def rope(lib, dtype=1, x=P, out=P, B=1, H=2, N=3, d=64, xs=(384, 192, 64), os=(384, 192, 64), pos=P, pa=3, pb=0, axes=1,
         inv=P, axis=P, rot=64):
    three = ctypes.c_longlong * 3
    return lib.fa_rope(dtype, x, out, B, H, N, d, None if xs is None else three(*xs), three(*os), pos, pa, pb, axes, inv,
                       axis, rot, 0, 0, None)


def test_rope_refusals(lib):
    for kw in (dict(dtype=3), dict(x=None), dict(out=ctypes.c_void_p(4104)), dict(B=0), dict(H=0), dict(N=0), dict(d=0),
               dict(xs=None), dict(xs=(384, 192, 60)), dict(os=(-8, 192, 64)), dict(pos=None), dict(pa=-1), dict(pb=-1),
               dict(axes=0), dict(axes=9), dict(inv=None), dict(axis=None), dict(rot=0), dict(rot=24), dict(rot=80)):
        assert rope(lib, **kw) == INVALID, kw
    for kw in (dict(d=80, rot=16), dict(B=2 ** 16, N=2 ** 15), dict(H=70000)):
        assert rope(lib, **kw) == UNSUPPORTED, kw


def append(lib, c=None, T=4, Hq=4, q=rows(), k=rows(), v=rows(), qo=rows(), slot=P, pos=P, pa=4, axes=1, inv=P, axis=P,
           rot=64):
    ref = lambda x: None if x is None else ctypes.byref(x)
    return lib.fa_rope_append(ref(c or cache()), T, Hq, ref(q), ref(k), ref(v), ref(qo), slot, pos, pa, axes, inv, axis,
                              rot, 0, None)


def test_append_refusals(lib):
    for kw, st in BAD_CACHES:
        assert append(lib, cache(**kw)) == st, kw
    assert lib.fa_rope_append(None, 1, 1, None, None, None, None, P, P, 1, 1, P, P, 64, 0, None) == INVALID
    for kw in (dict(T=-1), dict(Hq=0), dict(q=None), dict(qo=None), dict(k=None), dict(v=rows(None)),
               dict(k=rows(4100)), dict(q=rows(row=60)), dict(qo=rows(head=-8)), dict(slot=None), dict(pos=None),
               dict(axes=0), dict(inv=None), dict(axis=None), dict(rot=8), dict(rot=128)):
        assert append(lib, **kw) == INVALID, kw
    assert append(lib, T=0) == fa.FA_OK  # nothing to do


def tree(lib, c=None, q=rows(), o=rows(), lse=P, B=2, T=4, max_q=8, Hq=4, width=3, table=P, cu=P, seq=P, mask=None,
         scale=0.125, ws=P):
    ref = lambda x: None if x is None else ctypes.byref(x)
    return lib.fa_tree_fwd(ref(c or cache()), ref(q), ref(o), lse, B, T, max_q, Hq, width, table, cu, seq, mask, scale,
                           ws, None)


def test_tree_refusals(lib):
    for kw, st in BAD_CACHES:
        assert tree(lib, cache(**kw)) == st, kw
    for kw in (dict(q=None), dict(o=rows(4104)), dict(lse=None), dict(B=0), dict(T=-1), dict(max_q=0), dict(Hq=0),
               dict(Hq=5), dict(width=0), dict(table=None), dict(cu=None), dict(seq=ctypes.c_void_p(4098)),
               dict(mask=ctypes.c_void_p(4100)), dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=None),
               dict(ws=ctypes.c_void_p(4096 + 16)), dict(q=rows(row=100))):
        assert tree(lib, **kw) == INVALID, kw
    for kw in (dict(B=4097), dict(mask=P, max_q=513), dict(Hq=70000), dict(T=2 ** 30, Hq=4)):
        assert tree(lib, **kw) == UNSUPPORTED, kw
    assert tree(lib, T=0) == fa.FA_OK  # nothing to do
    assert lib.fa_debug_tree_withhold(ctypes.byref(cache()), ctypes.byref(rows()), ctypes.byref(rows()), P, 2, 4, 8, 4, 3, P,
                                      P, P, None, 0.125, P, 0, None) == INVALID
    size = lib.fa_tree_fwd_workspace_size
    assert size(2, 4, 8, 4, 2, 64) > 0
    for bad in ((0, 4, 8, 4, 2, 64), (2, -1, 8, 4, 2, 64), (2, 4, 0, 4, 2, 64), (2, 4, 8, 5, 2, 64), (2, 4, 8, 4, 2, 80)):
        assert size(*bad) == 0


def test_outputs_that_overlap_themselves(lib):
    for kw in (dict(page_stride=56), dict(head_stride=8), dict(row_stride=56)):
        c = cache(**kw)
        assert append(lib, c) == tree(lib, c) == INVALID, kw
    for kw in (dict(os=(384, 192, 0)), dict(os=(384, 0, 64)), dict(B=2, os=(0, 192, 64)), dict(os=(384, 192, 56))):
        assert rope(lib, **kw) == INVALID, kw
    for bad in (rows(row=0), rows(head=0), rows(head=56)):
        assert append(lib, qo=bad) == INVALID and tree(lib, o=bad) == INVALID


def test_commit_refusals(lib):
    def commit(c=None, B=2, width=3, acc=4, table=P, ctx=P, a=P, n=P, out=P):
        return lib.fa_cache_commit(ctypes.byref(c or cache()), B, width, acc, table, ctx, a, n, out, None)
    for kw, st in BAD_CACHES:
        assert commit(cache(**kw)) == st, kw
    for kw in (dict(B=0), dict(width=0), dict(acc=0), dict(table=None), dict(ctx=None), dict(a=None), dict(n=None),
               dict(out=ctypes.c_void_p(4098))):
        assert commit(**kw) == INVALID, kw
    assert commit(B=4097) == UNSUPPORTED


def test_binding_refuses_mismatched_tensors(lib):
    import torch
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    lse, ws = torch.zeros(3, 2), torch.zeros(1 << 20, dtype=torch.uint8)
    # nothing here is on a GPU, and several shapes do not fit: refused before any call
    for call in (lambda: fa.fa_rope_append(x, x, x, x, k, k, i32(3)),
                 lambda: fa.fa_rope_append(x, x, x, x, k, k[:3], i32(3)),
                 lambda: fa.fa_rope_append(x, x, x, x, k[0], k[0], i32(3)),
                 lambda: fa.fa_tree_fwd(x, k, k, i32(1, 4), i32(1), i32(2), x, lse, ws, max_q=3),
                 lambda: fa.fa_cache_commit(k, k, i32(1, 4), i32(1), i32(1, 2), i32(1), i32(1)),
                 lambda: fa.fa_rope(x[None], x[None], i32(1, 2), torch.zeros(32), torch.zeros(32, dtype=torch.uint8)),
                 lambda: fa.fa_cache_plan(i32(1), i32(2), i32(1, 4), i32(1), i32(4), i32(1), i32(1), i32(1), i32(1), 16, 1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        fa.fa_cache_commit(None, k, i32(1, 4), i32(1), i32(1, 2), i32(1), i32(1))
    with pytest.raises(AttributeError):
        fa.fa_no_such_call


def test_rope_tables(lib):
    inv, axis = fa.rope_tables(16, [4, 2, 2], device="cpu")
    assert axis.tolist() == [0, 0, 0, 0, 1, 1, 2, 2] and inv[1].item() == pytest.approx(10000.0 ** -0.125)
    assert fa.rope_tables(16, [4, 2, 2], interleaved=True, device="cpu")[1].tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    with pytest.raises(ValueError):
        fa.rope_tables(16, [4, 2], device="cpu")
