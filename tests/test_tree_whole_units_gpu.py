"""fa_tree_fwd where units are whole and each has its own CTA, and the paths of the kernel for more than 64
rows a head that Gaussian inputs over good pages do not take."""
import ctypes

import numpy as np
import pytest
import torch

import io_aware_exact_19_b200 as fa
from oracle import cache as C
from tests.cache_cases import Paged, assert_attention, attention_reference, f64, random_parents
from tests.test_tree_gpu import attend, mask_of, queries, workspace

pytestmark = pytest.mark.gpu


def units(p, Hq):
    """Units of the call, which go whole from 148 on (and in turn from 1184 on), rows of a request and head."""
    G, tile = Hq // p.H_kv, 64 if p.d == 256 else 128
    return p.H_kv * -(-p.T * G // tile), p.max_new * G


@pytest.mark.parametrize("ctx,new,Hq,H_kv,d,page,fmt", [
    ([700, 129, 40], [300, 333, 1], 32, 8, 128, 16, "bf16"),
    ([0, 1000], [500, 200], 28, 4, 64, 64, "fp16"),          # rows of a unit end inside a token
    ([90, 0, 300], [600, 650, 5], 8, 4, 256, 32, "bf16"),
    ([1000, 0], [512, 700], 16, 8, 96, 8, "fp16"),
    ([30] * 12, [150, 0, 1, 149] * 3, 32, 8, 128, 16, "bf16"),
])
def test_a_chain_of_whole_units(ctx, new, Hq, H_kv, d, page, fmt):
    p = Paged(ctx, new, H_kv, d, page, fmt, seed=sum(new) + d)
    whole, rows = units(p, Hq)
    assert 148 <= whole < 8 * 148 and rows >= 512
    q = queries(p, Hq, p.T + 5)
    o, lse = attend(p, q)
    assert_attention(p, o, lse, attention_reference(p, f64(q), d ** -0.5))
    assert torch.isnan(o[p.T:]).all() and torch.isnan(lse[p.T:]).all()
    again = attend(p, q)
    assert torch.equal(o[:p.T], again[0][:p.T]) and torch.equal(lse[:p.T], again[1][:p.T])


@pytest.mark.parametrize("ctx,new,Hq,H_kv,d,page,fmt,turns", [
    ([700, 129, 0], [512, 100, 33], 32, 8, 128, 16, "bf16", False),
    ([90, 0, 300, 63], [200, 500, 300, 512], 14, 2, 64, 8, "fp16", False),
    ([127, 5, 500], [512, 512, 300], 8, 8, 256, 32, "bf16", False),
    ([100, 0, 30] * 4, [500, 512, 1] * 4, 40, 8, 96, 64, "bf16", True),  # in turn
])
def test_trees_of_whole_units(ctx, new, Hq, H_kv, d, page, fmt, turns):
    p = Paged(ctx, new, H_kv, d, page, fmt, seed=sum(new) + d)
    whole, rows = units(p, Hq)
    assert rows >= 512 and (whole >= 8 * 148 if turns else 148 <= whole < 8 * 148)
    bits, mask = mask_of(p, random_parents(new, p.rng))
    q = queries(p, Hq)
    o, lse = attend(p, q, mask)
    assert_attention(p, o, lse, attention_reference(p, f64(q), d ** -0.5, bits))


@pytest.mark.parametrize("d,fmt,new,Hq,H_kv", [(64, "fp16", 100, 2, 1), (128, "bf16", 40, 8, 2), (128, "fp16", 350, 8, 4),
                                                (96, "bf16", 600, 32, 8)])
def test_growing_scores_rescale_many_rows(d, fmt, new, Hq, H_kv):
    # Keys grow along the sequence, in the direction of every other row's query: that row's reference moves in
    # tile after tile (by about 11 in log2 units at d = 64), the others' stays with the first tile. Cut units and
    # (the last) whole ones.
    p = Paged([1300], [new], H_kv, d, 16, fmt, seed=d + new)
    for r in range(0, 1300 + new, 16):
        page = int(p.table_host[0, r // 16])
        p.k[page] = torch.abs(p.k[page]).clamp(max=1e-2) + 0.03 * (r / 16)
    p.k.nan_to_num_(0.0)
    q = torch.full((new, Hq, d), 2.0, device="cuda").to(p.k.dtype)
    q[1::2] = -2.0
    o, lse = attend(p, q, scale=0.25)
    assert_attention(p, o, lse, attention_reference(p, f64(q), 0.25))


@pytest.mark.parametrize("d,page,fmt,new", [(64, 8, "bf16", 20), (128, 32, "fp16", 20), (128, 16, "bf16", 30),
                                            (64, 128, "bf16", 33), (128, 64, "bf16", 150)])
def test_bad_pages_are_not_seen_by_many_rows(d, page, fmt, new):
    # More than 64 rows a head, tiles with and without a bad page in turn, the last page bad in one request; with
    # 150 rows the units are whole.
    p = Paged([2900] * 6, [new] * 6, 8, d, page, fmt, seed=d + page)
    q = queries(p, 32)
    table, n = p.table.clone(), 2900 + new
    step = max(256 // page, 2)
    table[0, 1::step] = -1
    table[1:4, 1::step] = p.num_pages
    table[4:, 1::step] = 2 ** 30
    table[5, (n - 1) // page] = -2 ** 31
    o, lse = attend(p, q, table=table)
    for b in (0, 3, 5):
        good = np.arange(n) // page % step != 1
        if b == 5:
            good &= np.arange(n) // page != (n - 1) // page
        at = slice(b * new, (b + 1) * new)
        ref = C.tree_attention(f64(q[at]), p.rows_of(p.k, b), p.rows_of(p.v, b), d ** -0.5, C.seen_keys(new, n) & good)
        assert_attention(p, o[at], lse[at], [ref])
    again = attend(p, q, table=table)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("d,Hq,H_kv,new", [(128, 32, 8, [300, 333, 1]), (64, 40, 8, [500] * 8), (256, 8, 4, [600, 650, 5])])
def test_waits_of_whole_units_that_run_out_end_the_call(d, Hq, H_kv, new):
    # No load is issued: every CTA's first wait reaches its limit, its later ones return at once, the call ends,
    # the status tells, and the next call works. With a CTA for each unit, and (the second) in turn.
    p = Paged([50] * len(new), new, H_kv, d, 16, "bf16", seed=20)
    whole, rows = units(p, Hq)
    assert rows >= 512 and (whole >= 8 * 148 if len(new) == 8 else 148 <= whole < 8 * 148)
    q = queries(p, Hq)
    want = attend(p, q)
    o, lse, ws = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), workspace(p, Hq)
    desc = fa.KVCacheDesc(p.k.data_ptr(), p.v.data_ptr(), fa.FA_BF16, p.num_pages, 16, H_kv, d, *p.k.stride()[:3])
    at = [fa.RowsDesc(t.data_ptr(), Hq * d, d) for t in (q, o)]
    st = fa.load_library().fa_debug_tree_withhold(
        ctypes.byref(desc), *(ctypes.byref(r) for r in at), lse.data_ptr(), len(new), p.T, p.max_new, Hq, p.table.shape[1],
        p.table.data_ptr(), p.cu.data_ptr(), p.seq_len.data_ptr(), None, d ** -0.5, ws.data_ptr(), 20,
        torch.cuda.current_stream().cuda_stream)
    assert st == fa.FA_OK
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_ERR_TIMEOUT
    assert fa.fa_device_status() == fa.FA_OK
    again = attend(p, q)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
