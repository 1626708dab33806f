"""fa_tree_fwd against the float64 oracle: chains and drafted trees over a paged cache."""
import numpy as np
import pytest
import torch

import io_aware_exact_19_b200 as fa
from oracle import cache as C
from tests.cache_cases import DT, Paged, assert_attention, attention_reference, f64, ints, random_parents

pytestmark = pytest.mark.gpu


def mask_of(p, parents):
    bits = [C.ancestors(parents[p.cu_host[b]:p.cu_host[b] + n]) for b, n in enumerate(p.new)]
    words = -(-p.max_new // 64)
    host = np.concatenate([C.pack_mask(x, words) for x in bits if len(x)])
    return bits, torch.from_numpy(host).cuda()


def queries(p, Hq, rows=None):
    x = p.rng.standard_normal((rows or p.T, Hq, p.d))
    return torch.from_numpy(x).to(DT[p.fmt]).cuda()


def workspace(p, Hq, rows=None, max_q=None):
    n = fa.fa_tree_fwd_workspace_size(len(p.new), rows or p.T, max_q or p.max_new, Hq, p.H_kv, p.d)
    assert n > 0
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


def attend(p, q, mask=None, max_q=None, scale=None, o=None, table=None, **kw):
    o = torch.full_like(q, float("nan")) if o is None else o
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
    fa.fa_tree_fwd(q, p.k, p.v, p.table if table is None else table, p.seq_len, p.cu, o, lse,
                   workspace(p, q.shape[1], q.shape[0], max_q), max_q=max_q or p.max_new, tree_mask=mask, scale=scale,
                   **kw)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    return o, lse


@pytest.mark.parametrize("ctx,new,Hq,H_kv,d,page,fmt,layout", [
    ([0], [1], 1, 1, 64, 16, "bf16", "hnd"),                        # one row, one key
    ([1000], [1], 8, 2, 128, 16, "bf16", "hnd"),                    # decoding
    ([127, 128, 129, 0, 5, 255], [1] * 6, 4, 4, 64, 16, "fp16", "nhd"),  # lengths around a key tile
    ([3000, 10, 777], [1, 1, 1], 32, 4, 128, 64, "bf16", "slice"),
    ([500, 0, 64], [5, 3, 0], 6, 2, 96, 8, "bf16", "hnd"),          # a request without new rows
    ([0, 200], [130, 70], 4, 2, 128, 32, "fp16", "nhd"),            # prompt chunks, an empty context
    ([300], [300], 5, 1, 64, 128, "bf16", "hnd"),                   # an odd group: rows of a tile end inside a token
    ([90, 2000], [17, 9], 7, 1, 32, 16, "bf16", "hnd"),
    ([40, 1500], [2, 33], 4, 2, 256, 64, "bf16", "hnd"),            # head dimension 256
    ([100], [520], 16, 2, 128, 1024, "bf16", "hnd"),                # one page larger than a key tile
    ([0], [1000], 8, 8, 64, 64, "fp16", "hnd"),
    ([9000], [1], 3, 3, 256, 16, "fp16", "hnd"),
])
def test_chain(ctx, new, Hq, H_kv, d, page, fmt, layout):
    p = Paged(ctx, new, H_kv, d, page, fmt, layout, seed=len(ctx) + d + page)
    q = queries(p, Hq)
    o, lse = attend(p, q)
    assert_attention(p, o, lse, attention_reference(p, f64(q), d ** -0.5))


@pytest.mark.parametrize("ctx,new,Hq,H_kv,d,page,fmt,layout", [
    ([200], [8], 4, 1, 128, 16, "bf16", "hnd"),
    ([0, 300, 1000], [16, 1, 40], 8, 2, 64, 16, "fp16", "nhd"),
    ([777, 5], [64, 63], 28, 4, 128, 32, "bf16", "slice"),           # trees of a whole word of mask
    ([125, 60], [65, 130], 6, 2, 96, 8, "bf16", "hnd"),             # trees across words and key tiles
    ([33], [512], 4, 4, 64, 64, "bf16", "hnd"),                     # the largest tree
    ([10, 900], [20, 7], 10, 2, 256, 16, "fp16", "hnd"),
    ([5000], [12], 8, 1, 32, 128, "fp16", "hnd"),
])
def test_tree(ctx, new, Hq, H_kv, d, page, fmt, layout):
    p = Paged(ctx, new, H_kv, d, page, fmt, layout, seed=sum(new) + d)
    bits, mask = mask_of(p, random_parents(new, p.rng))
    q = queries(p, Hq)
    o, lse = attend(p, q, mask)
    assert_attention(p, o, lse, attention_reference(p, f64(q), d ** -0.5, bits))


def test_many_requests_share_the_workers():
    rng = np.random.default_rng(5)
    ctx = [int(x) for x in np.exp(rng.uniform(0, np.log(3000), 300))]
    p = Paged(ctx, [1] * 300, 2, 64, 16, "bf16", seed=1)
    q = queries(p, 6)
    o, lse = attend(p, q)
    assert_attention(p, o, lse, attention_reference(p, f64(q), 0.125))


@pytest.mark.parametrize("d,fmt,page,Hq,H_kv,new", [(256, "fp16", 32, 56, 8, 1), (256, "bf16", 8, 16, 4, 13),
                                                    (128, "bf16", 16, 16, 4, 13), (64, "fp16", 8, 16, 8, 70)])
def test_last_tiles_under_load(d, fmt, page, Hq, H_kv, new):
    # Every SM streams and each request ends inside a tile: the rows of V behind its last key are cleared
    # while tiles before it may still be read. The same bits every time, and the oracle's values.
    rng = np.random.default_rng(d + new)
    p = Paged([int(x) for x in rng.integers(1100, 1387, 15)], [new] * 15, H_kv, d, page, fmt, seed=d)
    q = queries(p, Hq)
    o, lse = attend(p, q)
    assert_attention(p, o, lse, attention_reference(p, f64(q), d ** -0.5))
    for _ in range(20):
        again = attend(p, q)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("d,fmt,Hq,H_kv,new", [(64, "bf16", 16, 16, 40), (128, "fp16", 16, 16, 64),
                                                (256, "bf16", 16, 16, 50), (64, "fp16", 40, 8, 12)])
def test_short_units_of_two_groups(d, fmt, Hq, H_kv, new):
    # Units of 33 to 64 rows and a tile or two, many to a CTA: one group of 32 rows hands over its
    # output while the other begins the next unit.
    p = Paged([int(x) for x in np.random.default_rng(d).integers(0, 150, 40)], [new] * 40, H_kv, d, 16, fmt, seed=d)
    q = queries(p, Hq)
    o, lse = attend(p, q)
    assert_attention(p, o, lse, attention_reference(p, f64(q), d ** -0.5))
    for _ in range(50):
        again = attend(p, q)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("d,fmt,Hq,H_kv,new", [(64, "bf16", 32, 16, [400, 300, 0, 450] * 5), (256, "fp16", 16, 8, [260] * 20),
                                                (128, "bf16", 40, 8, [128, 0, 1, 260, 300] * 6)])
def test_whole_units_in_turn(d, fmt, Hq, H_kv, new):
    # Several whole units a CTA, with requests of none and of one between them.
    p = Paged([int(x) for x in np.random.default_rng(d).integers(0, 300, len(new))], new, H_kv, d, 16, fmt, seed=d)
    q = queries(p, Hq, p.T + 9)
    o, lse = attend(p, q)
    assert_attention(p, o, lse, attention_reference(p, f64(q), d ** -0.5))
    assert torch.isnan(o[p.T:]).all() and torch.isnan(lse[p.T:]).all()
    for _ in range(3):
        again = attend(p, q)
        assert torch.equal(o[:p.T], again[0][:p.T]) and torch.equal(lse[:p.T], again[1][:p.T])


def test_rows_that_see_nothing():
    # An all-zero mask over an empty context, a request that was refused (length 0), lengths below the new rows.
    p = Paged([0, 50, 0], [3, 2, 4], 2, 64, 16, "bf16", seed=3)
    q = queries(p, 4)
    bits = [np.zeros((3, 3), bool), np.eye(2, dtype=bool), np.tril(np.ones((4, 4), bool))]
    bits[0][2, 1] = True
    mask = torch.from_numpy(np.concatenate([C.pack_mask(x, 1) for x in bits])).cuda()
    o, lse = attend(p, q, mask)
    assert_attention(p, o, lse, attention_reference(p, f64(q), 0.125, bits))
    assert (o[:2] == 0).all() and torch.isneginf(lse[:2]).all()
    p.seq_len = ints([2, 0, 4])  # rows 0 of the first request and all of the second see no key
    o, lse = attend(p, q)
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all() and torch.isfinite(lse[1:3]).all()
    assert (o[3:5] == 0).all() and torch.isneginf(lse[3:5]).all() and torch.isfinite(lse[5:]).all()


def test_bad_pages_are_not_seen():
    p = Paged([500], [4], 2, 64, 16, "bf16", seed=4)
    q = queries(p, 4)
    bad = {3: -1, 9: p.num_pages, 20: 2 ** 30, 31: -2 ** 31}  # 31 holds the last rows
    table = p.table.clone()
    for i, x in bad.items():
        table[0, i] = x
    o, lse = attend(p, q, table=table)
    keep = np.array([j // 16 not in bad for j in range(504)])
    seen = C.seen_keys(4, 504) & keep
    ref = [C.tree_attention(f64(q), p.rows_of(p.k, 0), p.rows_of(p.v, 0), 0.125, seen)]
    assert_attention(p, o, lse, ref)


@pytest.mark.parametrize("d,fmt,new", [(256, "bf16", 1), (256, "fp16", 9), (64, "bf16", 40)])
def test_bad_pages_of_a_long_run_stay_with_their_tiles(d, fmt, new):
    # Tiles with and without a bad page in turn, one after the other on one CTA.
    p = Paged([5000] * 20, [new] * 20, 8, d, 32, fmt, seed=d)
    q = queries(p, 8)
    table = p.table.clone()
    table[:, 1::8] = -1  # of tiles 0, 2, 4, ... the second page
    o, lse = attend(p, q, table=table)
    n = 5000 + new
    seen = C.seen_keys(new, n) & (np.arange(n) // 32 % 8 != 1)
    for b in (0, 7, 19):
        at = slice(b * new, (b + 1) * new)
        ref = C.tree_attention(f64(q[at]), p.rows_of(p.k, b), p.rows_of(p.v, b), d ** -0.5, seen)
        assert_attention(p, o[at], lse[at], [ref])
    for _ in range(5):
        again = attend(p, q, table=table)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_table_shorter_than_the_length():
    # seq_len claims more rows than max_pages holds: what the table holds is seen.
    p = Paged([40], [1], 1, 64, 16, "bf16", spare=0, seed=6)
    q = queries(p, 1)
    p.seq_len = ints([1000])
    o, lse = attend(p, q, table=p.table[:, :2].contiguous())
    ref = [C.tree_attention(f64(q), p.rows_of(p.k, 0), p.rows_of(p.v, 0), 0.125, np.arange(41)[None, :] < 32)]
    assert_attention(p, o, lse, ref)


def test_padding_rows_and_a_larger_bound():
    # Rows behind the last request and a max_q above every request's count.
    p = Paged([70, 300], [5, 2], 2, 128, 32, "fp16", seed=7)
    q = queries(p, 8, rows=20)
    o, lse = attend(p, q, max_q=40)
    assert torch.isnan(o[7:]).all() and torch.isnan(lse[7:]).all()
    assert_attention(p, o, lse, attention_reference(p, f64(q), 128 ** -0.5))


@pytest.mark.parametrize("max_q", [3, 16, 17, 33, 65, 200])
def test_every_row_tile(max_q):
    p = Paged([260, 15], [3, 2], 1, 64, 16, "bf16", seed=8)
    q = queries(p, 1)
    o, lse = attend(p, q, max_q=max_q)
    assert_attention(p, o, lse, attention_reference(p, f64(q), 0.125))


def test_strided_queries_and_output():
    p = Paged([100, 9], [6, 30], 2, 64, 16, "bf16", seed=9)
    packed = queries(p, 4 + 2 * 2)
    q = packed[:, :4]
    out = torch.full((p.T, 2, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    o, lse = attend(p, q, o=out[:, 1])
    assert torch.isnan(out[:, 0]).all()
    assert_attention(p, o, lse, attention_reference(p, f64(q), 0.125))


@pytest.mark.parametrize("scale", [0.0, -0.25, 3.0])
def test_scales(scale):
    p = Paged([400], [3], 2, 64, 16, "bf16", seed=10)
    q = queries(p, 4)
    o, lse = attend(p, q, scale=scale)
    assert_attention(p, o, lse, attention_reference(p, f64(q), scale))


def test_growing_scores_rescale():
    # Keys whose scores grow along the sequence: the running maximum moves in tile after tile.
    p = Paged([1500], [20], 1, 64, 16, "fp16", seed=11)
    for r in range(0, 1520, 16):
        page = int(p.table_host[0, r // 16])
        p.k[page, 0] = torch.sign(p.k[page, 0]) * (0.02 * r / 16 + 0.02)
    p.k.nan_to_num_(0.0)
    q = torch.sign(p.k[int(p.table_host[0, 94]), 0]).repeat(5, 1)[:40].reshape(20, 2, 64).contiguous() * 2
    o, lse = attend(p, q)
    assert_attention(p, o, lse, attention_reference(p, f64(q), 0.125))


def test_infinite_and_nan_values_behind_the_rows():
    p = Paged([100], [5], 2, 64, 64, "bf16", seed=12)  # Paged fills the rest with NaN
    q = queries(p, 4)
    ref = attention_reference(p, f64(q), 0.125)
    assert_attention(p, *attend(p, q), ref)
    for t in (p.k, p.v):
        t[torch.isnan(t)] = float("inf")
    assert_attention(p, *attend(p, q), ref)


def test_same_result_twice_and_replayed_with_other_lengths():
    p = Paged([900, 33], [4, 4], 2, 128, 16, "bf16", seed=13)
    q = queries(p, 8)
    o1, l1 = attend(p, q)
    o2, l2 = attend(p, q)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    ws = workspace(p, 8)
    o, lse = torch.empty_like(q), torch.empty_like(l1)
    args = (q, p.k, p.v, p.table, p.seq_len, p.cu, o, lse, ws)
    fa.fa_tree_fwd(*args, max_q=4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fa_tree_fwd(*args, max_q=4)
    g2 = torch.cuda.CUDAGraph()  # a second graph on the same workspace
    with torch.cuda.graph(g2):
        fa.fa_tree_fwd(*args, max_q=4)
    for length in ([904, 37], [300, 20], [5, 4]):
        p.seq_len.copy_(ints(length))
        for graph in (g, g2):
            o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for b, n in enumerate(length):
                O, L, size, big = C.tree_attention(f64(q[4 * b:4 * b + 4]), p.rows_of(p.k, b)[:n], p.rows_of(p.v, b)[:n],
                                                   128 ** -0.5, C.seen_keys(4, n))
                assert np.abs(f64(o[4 * b:4 * b + 4]) - O).max() < 0.02
    p.seq_len.copy_(ints([904, 37]))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, o1) and torch.equal(lse, l1)


def test_on_another_stream():
    p = Paged([600], [8], 2, 64, 16, "bf16", seed=14)
    q = queries(p, 4)
    want = attend(p, q)
    st = torch.cuda.Stream()
    o, lse = torch.empty_like(q), torch.empty_like(want[1])
    ws = workspace(p, 4)
    st.wait_stream(torch.cuda.current_stream())
    fa.fa_tree_fwd(q, p.k, p.v, p.table, p.seq_len, p.cu, o, lse, ws, max_q=8, stream=st)
    st.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_two_calls_at_once():
    a, b = (Paged([3000, 20], [6, 6], 2, 128, 16, "bf16", seed=s) for s in (15, 16))
    qa, qb = queries(a, 8), queries(b, 8)
    want = [attend(a, qa), attend(b, qb)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    out = []
    torch.cuda.synchronize()
    bufs = [(torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), workspace(p, 8))
            for p, q in ((a, qa), (b, qb))]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, p, q, (o, lse, ws) in zip(streams, (a, b), (qa, qb), bufs):
            fa.fa_tree_fwd(q, p.k, p.v, p.table, p.seq_len, p.cu, o, lse, ws, max_q=6, stream=st)
    torch.cuda.synchronize()
    for (o, lse, _), w in zip(bufs, want):
        assert torch.equal(o, w[0]) and torch.equal(lse, w[1])


def test_agrees_with_the_contiguous_forward():
    # One page run in order is the contiguous layout: fa_fwd_qk on the same keys.
    B, H, n, length, d = 1, 4, 40, 1000, 128
    p = Paged([length - n], [n], H, d, 8, "bf16", seed=17)
    q = queries(p, H)
    o, lse = attend(p, q)
    k, v = (torch.stack([t[int(x)] for x in p.table_host[0, :125]], 1).reshape(1, H, length, d) for t in (p.k, p.v))
    qq = q.transpose(0, 1)[None].contiguous()
    o2, lse2 = torch.empty_like(qq), torch.empty((1, H, n), device="cuda")
    fa.fa_fwd_qk(qq, k.contiguous(), v.contiguous(), o2, lse2, causal=True)
    torch.cuda.synchronize()
    assert (o.float() - o2[0].transpose(0, 1).float()).abs().max() < 5e-3  # both round P and O once: 4 half steps
    assert (lse - lse2[0].t()).abs().max() < 1e-4


def test_offsets_beyond_32_bits():
    # A cache of more than 2^32 elements whose used pages lie at its end.
    pages, H, page, d = 70000, 4, 128, 128
    k = torch.zeros((pages, H, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 2 ** 32
    p = Paged([200], [3], H, d, page, "bf16", seed=18)
    q = queries(p, 8)
    where = [pages - 1, pages - 2]
    for src, dst in ((p.k, k), (p.v, v)):
        for i, at in enumerate(where):
            dst[at] = src[int(p.table_host[0, i])]
    o, lse = attend(p, q)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    fa.fa_tree_fwd(q, k, v, ints([where]), p.seq_len, p.cu, o2, lse2, workspace(p, 8), max_q=3)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d,Hq,max_q", [(64, 2, 2), (128, 8, 20), (256, 4, 40), (128, 8, 200)])
def test_waits_that_run_out_end_the_call(d, Hq, max_q):
    # No load is issued, so the waits reach their limit: the call ends, the status tells, and the
    # next call works.
    import ctypes
    p = Paged([700, 5, 0], [max_q, 1, 2], 2, d, 16, "bf16", seed=19)
    q = queries(p, Hq)
    want = attend(p, q)
    o, lse, ws = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda"), workspace(p, Hq)
    desc = fa.KVCacheDesc(p.k.data_ptr(), p.v.data_ptr(), fa.FA_BF16, p.num_pages, 16, 2, d, *p.k.stride()[:3])
    rows = [fa.RowsDesc(t.data_ptr(), Hq * d, d) for t in (q, o)]
    st = fa.load_library().fa_debug_tree_withhold(
        ctypes.byref(desc), *(ctypes.byref(r) for r in rows), lse.data_ptr(), 3, p.T, max_q, Hq, p.table.shape[1],
        p.table.data_ptr(), p.cu.data_ptr(), p.seq_len.data_ptr(), None, d ** -0.5, ws.data_ptr(), 20,
        torch.cuda.current_stream().cuda_stream)
    assert st == fa.FA_OK
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_ERR_TIMEOUT
    assert fa.fa_device_status() == fa.FA_OK
    again = attend(p, q)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
