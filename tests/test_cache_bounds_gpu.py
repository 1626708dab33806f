"""Steps whose rows do not fit the buffers they are given, PagedCache's optional buffers, rotations on
another stream."""
import numpy as np
import pytest
import torch

import io_aware_exact_19_b200 as fa
from tests.cache_cases import Paged, assert_attention, attention_reference, f64, ints, random_parents
from tests.test_cache_gpu import State
from tests.test_tree_gpu import attend, mask_of, queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("new,rows", [([8, 8, 8], 20), ([8, 8, 8], 16), ([30, 1, 0], 29), ([5, 0, 9, 0, 1], 13), ([3], 0)])
def test_plan_refuses_rows_behind_the_buffers(new, rows, tree):
    st = State(len(new), 8, 40)
    parent = random_parents(new, np.random.default_rng(rows))[:rows] if tree else None
    ctx = [3 * b for b in range(len(new))]
    st.step(ctx, [0] * len(new), 8, 32, rows, [-1] * rows if tree else None)  # pages of the cached rows
    seq = st.step(ctx, new, 8, 32, rows, parent)
    ends = np.cumsum(new)
    assert seq == [c + n if n == 0 or e <= rows else 0 for c, n, e in zip(ctx, new, ends)]


def test_plan_refuses_broken_offsets_and_writes_inside():
    # Offsets that fall or point outside the rows: the requests outside are refused, no page is lost or given
    # out twice, and nothing around the outputs is written.
    for cu, seq_want in (([-5, -2, 1, 4], [0, 0, 4]), ([0, 2, 4, 100], [3, 3, 0]), ([0, 2, 4, 7], [3, 3, 0]),
                         ([2, 3, 6, 6], [2, 4, 1]), ([0, 4, 2, 6], [5, 0, 5]), ([7, 8, 8, 9], [0, 1, 0])):
        wide = lambda n, fill, dtype=torch.int32: torch.full((n + 16,), fill, dtype=dtype, device="cuda")  # noqa: E731
        pads = [wide(6, 77), wide(6, 77), wide(6, 77, torch.int64), wide(3, 77), wide(3, 77), wide(12, -1)]
        slot, pos, mask, seq, held, table = (x[8:-8] for x in pads)
        held.zero_()
        free, count = ints(range(12)), ints([12])
        fa.fa_cache_plan(ints([1, 1, 1]), ints(cu), table.view(3, 4), held, free, count, seq, slot, pos, page_size=8,
                         max_new=8, parent=ints([-1] * 6), tree_mask=mask.view(6, 1))
        torch.cuda.synchronize()
        for x, fill in zip(pads, (77, 77, 77, 77, 77, -1)):
            assert (x[:8] == fill).all() and (x[-8:] == fill).all(), cu
        assert seq.tolist() == seq_want, cu
        pages = [table.view(3, 4)[b, i].item() for b in range(3) for i in range(held[b].item())]
        assert sorted(pages + free[:count.item()].tolist()) == list(range(12)), cu
        assert slot.max() < 96 and slot.min() >= -1


def test_a_step_of_too_many_rows_leaves_the_request_as_it_was():
    # Three requests of 8 rows and buffers for 20: the third is refused whole, eagerly and in a replayed graph,
    # and goes on from where it was in the next step.
    cache = fa.PagedCache(num_pages=40, page_size=8, batch=3, max_len=100, H_kv=1, d=64, max_rows=20, max_new=8)
    x = torch.randn((20, 1, 64), device="cuda").to(torch.bfloat16)
    o, lse = torch.zeros_like(x), torch.zeros((20, 1), device="cuda")
    new = ints([5, 5, 5])

    def step():
        cache.plan(new)
        cache.append(0, x, x, x)
        cache.attend(0, x, o=o, lse=lse)
        cache.keep()

    step()
    assert cache.ctx_len.tolist() == [5, 5, 5]
    new.copy_(ints([8, 8, 8]))
    step()
    torch.cuda.synchronize()
    assert cache.seq_len.tolist() == [13, 13, 0] and cache.ctx_len.tolist() == [13, 13, 5]
    assert torch.isfinite(o[:16].float()).all() and torch.isneginf(lse[16:]).all() and (o[16:] == 0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n, want in (([8, 8, 8], [21, 21, 5]), ([1, 1, 8], [22, 22, 13]), ([8, 0, 13], [30, 22, 13]), ([0, 8, 8], [30, 30, 21])):
        new.copy_(ints(n))
        graph.replay()
        torch.cuda.synchronize()
        assert cache.ctx_len.tolist() == want
    held = sum(cache.n_pages.tolist())
    assert cache.free_count.item() + held == 40 and held == sum(-(-c // 8) for c in cache.ctx_len.tolist())


@pytest.mark.parametrize("ctx,new,rows,Hq,H_kv,d,tree", [
    ([40, 300], [6, 9], 11, 4, 2, 64, False), ([40, 300], [6, 9], 11, 4, 2, 64, True),
    ([200, 90], [3, 60], 40, 8, 2, 128, False), ([200, 90], [3, 60], 40, 8, 2, 128, True),
    ([50, 130], [7, 30], 12, 2, 1, 256, False), ([500, 300, 700], [200, 333, 300], 700, 32, 8, 64, False),
])
def test_rows_behind_the_batch_leave_the_others_in_their_places(ctx, new, rows, Hq, H_kv, d, tree):
    # cu_q goes beyond the rows that are given: those there are the first of their request, not the last.
    p = Paged(ctx, new, H_kv, d, 16, "bf16", seed=rows)
    bits, mask = mask_of(p, random_parents(new, p.rng)) if tree else (None, None)
    q = queries(p, Hq)
    ref = attention_reference(p, f64(q), d ** -0.5, bits)
    o, lse = attend(p, q[:rows], None if mask is None else mask[:rows].contiguous())
    there = [max(0, min(n, rows - int(t0))) for n, t0 in zip(new, p.cu_host)]
    p.new = there
    assert sum(there) == rows
    assert_attention(p, o, lse, [(O[:m], L[:m], size[:m], big) for m, (O, L, size, big) in zip(there, ref)])


def test_append_without_a_rotation_fills_the_buffer():
    # A step with fixed buffers reads its queries there, rotated or not.
    cache = fa.PagedCache(num_pages=4, page_size=16, batch=1, max_len=64, H_kv=1, d=64, max_rows=6, max_new=6)
    packed = torch.randn((6, 6, 64), device="cuda").to(torch.bfloat16)
    q, k, v = packed.split([4, 1, 1], 1)
    q_out = torch.full((6, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    cache.plan(ints([6]))
    assert cache.append(0, q, k, v, q_out=q_out) is q_out and torch.equal(q_out, q)
    first = cache.block_table[0, 0].item()
    assert torch.equal(cache.k[0, first, 0, :6], k[:, 0]) and torch.equal(cache.v[0, first, 0, :6], v[:, 0])
    assert cache.append(0, q, k, v) is q


def test_rotation_on_another_stream_takes_no_memory_still_in_use():
    # A freed block of the current stream is still to be written there; the rotated tensor, written on another
    # stream at once, must not lie in it, and must not be handed out again before its own work is done.
    rope = fa.Rope(*fa.rope_tables(64), positions=torch.arange(512, dtype=torch.int32, device="cuda")[None])
    x = torch.randn((2, 4, 512, 64), device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    want, minus, after = rope.turn(x), -x, torch.empty_like(x)
    rope.turn(x, after)
    torch.cuda.synchronize()
    old = torch.empty_like(x)
    where = old.data_ptr()
    torch.cuda._sleep(100_000_000)  # some 50 ms
    old.fill_(7.0)
    del old
    out = rope.turn(x, stream=side)
    assert out.data_ptr() != where
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # used on the current stream and let go: the block waits for that use
    side.synchronize()
    torch.cuda._sleep(100_000_000)
    after.copy_(out)
    del out
    again = rope.turn(minus, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(after, want) and torch.equal(again, -want)


def test_attention_with_rotation_on_another_stream():
    rope = fa.Rope(*fa.rope_tables(64), positions=torch.arange(300, dtype=torch.int32, device="cuda")[None])
    q, k, v, do = (torch.randn((1, 2, 300, 64), device="cuda").to(torch.bfloat16) for _ in range(4))
    o, lse = fa.attention_forward(q, k, v, causal=True, rope=rope)
    want = (o, lse, *fa.attention_backward(q, k, v, o, lse, do, causal=True, rope=rope))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, lse = fa.attention_forward(q, k, v, causal=True, rope=rope, stream=side)
    workspace = torch.empty(fa.fa_bwd_workspace_size(1, 2, 300, 64), dtype=torch.uint8, device="cuda")
    got = (o, lse, *fa.attention_backward(q, k, v, o, lse, do, causal=True, rope=rope, workspace=workspace, stream=side))
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_backward_on_another_stream_keeps_its_workspace_to_itself(monkeypatch):
    # The workspace that the call makes is let go at its end, with its kernels still to run (here: none is
    # launched): the current stream must not get that memory.
    q, k, v, do, o = (torch.zeros((1, 2, 256, 64), dtype=torch.bfloat16, device="cuda") for _ in range(5))
    lse, side, seen = torch.zeros((1, 2, 256), device="cuda"), torch.cuda.Stream(), []
    monkeypatch.setattr(fa, "fa_bwd", lambda *a: seen.append((a[9].data_ptr(), a[9].numel())))
    fa.attention_backward(q, k, v, o, lse, do, stream=side)
    (at, size), = seen
    assert size == fa.fa_bwd_workspace_size(1, 2, 256, 64)
    assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() != at
    with torch.cuda.stream(side):
        assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() == at
