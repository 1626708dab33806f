"""fa_cache_plan and fa_cache_commit against the host oracle, exactly."""
import numpy as np
import pytest
import torch

import io_aware_exact_19_b200 as fa
from oracle import cache as C
from tests.cache_cases import Paged, f64, ints, random_parents

pytestmark = pytest.mark.gpu


class State:
    def __init__(self, B, width, P, seed=0):
        self.table = [[-1] * width for _ in range(B)]
        self.held, self.count = [0] * B, P
        self.free = [int(x) for x in np.random.default_rng(seed).permutation(P)]
        self.dev = [ints(self.table), ints(self.held), ints(self.free), ints([P])]

    def step(self, ctx, new, page, max_new, rows, parent=None):
        B = len(ctx)
        cu = np.concatenate([[0], np.cumsum(new)]).astype(int).tolist()
        want = C.plan(ctx, cu, self.table, self.held, self.free, self.count, page, rows, max_new, parent)
        table, held, free, count = self.dev
        seq = torch.full((B,), -7, dtype=torch.int32, device="cuda")
        slot, pos = (torch.full((rows,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
        mask = up = None
        if parent is not None:
            mask = torch.full((rows, -(-max_new // 64)), -7, dtype=torch.int64, device="cuda")
            up = ints(list(parent) + [0] * (rows - len(parent)))
        fa.fa_cache_plan(ints(ctx), ints(cu), table, held, free, count, seq, slot, pos, page_size=page, max_new=max_new,
                         parent=up, tree_mask=mask)
        torch.cuda.synchronize()
        self.table, self.held, self.free, self.count = want[:4]
        assert table.tolist() == want[0] and held.tolist() == want[1] and count.item() == want[3]
        assert free[:want[3]].tolist() == want[2][:want[3]]
        assert seq.tolist() == want[4] and slot.tolist() == want[5] and pos.tolist() == want[6]
        if mask is not None:
            got = mask.cpu().numpy()
            for t in range(rows):
                assert np.array_equal(got[t], want[7][t] if t in want[7] else np.full_like(got[t], -7)), t
        return want[4]


@pytest.mark.parametrize("B,page,P,tree,max_new", [
    (1, 16, 8, False, 1), (3, 8, 30, True, 5), (8, 16, 100, True, 33), (37, 64, 60, False, 100), (5, 8, 400, True, 512),
    (600, 16, 2000, False, 3), (700, 32, 900, True, 64), (4096, 8, 9000, False, 2),
])
def test_plan_follows_the_oracle(B, page, P, tree, max_new):
    # Several steps on one state: requests grow, are refused when pages run out, shrink and finish.
    rng = np.random.default_rng(B + page)
    width = 12 if B > 5 else 80
    st = State(B, width, P, seed=B)
    ctx = [0] * B
    for step in range(6):
        new = rng.integers(0 if step else 1, max_new + 1, B)
        new[rng.integers(0, B)] = max_new
        parent = None
        if tree:
            parent = random_parents(new, rng)
            parent = [p if rng.random() < 0.98 else 9999 for p in parent]
        seq = st.step(ctx, new.tolist(), page, max_new, int(new.sum()) + (step % 2) * 3, parent)
        ctx = [0 if rng.random() < 0.3 else max(0, s - int(rng.integers(0, 3))) for s in seq]


def test_plan_refuses_what_does_not_fit():
    st = State(5, 4, 6)
    # more pages than a table row; a negative context; more new rows than max_new; then one that fits, one that does not
    st.step([100, -3, 0, 20, 0], [1, 1, 9, 4, 20], 8, 8 + 12, 40)
    st = State(3, 4, 6)
    st.step([8, 0, 0], [16, 30, 1], 8, 30, 47)   # 3 pages, 4 (refused: 7 > 6), then the third is refused too
    st.step([0, 0, 0], [0, 30, 1], 8, 30, 31)    # the first gives its pages back: both fit
    st.step([0, 0, 0], [0, 0, 0], 8, 30, 0)      # everything back, no rows
    assert st.count == 6 and st.dev[0].eq(-1).all()


def test_plan_with_broken_offsets_writes_inside():
    # Offsets that fall or point outside the rows: no slot, and nothing outside is written.
    table, held, free, count = ints([[-1] * 4] * 3), ints([0] * 3), ints(range(12)), ints([12])
    seq, slot, pos = ints([0] * 3), ints([5] * 6), ints([5] * 6)
    mask = torch.zeros((6, 1), dtype=torch.int64, device="cuda")
    for cu in ([0, 4, 2, 6], [-5, -2, 1, 9], [0, 2, 4, 100]):
        fa.fa_cache_plan(ints([1, 1, 1]), ints(cu), table, held, free, count, seq, slot, pos, page_size=8, max_new=8,
                         parent=ints([-1] * 6), tree_mask=mask)
        torch.cuda.synchronize()
        assert slot.max() < 96


def test_plan_in_a_graph():
    B, page = 4, 16
    st = State(B, 8, 40)
    ctx, cu = ints([0] * B), ints([0, 3, 3, 7, 9])
    seq, slot, pos = ints([0] * B), ints([0] * 9), ints([0] * 9)
    args = (ctx, cu, *st.dev, seq, slot, pos)
    fa.fa_cache_plan(*args, page_size=page, max_new=8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa.fa_cache_plan(*args, page_size=page, max_new=8)
    host = C.plan([0] * B, cu.tolist(), st.table, st.held, st.free, st.count, page, 9, 8)
    for ctx_now in ([3, 0, 20, 2], [70, 0, 0, 31]):
        ctx.copy_(ints(ctx_now))
        g.replay()
        torch.cuda.synchronize()
        host = C.plan(ctx_now, cu.tolist(), *host[:4], page, 9, 8)
        assert st.dev[0].tolist() == host[0] and slot.tolist() == host[5] and st.dev[3].item() == host[3]


@pytest.mark.parametrize("fmt,d,page,H_kv,layout", [("bf16", 128, 16, 2, "hnd"), ("fp16", 96, 8, 3, "nhd"),
                                                    ("bf16", 256, 64, 1, "slice"), ("bf16", 32, 1024, 5, "hnd")])
def test_commit(fmt, d, page, H_kv, layout):
    rng = np.random.default_rng(d)
    new = [1, 20, 64, 300, 7, 5]
    p = Paged([0, 5, 100, 30, 15, 9], new, H_kv, d, page, fmt, layout, seed=d)
    width = 200
    accepted = np.full((6, width), -1)
    count = []
    for b, n in enumerate(new):
        c = int(rng.integers(1, min(n, width) + 1)) if b else 1
        accepted[b, :c] = np.sort(rng.choice(n, c, replace=False))
        count.append(c)
    accepted[2, :5] = np.arange(5)       # a path that stays where it is
    accepted[4, :4] = [2, 2, 5, 6]       # the same index twice: the path ends there
    count[4], count[5] = 4, 0            # nothing accepted
    new_len = torch.zeros(6, dtype=torch.int32, device="cuda")
    before = [[p.rows_of(t, b) for b in range(6)] for t in (p.k, p.v)]
    stale = [torch.isnan(t).sum().item() for t in (p.k, p.v)]
    fa.fa_cache_commit(p.k, p.v, p.table, ints(p.ctx), ints(accepted), ints(count), new_len)
    torch.cuda.synchronize()
    for t, rows, nan in zip((p.k, p.v), before, stale):
        for b in range(6):
            want = rows[b].copy()
            kept = C.commit(want, p.ctx[b], accepted[b, :count[b]])
            assert new_len[b].item() == kept
            assert np.array_equal(p.rows_of(t, b), want), b
        assert torch.isnan(t).sum().item() == nan


def test_commit_in_place_length_and_missing_pages():
    p = Paged([20, 20], [12, 12], 1, 64, 8, "bf16", seed=2)
    ctx = ints(p.ctx)
    table = p.table.clone()
    table[1, 3] = -1  # rows 24..31 of the second request
    keep = [p.rows_of(p.k, b) for b in range(2)]
    fa.fa_cache_commit(p.k, p.v, table, ctx, ints([[1, 3, 11], [2, 3, 11]]), ints([3, 3]), ctx)
    torch.cuda.synchronize()
    assert ctx.tolist() == [23, 22]  # the second path stops at row 31
    got = p.rows_of(p.k, 0)
    assert np.array_equal(got[20:23], keep[0][[21, 23, 31]])
    assert np.array_equal(p.rows_of(p.k, 1)[20:22], keep[1][[22, 23]])
