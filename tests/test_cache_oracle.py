"""Pins of the paged-cache oracle (CPU): its attention against the contiguous oracle, its
rotation against complex multiplication and finite differences, its bookkeeping by invariants."""
import numpy as np
import pytest

import oracle
from oracle import cache as C


def test_chain_attention_is_the_causal_forward():
    rng = np.random.default_rng(0)
    n, length, H, d = 5, 12, 4, 8
    q, k, v = rng.standard_normal((n, H, d)), rng.standard_normal((length, 2, d)), rng.standard_normal((length, 2, d))
    o, lse, _, _ = C.tree_attention(q, k, v, 0.3, C.seen_keys(n, length))
    kk, vv = np.repeat(k, 2, 1).transpose(1, 0, 2), np.repeat(v, 2, 1).transpose(1, 0, 2)
    O, L = oracle.forward(q.transpose(1, 0, 2), kk, vv, 0.3, causal=True)
    assert np.allclose(o.transpose(1, 0, 2), O, atol=1e-13) and np.allclose(lse.T, L, atol=1e-13)


def test_a_path_of_a_tree_attends_like_a_chain():
    # Token by token along one branch, the tree's rows equal a chain over the context and that branch.
    rng = np.random.default_rng(1)
    parent = [-1, 0, 0, 1, 2, 3, -1]
    n, ctx, d = len(parent), 6, 8
    q, k, v = (rng.standard_normal((m, 1, d)) for m in (n, ctx + n, ctx + n))
    bits = C.ancestors(parent)
    o, lse, _, _ = C.tree_attention(q, k, v, 0.5, C.seen_keys(n, ctx + n, bits))
    for t in range(n):
        keys = list(range(ctx)) + [ctx + j for j in range(n) if bits[t, j]]
        O, L, _, _ = C.tree_attention(q[t:t + 1], k[keys], v[keys], 0.5, np.ones((1, len(keys)), bool))
        assert np.allclose(o[t], O[0], atol=1e-13) and np.allclose(lse[t], L[0], atol=1e-13)
    assert bits[5].tolist() == [True, True, False, True, False, True, False]


def test_ancestors_ignore_parents_out_of_range():
    assert np.array_equal(C.ancestors([5, 1, 0, -7]), [[1, 0, 0, 0], [0, 1, 0, 0], [1, 0, 1, 0], [0, 0, 0, 1]])


def test_pack_mask():
    bits = np.zeros((1, 70), bool)
    bits[0, [0, 63, 64, 69]] = True
    assert C.pack_mask(bits, 2).view(np.uint64).tolist() == [[1 + (1 << 63), 1 + (1 << 5)]]


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_is_a_rotation_and_its_inverse_the_gradient(pairs):
    rng = np.random.default_rng(2)
    n, d, half = 3, 12, 4
    x, g = rng.standard_normal((n, d)), rng.standard_normal((n, d))
    pos, inv, axis = rng.integers(0, 50, (2, n)), np.array([1.0, 0.3, 0.1, 0.02]), [0, 1, 1, 0]
    y = C.rope(x, pos, inv, axis, pairs=pairs)
    a, b = (slice(0, 8, 2), slice(1, 8, 2)) if pairs else (slice(0, 4), slice(4, 8))
    z = (x[:, a] + 1j * x[:, b]) * np.exp(1j * pos[axis].T * inv)
    assert np.allclose(y[:, a], z.real) and np.allclose(y[:, b], z.imag) and np.array_equal(y[:, 8:], x[:, 8:])
    dx = C.rope(g, pos, inv, axis, inverse=True, pairs=pairs)
    for _ in range(6):
        e = rng.standard_normal((n, d))
        num = ((C.rope(x + 1e-5 * e, pos, inv, axis, pairs=pairs) - C.rope(x - 1e-5 * e, pos, inv, axis, pairs=pairs))
               * g).sum() / 2e-5
        assert abs(num - (dx * e).sum()) < 1e-8


def test_plan_hands_out_each_page_once():
    rng = np.random.default_rng(3)
    B, page, P, width = 6, 8, 40, 12
    table, held, free, count = [[-1] * width for _ in range(B)], [0] * B, list(range(P)), P
    ctx = [0] * B
    for _ in range(30):
        new = rng.integers(0, 20, B)
        cu = [0] + np.cumsum(new).tolist()
        table, held, free, count, seq, slot, pos, _ = C.plan(ctx, cu, table, held, free, count, page, cu[-1] + 2, 32)
        owned = [table[b][i] for b in range(B) for i in range(held[b])]
        assert sorted(owned + free[:count]) == list(range(P))
        used = [s for s in slot if s >= 0]
        assert len(set(used)) == len(used) and all(table[b][i] == -1 for b in range(B) for i in range(held[b], width))
        ctx = [0 if rng.random() < 0.3 else min(int(s), 60) for s in seq]


def test_plan_refuses_rows_behind_the_buffers():
    # 20 rows for 3 x 8 new tokens: the third request keeps its pages and length, its rows get no slot, and one
    # without new rows behind it is served.
    args = [[5, 5, 5, 5], [0, 8, 16, 24, 24], [[0, -1], [1, -1], [2, -1], [3, -1]], [1] * 4, [4, 5, 6] + [-1] * 4, 3, 8, 20, 8]
    table, held, _, count, seq, slot, pos, mask = C.plan(*args, parent=[-1] * 20)
    assert seq == [13, 13, 0, 5] and held == [2, 2, 1, 1] and count == 1 and table[2] == [2, -1]
    assert slot[:8] == [5, 6, 7, 48, 49, 50, 51, 52] and slot[16:] == [-1] * 4 and pos[16:] == [5] * 4 and len(mask) == 20


def test_commit_moves_a_path():
    rows = np.arange(10)
    assert C.commit(rows, 3, [1, 2, 5]) == 6 and rows.tolist() == [0, 1, 2, 4, 5, 8, 6, 7, 8, 9]
    assert C.commit(np.arange(10), 3, [2, 2, 5]) == 4
