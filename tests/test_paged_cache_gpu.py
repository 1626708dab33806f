"""The paged-cache operators together, as a serving program uses them (PagedCache), and the rotation
in the training path, each against a plain computation in float64."""
import numpy as np
import pytest
import torch

import io_aware_exact_19_b200 as fa
import oracle
from oracle import cache as C
from tests.cache_cases import DT, f64, ints, random_parents
from tests.gpu_inputs import Case, assert_grads, max_abs

pytestmark = pytest.mark.gpu


class Plain:
    """The same requests as growing float64 arrays of rotated K and V."""

    def __init__(self, batch, layers, H_kv, d):
        self.k = [[np.zeros((0, H_kv, d)) for _ in range(batch)] for _ in range(layers)]
        self.v = [[np.zeros((0, H_kv, d)) for _ in range(batch)] for _ in range(layers)]


def _step(cache, plain, rng, new, fmt, Hq, rope, tables, accept=None, pad=0, most=None):
    """One step of all layers; returns nothing, asserts every output. With `accept` (a function of the
    tree sizes) the new rows are drafted trees of which a path is kept."""
    layers, _, H_kv, _, d = cache.k.shape
    ctx = [len(x) for x in plain.k[0]]
    T = int(sum(new))
    cu = np.concatenate([[0], np.cumsum(new)])
    parents = random_parents(new, rng) if accept else None
    cache.plan(ints(new), None if parents is None else ints(parents), most=most)
    bits = [C.ancestors(parents[cu[b]:cu[b + 1]]) if accept else None for b in range(len(new))]
    pos = np.concatenate([ctx[b] + (np.arange(n) if bits[b] is None else bits[b].sum(1) - 1) for b, n in enumerate(new)])
    assert cache.position[:T].tolist() == pos.tolist()
    assert cache.seq_len.tolist() == [c + n for c, n in zip(ctx, new)]
    inv, axis, axes = tables
    for layer in range(layers):
        packed = torch.from_numpy(rng.standard_normal((T + pad, Hq + 2 * H_kv, d))).to(DT[fmt]).cuda()
        q, k, v = packed.split([Hq, H_kv, H_kv], 1)
        q_out = cache.append(layer, q, k, v, rope)
        o, lse = cache.attend(layer, q_out)
        torch.cuda.synchronize()
        assert fa.fa_device_status() == fa.FA_OK
        at = np.stack([pos] * axes)[:, :, None]
        u = torch.finfo(DT[fmt]).eps / 2
        K = C.rope(f64(k)[:T], at, inv, axis)
        for b, n in enumerate(new):
            # the kernels round the rotated rows once; the reference goes on with what they hold
            held = torch.stack([cache.k[layer][int(s) // cache.page_size, :, int(s) % cache.page_size]
                                for s in cache.slot[cu[b]:cu[b + 1]].tolist()]) if n else None
            if n:
                got = f64(held)
                assert (np.abs(got - K[cu[b]:cu[b + 1]]) <= u * np.abs(K[cu[b]:cu[b + 1]]) * 1.01 + 1e-5).all()
                plain.k[layer][b] = np.concatenate([plain.k[layer][b], got])
                plain.v[layer][b] = np.concatenate([plain.v[layer][b], f64(v)[cu[b]:cu[b + 1]]])
            L = ctx[b] + n
            O, LSE, size, big = C.tree_attention(f64(q_out)[cu[b]:cu[b + 1]], plain.k[layer][b], plain.v[layer][b],
                                                 d ** -0.5, C.seen_keys(n, L, bits[b]))
            score = 2.0 ** -24 * (d * big + 16)
            err = np.abs(f64(o[cu[b]:cu[b + 1]]) - O)
            assert (err <= (2 * u + 4 * score + 2 ** -17) * size * 1.01 + 1e-5).all(), (layer, b, err.max())
            assert max_abs(f64(lse[cu[b]:cu[b + 1]]), LSE) <= 1e-4
    if accept is None:
        cache.keep()
        return
    count, rows = [], np.full((len(new), 12), -1)
    for b, n in enumerate(new):
        path = np.flatnonzero(bits[b][int(rng.integers(0, n))])[:12] if n else []
        rows[b, :len(path)] = path
        count.append(len(path))
        for layer in range(layers):
            for x in (plain.k[layer], plain.v[layer]):
                x[b] = np.concatenate([x[b][:ctx[b]], x[b][ctx[b]:][list(path)]])
    cache.commit(ints(rows), ints(count))
    assert cache.ctx_len.tolist() == [len(x) for x in plain.k[0]]


@pytest.mark.parametrize("fmt,d,page,H_kv,Hq,sections", [("bf16", 128, 16, 2, 8, None), ("fp16", 64, 8, 1, 5, [8, 12, 12]),
                                                         ("bf16", 96, 64, 3, 3, [16, 32])])
def test_serving(fmt, d, page, H_kv, Hq, sections):
    rng = np.random.default_rng(d)
    batch, layers = 5, 2
    cache = fa.PagedCache(num_pages=1200 // page + 6, page_size=page, batch=batch, max_len=400, H_kv=H_kv, d=d,
                          max_rows=700, max_new=200, layers=layers, dtype=DT[fmt])
    inv_freq, axis = fa.rope_tables(2 * sum(sections) if sections else d, sections, base=500000.0)
    rope = fa.Rope(inv_freq, axis)
    tables = inv_freq.cpu().numpy(), axis.cpu().numpy(), 8
    plain = Plain(batch, layers, H_kv, d)
    args = (cache, plain, rng)
    _step(*args, [130, 1, 77, 0, 5], fmt, Hq, rope, tables)                                  # prompts
    _step(*args, [1, 1, 1, 0, 1], fmt, Hq, rope, tables, pad=3, most=1)                      # decoding, a padded batch
    for most in (70, 128):
        _step(*args, [9, 20, 70, 0, 3], fmt, Hq, rope, tables, accept=True, most=most)       # drafted trees
    cache.release(2)                                                                         # one is done, one begins
    for layer in range(layers):
        plain.k[layer][2] = plain.k[layer][2][:0]
        plain.v[layer][2] = plain.v[layer][2][:0]
    _step(*args, [1, 30, 0, 200, 1], fmt, Hq, rope, tables)
    _step(*args, [4, 1, 33, 8, 64], fmt, Hq, rope, tables, accept=True)
    held = sum(cache.n_pages.tolist())
    assert cache.free_count.item() + held == cache.free_list.numel()
    used = [x for row, n in zip(cache.block_table.tolist(), cache.n_pages.tolist()) for x in row[:n]]
    assert len(set(used)) == held


def test_a_refused_request_waits():
    cache = fa.PagedCache(num_pages=4, page_size=16, batch=2, max_len=64, H_kv=1, d=64, max_rows=80, max_new=64)
    x = torch.randn((80, 1, 64), device="cuda").to(torch.bfloat16)
    cache.plan(ints([40, 40]))  # 3 + 3 pages, 4 are there
    cache.append(0, x, x, x)
    o, lse = cache.attend(0, x)
    cache.keep()
    torch.cuda.synchronize()
    assert cache.seq_len.tolist() == [40, 0] and cache.ctx_len.tolist() == [40, 0]
    assert torch.isfinite(lse[:40]).all() and torch.isneginf(lse[40:]).all() and (o[40:] == 0).all()
    cache.release(0)
    cache.plan(ints([0, 40]))
    assert cache.seq_len.tolist() == [0, 40] and cache.free_count.item() == 1


def test_a_refused_draft_keeps_nothing():
    # Its pages would hold the first of the rows that it claims, but no row was written.
    cache = fa.PagedCache(num_pages=2, page_size=16, batch=2, max_len=64, H_kv=1, d=64, max_rows=50, max_new=40)
    x = torch.randn((50, 1, 64), device="cuda").to(torch.bfloat16)
    cache.plan(ints([5, 5]))
    cache.append(0, x[:10], x[:10], x[:10])
    cache.keep()
    before = cache.k.clone()
    cache.plan(ints([4, 30]), parent=ints([-1, 0, 1, 0] + list(range(-1, 29))))
    cache.append(0, x[:34], x[:34], x[:34])
    assert cache.seq_len.tolist() == [9, 0]
    second = cache.block_table[1, 0].item()
    cache.commit(ints([[0, 3], [0, 1]]), ints([2, 2]))
    assert cache.ctx_len.tolist() == [7, 5] and torch.equal(cache.k[:, second, :, :5], before[:, second, :, :5])


def test_a_step_in_a_graph():
    # Captured once, replayed while the sequences grow; the same steps run eagerly give the same bits.
    def make():
        torch.manual_seed(0)
        return fa.PagedCache(num_pages=64, page_size=16, batch=3, max_len=200, H_kv=2, d=64, max_rows=12, max_new=4)
    rope = fa.Rope(*fa.rope_tables(64))
    g = torch.Generator(device="cuda").manual_seed(3)
    steps = [torch.randn((12, 8, 64), generator=g, device="cuda").to(torch.bfloat16) for _ in range(5)]
    new = [ints([4, 2, 3]), ints([1, 4, 4]), ints([4, 4, 4]), ints([0, 1, 2]), ints([2, 2, 2])]

    def step(cache, x, n, q_out, o, lse):
        q, k, v = x.split([4, 2, 2], 1)
        cache.plan(n)
        cache.append(0, q, k, v, rope, q_out=q_out)
        cache.attend(0, q_out, o=o, lse=lse)
        cache.keep()

    def buffers():
        return (torch.zeros((12, 4, 64), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((12, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((12, 4), device="cuda"))

    eager, want = make(), []
    q_out, o, lse = buffers()
    for x, n in zip(steps, new):
        step(eager, x, n, q_out, o, lse)
        torch.cuda.synchronize()
        want.append((o.clone(), lse.clone(), eager.ctx_len.tolist()))
    cache = make()
    q_out, o, lse = buffers()
    x, n = steps[0].clone(), new[0].clone()
    step(cache, x, n, q_out, o, lse)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, x, n, q_out, o, lse)
    for i in range(1, 5):
        x.copy_(steps[i])
        n.copy_(new[i])
        graph.replay()
        torch.cuda.synchronize()
        rows = int(n.sum())
        assert torch.equal(o[:rows], want[i][0][:rows]) and torch.equal(lse[:rows], want[i][1][:rows])
        assert cache.ctx_len.tolist() == want[i][2]


def test_a_captured_step_outlives_a_larger_one():
    # Steps of one row and of many share a workspace: the larger one, coming later, must not move it.
    cache = fa.PagedCache(num_pages=64, page_size=16, batch=2, max_len=400, H_kv=1, d=64, max_rows=300, max_new=150)
    x = torch.randn((300, 4, 64), device="cuda").to(torch.bfloat16)
    cache.plan(ints([100, 60]))
    cache.append(0, x[:160], x[:160, :1], x[:160, 1:2])
    cache.keep()
    o, lse = torch.zeros_like(x[:2]), torch.zeros((2, 4), device="cuda")

    def step():
        cache.plan(n, most=1)
        cache.append(0, x[:2], x[:2, :1], x[:2, 1:2])
        cache.attend(0, x[:2], o=o, lse=lse)

    n = ints([1, 1])
    step()
    torch.cuda.synchronize()
    want = o.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = {h: w.data_ptr() for h, w in cache._workspace.items()}
    cache.plan(ints([150, 150]))
    cache.append(0, x, x[:, :1], x[:, 1:2])
    cache.attend(0, x)
    assert held == {h: w.data_ptr() for h, w in cache._workspace.items()}
    torch.cuda.synchronize()
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK and torch.equal(o, want)


@pytest.mark.parametrize("B,H,N,d,axes,causal", [(1, 2, 300, 64, 1, True), (2, 3, 200, 128, 3, False), (1, 2, 129, 96, 2, True)])
def test_training_with_rotary_positions(B, H, N, d, axes, causal):
    c = Case(B, H, N, d, "bf16", seed=N)
    rng = np.random.default_rng(d)
    half = d // 2
    sections = [half - 8 * (axes - 1)] + [8] * (axes - 1)
    inv_freq, axis = fa.rope_tables(d, sections, base=10000.0, interleaved=axes == 3)
    pos = rng.integers(0, 3000, (axes, B, N))
    rope = fa.Rope(inv_freq, axis, ints(pos))
    q, k, v, do = (c.dev[n] for n in ("q", "k", "v", "do"))
    o, lse = fa.attention_forward(q, k, v, causal=causal, rope=rope)
    grads = fa.attention_backward(q, k, v, o, lse, do, causal=causal, rope=rope)
    torch.cuda.synchronize()
    assert fa.fa_device_status() == fa.FA_OK
    turn = lambda x, inverse=False: C.rope(x.reshape(B, H, N, d), pos[:, :, None], inv_freq.cpu().numpy(),  # noqa: E731
                                           axis.tolist(), inverse=inverse).reshape(B * H, N, d)
    Q, K, V, DO = (c.values(n) for n in ("q", "k", "v", "do"))
    RQ, RK = turn(Q), turn(K)
    O, L = oracle.forward(RQ, RK, V, c.scale, causal=causal)
    assert max_abs(c.flat(o), O) <= 1e-2
    # the rotated q and k are rounded once: a score is off by 2 * 2^-9 of scale |q||k|, about 6 at the most here
    assert max_abs(c.flat(lse), L) <= 2 * 2.0 ** -9 * 6
    DQ, DK, DV = oracle.backward(RQ, RK, V, DO, c.scale, causal=causal)
    assert_grads([(c.flat(g), G) for g, G in zip(grads, (turn(DQ, True), turn(DK, True), DV))])
