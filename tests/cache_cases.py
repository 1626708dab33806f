"""Ragged batches over a paged cache for the GPU tests: device tensors and their float64 values."""
import numpy as np
import torch

from oracle import cache as C

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def random_parents(new, rng):
    return [int(rng.integers(-1, t)) if t else -1 for n in new for t in range(n)]


class Paged:
    """A filled cache of requests with `ctx` cached and `new` new rows.

    layout "hnd": pages [head][row][d]; "nhd": pages [row][head][d]; "slice": one layer
    of a pool with two. What lies behind the requests' rows and in pages of no request
    is NaN."""

    def __init__(self, ctx, new, H_kv, d, page, fmt, layout="hnd", spare=2, seed=0):
        self.ctx, self.new, self.page, self.H_kv, self.d, self.fmt = list(ctx), list(new), page, H_kv, d, fmt
        self.rng = rng = np.random.default_rng(seed)
        self.len = [c + n for c, n in zip(ctx, new)]
        held = [-(-n // page) for n in self.len]
        P = sum(held) + spare
        order = rng.permutation(P)
        width = max(held + [1]) + 1
        table = np.full((len(ctx), width), -1)
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = order[at:at + h]
            at += h
        self.table_host, self.held, self.num_pages = table, held, P
        self.free_host = [int(x) for x in order[at:]]
        self.k, self.v = self._make(layout, P), self._make(layout, P)
        for t in (self.k, self.v):
            t.fill_(float("nan"))
            for b, n in enumerate(self.len):
                for r in range(0, n, page):
                    rows = min(page, n - r)
                    x = rng.standard_normal((H_kv, rows, d))
                    t[int(table[b, r // page]), :, :rows] = torch.from_numpy(x).to(DT[fmt]).cuda()
        self.table = ints(table)
        self.seq_len = ints(self.len)
        self.cu_host = np.concatenate([[0], np.cumsum(new)]).astype(int)
        self.cu = ints(self.cu_host)
        self.T, self.max_new = int(self.cu_host[-1]), max(list(new) + [1])

    def _make(self, layout, P):
        H, page, d, dt = self.H_kv, self.page, self.d, DT[self.fmt]
        if layout == "hnd":
            return torch.empty((P, H, page, d), dtype=dt, device="cuda")
        if layout == "nhd":
            return torch.empty((P, page, H, d), dtype=dt, device="cuda").transpose(1, 2)
        return torch.empty((P, 2, H, page, d), dtype=dt, device="cuda")[:, 1]

    def rows_of(self, t, b):
        """Request b's rows of a cache as float64 [len, H_kv, d]."""
        n = self.len[b]
        pages = self.table_host[b, :self.held[b]]
        x = f64(t)[pages].transpose(0, 2, 1, 3).reshape(-1, self.H_kv, self.d)
        return x[:n]


def attention_reference(p, q, scale, bits=None):
    """Oracle over all requests: q float64 [T, Hq, d]; bits: list of [n, n] or None."""
    out = []
    for b, n in enumerate(p.new):
        t0 = p.cu_host[b]
        seen = C.seen_keys(n, p.len[b], None if bits is None else bits[b])
        out.append(C.tree_attention(q[t0:t0 + n], p.rows_of(p.k, b), p.rows_of(p.v, b), scale, seen))
    return out


def assert_attention(p, o, lse, ref):
    """Elementwise bounds. Each P is rounded to the element type once (half a step, u) and so is O; a
    score errs by at most d products' worth of fp32 roundings of scale*|q||k|, and ex2, lg2 and the sums
    by a few more. |O| and |P V| are at most sum p|v|."""
    u = torch.finfo(DT[p.fmt]).eps / 2
    tiny = 2.0 ** -24 if p.fmt == "fp16" else 0.0  # P below the normal range of fp16 is off by half its step
    for b, (O, L, size, big) in enumerate(ref):
        t0, n = p.cu_host[b], p.new[b]
        score = 2.0 ** -24 * (p.d * big + 16)
        chain = 2.0 ** -24 * (p.len[b] / 64 + 64)
        bound = (2 * u + 4 * score + 2 * chain) * size * 1.01 + tiny * p.len[b] + 1e-30
        err = np.abs(f64(o[t0:t0 + n]) - O)
        assert (err <= bound).all(), (b, float((err - bound).max()), float((err / bound).max()))
        got = f64(lse[t0:t0 + n])
        dead = np.isneginf(L)
        assert np.array_equal(np.isneginf(got), dead), b
        assert (f64(o[t0:t0 + n])[dead] == 0).all(), b
        lim = 2 * score + chain + 2.0 ** -20 + 2.0 ** -22 * np.abs(L[~dead])
        assert (np.abs(got[~dead] - L[~dead]) <= lim).all(), (b, np.abs(got[~dead] - L[~dead]).max())
