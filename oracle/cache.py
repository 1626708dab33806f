"""Plain forms of the paged-cache operators: page bookkeeping as Python loops, rotary
positions and tree attention in float64, request by request."""
from __future__ import annotations

import numpy as np

NEG_INF = -np.inf


# ----------------------------------------------------------------------------- bookkeeping

def ancestors(parent) -> np.ndarray:
    """[n, n] truth values: row t holds t and its ancestors; a parent outside [-1, t) counts as -1."""
    n = len(parent)
    m = np.zeros((n, n), bool)
    for t in range(n):
        m[t, t] = True
        p = int(parent[t])
        if 0 <= p < t:
            m[t] |= m[p]
    return m


def pack_mask(bits: np.ndarray, words: int) -> np.ndarray:
    """Truth values [n, k] as int64 words [n, words], the lowest bit first."""
    out = np.zeros((bits.shape[0], words), np.uint64)
    for j in range(bits.shape[1]):
        out[:, j // 64] |= bits[:, j].astype(np.uint64) << np.uint64(j % 64)
    return out.view(np.int64)


def plan(ctx, cu, table, held, free, free_count, page, rows, max_new, parent=None):
    """One call of fa_cache_plan on host lists; returns the new state and the step's maps.

    ``table`` is a list of lists, ``free`` a list whose first ``free_count`` entries are free."""
    table, held, free = [list(r) for r in table], list(held), list(free)
    num_pages, max_pages, B = len(free), len(table[0]), len(ctx)
    want = []
    for b in range(B):
        n = cu[b + 1] - cu[b]
        w = -(-(ctx[b] + n) // page)
        inside = n == 0 or (cu[b] >= 0 and cu[b + 1] <= rows)
        want.append(w if ctx[b] >= 0 and 0 <= n <= max_new and inside and w <= max_pages else None)
    count = free_count
    for b in range(B):
        if want[b] is not None:
            for i in range(want[b], held[b]):
                free[count] = table[b][i]
                table[b][i] = -1
                count += 1
    seq, granted, asked, top = [0] * B, [False] * B, 0, count
    for b in range(B):
        if want[b] is None:
            continue
        need = max(0, want[b] - held[b])
        if need == 0 or asked + need <= top:
            for i in range(need):
                table[b][held[b] + i] = free[top - 1 - asked - i]
            count -= need
            held[b], granted[b], seq[b] = want[b], True, ctx[b] + cu[b + 1] - cu[b]
        asked += need
    assert 0 <= count <= num_pages
    slot, position = [-1] * rows, [0] * rows
    words = -(-max_new // 64)
    mask = {}
    for b in range(B):
        n = cu[b + 1] - cu[b]
        up = None if parent is None else ancestors(parent[cu[b]:cu[b] + n])
        for i in range(min(n, rows - cu[b])):
            t, at = cu[b] + i, ctx[b] + i
            if granted[b]:
                slot[t] = table[b][at // page] * page + at % page
            position[t] = at if up is None else ctx[b] + int(up[i].sum()) - 1
            if up is not None:
                mask[t] = pack_mask(up[i:i + 1], words)[0]
    return table, held, free, count, seq, slot, position, mask


# ----------------------------------------------------------------------------- rotary

def rope(x, positions, inv_freq, axis, inverse=False, pairs=False):
    """x [..., n, d] in float64; positions [axes, ..., n] broadcast against x without d."""
    x = np.array(x, np.float64)
    half = len(inv_freq)
    for i in range(half):
        angle = np.asarray(positions[axis[i]], np.float64) * float(inv_freq[i]) if axis[i] < len(positions) else 0.0
        c, s = np.cos(angle), np.sin(angle) * (-1.0 if inverse else 1.0)
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        xa, xb = x[..., a].copy(), x[..., b].copy()
        x[..., a] = xa * c - xb * s
        x[..., b] = xa * s + xb * c
    return x


# ----------------------------------------------------------------------------- attention

def seen_keys(n, length, bits=None) -> np.ndarray:
    """[n, length] truth values: which keys each of a request's n new rows sees."""
    i, j = np.arange(n)[:, None], np.arange(length)[None, :]
    if bits is None:
        return j <= i + length - n
    u = j - (length - n)
    inside = np.clip(u, 0, bits.shape[1] - 1) + np.zeros_like(i)
    return (u < 0) | (np.take_along_axis(bits, inside, 1) & (u < bits.shape[1]))


def tree_attention(q, k, v, scale, seen):
    """q [n, Hq, d], k and v [len, H_kv, d] in float64, seen [n, len] -> (o, lse, sum p|v|, max scale*|q||k|)."""
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    o, size = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse = np.full((n, Hq), NEG_INF)
    big = 0.0
    v = np.where(seen.any(0)[:, None, None], v, 0.0)
    for h in range(Hq):
        kh, vh = k[:, h // G], v[:, h // G]
        with np.errstate(invalid="ignore"):
            s = np.where(seen, scale * (q[:, h] @ kh.T), NEG_INF)
            a = np.where(seen, abs(scale) * (np.abs(q[:, h]) @ np.abs(kh).T), 0.0)
        big = max(big, float(a.max()) if a.size else 0.0)
        m = s.max(1, initial=NEG_INF)
        some = m > NEG_INF
        e = np.where(seen, np.exp(s - np.where(some, m, 0.0)[:, None]), 0.0)
        l = e.sum(1)
        p = e / np.where(l > 0, l, 1.0)[:, None]
        o[:, h], size[:, h] = p @ vh, p @ np.abs(vh)
        lse[some, h] = m[some] + np.log(l[some])
    return o, lse, size, big


def commit(cache_rows, ctx, accepted):
    """Move rows ctx + accepted[j] to ctx + j of one request's rows; returns the rows kept."""
    last, kept = -1, 0
    for j, a in enumerate(accepted):
        if a <= last:
            break
        cache_rows[ctx + j] = cache_rows[ctx + a]
        last, kept = a, j + 1
    return ctx + kept
