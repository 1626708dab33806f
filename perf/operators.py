"""Measured cases of the paged key/value cache operators.

Four operators that run one after the other in a serving step over a paged cache,
the second also in training:

* ``plan``:   pages, slot map, positions and tree masks from request lengths
* ``rope``:   rotary positions over several axes (time, height, width); either with
              K and V written to the cache, or as the gradient of a training step
* ``attend``: attention of a drafted token tree (or a chain) over the cache
* ``commit``: the accepted path of each tree moved to the front of its rows

A case is a dict of plain values; the lengths of a ragged batch follow from the case
alone (``_lengths``), everything else from the seed. Where ``own`` is false, ``run``
computes in elementary torch operations in 32 bits (angles in 64), rounded once.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_DEV = "cuda"


# --------------------------------------------------------------------------- cases

def listed():
    """The measured range: smallest calls, ordinary ones, the largest."""
    return [
        # A small batch in plain decoding: one new token each, latency counts.
        dict(name="plan_decode_8", op="plan", B=8, ctx=4000, new=1, tree=False, page=16, spread=0.5),
        # A large batch with a drafted tree of up to 64 tokens each.
        dict(name="plan_tree_256", op="plan", B=256, ctx=8000, new=64, tree=True, page=16, spread=0.9),
        # A few new tokens of a small batch, rotated and written to the cache.
        dict(name="append_decode_8", op="rope", mode="append", B=8, new=1, Hq=32, Hkv=8, d=128, rot=128, axes=1,
             page=16, dtype="bf16", pairs=False),
        # A prompt chunk with image or video tokens: three position axes.
        dict(name="append_video_16k", op="rope", mode="append", B=2, new=8192, Hq=32, Hkv=8, d=128, rot=128, axes=3,
             page=64, dtype="bf16", pairs=False),
        # The gradient of the rotation in the long-context training shape (B=4 H=16 N=4096 d=128).
        dict(name="rope_grad_4k", op="rope", mode="grad", B=4, new=4096, Hq=16, Hkv=16, d=128, rot=128, axes=3,
             page=0, dtype="bf16", pairs=False),
        # One request, one token, a short context: the smallest call.
        dict(name="attend_decode_1", op="attend", B=1, ctx=1000, new=1, tree=False, Hq=32, Hkv=8, d=128, page=16,
             dtype="bf16", spread=0.0),
        # Ordinary decoding: 64 requests of very different lengths.
        dict(name="attend_decode_64", op="attend", B=64, ctx=8000, new=1, tree=False, Hq=32, Hkv=8, d=128, page=16,
             dtype="bf16", spread=0.9),
        # Verifying drafted trees of up to 48 tokens, odd group size, ragged pages.
        dict(name="attend_tree_16", op="attend", B=16, ctx=4003, new=48, tree=True, Hq=28, Hkv=4, d=128, page=32,
             dtype="fp16", spread=0.7),
        # One long request with a tree, no shared heads (the 64K decoding shape, 16 heads of 64).
        dict(name="attend_tree_64k", op="attend", B=1, ctx=65536, new=64, tree=True, Hq=16, Hkv=16, d=64, page=64,
             dtype="bf16", spread=0.0),
        # A prompt chunk after a cached prefix: the largest, bound by the products.
        dict(name="attend_chunk_2k", op="attend", B=2, ctx=8192, new=2048, tree=False, Hq=32, Hkv=8, d=128, page=64,
             dtype="bf16", spread=0.1),
        # A small batch's accepted drafts.
        dict(name="commit_8", op="commit", B=8, ctx=2000, new=16, Hkv=8, d=128, page=16, dtype="bf16"),
        # A large batch's.
        dict(name="commit_256", op="commit", B=256, ctx=500, new=64, Hkv=8, d=128, page=16, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above, at most as costly as the largest listed one."""
    op = rng.choice(["plan", "rope", "attend", "attend", "attend", "commit"])
    if op == "plan":
        tree = rng.random() < 0.6
        B = _log(rng, 1, 512)
        new = _log(rng, 1, 128) if tree else _log(rng, 1, max(1, 32768 // B))
        return dict(op="plan", B=B, ctx=_log(rng, 1, 16000), new=new, tree=tree, page=rng.choice([8, 16, 32, 64, 128]),
                    spread=round(rng.random(), 2))
    d = rng.choice([32, 64, 96, 128, 128, 256])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    dtype = rng.choice(["bf16", "fp16"])
    page = rng.choice([8, 16, 32, 64, 128])
    if op == "rope":
        rot = rng.choice([d, d, d // 2])
        mode = rng.choice(["append", "grad"])
        B = _log(rng, 1, 32)
        return dict(op="rope", mode=mode, B=B, new=_log(rng, 1, 16000 // B), Hq=Hkv * G, Hkv=Hkv, d=d, rot=rot,
                    axes=rng.choice([1, 2, 3]), page=page if mode == "append" else 0, dtype=dtype,
                    pairs=rng.random() < 0.3)
    if op == "commit":
        return dict(op="commit", B=_log(rng, 1, 256), ctx=_log(rng, 1, 1000), new=_log(rng, 1, 100), Hkv=Hkv, d=d,
                    page=page, dtype=dtype)
    tree = rng.random() < 0.5
    B = _log(rng, 1, 64)
    ctx = _log(rng, 16, 30000)
    new = _log(rng, 1, 128) if tree else _log(rng, 1, 1000)
    while B > 1 and (B * (ctx + new) * Hkv * d > 3e8 or B * new * Hkv * G * (ctx + new) * d > 3e10):
        B //= 2
    while new > 1 and B * new * Hkv * G * (ctx + new) * d > 3e10:
        new //= 2
    return dict(op="attend", B=B, ctx=ctx, new=new, tree=tree, Hq=Hkv * G, Hkv=Hkv, d=d, page=page, dtype=dtype,
                spread=round(rng.random(), 2))


def _lengths(case):
    """(context lengths, new tokens) of the requests, spread below `ctx` and `new`."""
    r = random.Random(case["B"] * 1000003 + case["ctx"] * 101 + case["new"])
    s = case.get("spread", 0.5)
    ctx = [max(0, int(case["ctx"] * (1 - s * r.random()))) for _ in range(case["B"])]
    if case["new"] == 1:
        return ctx, [1] * case["B"]
    return ctx, [max(1, int(round(case["new"] * (1 - 0.5 * min(s, 1.0) * r.random())))) for _ in range(case["B"])]


def _pages(n, page):
    return -(-n // page)


# --------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    return g


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=_DEV)


def _cu(new):
    return torch.nn.functional.pad(_int(new).cumsum(0, dtype=torch.int32), (1, 0))


def _parents(new, seed):
    """A drafted tree for each request: a token's parent is an earlier one or -1, mostly a recent one."""
    r = random.Random(seed * 7 + 3)
    out = []
    for n in new:
        out += [-1 if t == 0 or r.random() < 0.05 else max(0, t - 1 - int(r.expovariate(0.4))) for t in range(n)]
    return _int(out)


def _table(held, width, num_pages, seed):
    """A block table with `held` pages for each request in shuffled order, and the free pages behind them."""
    order = torch.randperm(num_pages, generator=_gen(seed), device=_DEV).to(torch.int32)
    table = torch.full((len(held), width), -1, dtype=torch.int32, device=_DEV)
    h = _int(held)
    inside = torch.arange(width, device=_DEV)[None, :] < h[:, None]
    table[inside] = order[: sum(held)]
    free = torch.cat([order[sum(held):], torch.full((sum(held),), -1, dtype=torch.int32, device=_DEV)])
    return table, h, free, _int([num_pages - sum(held)])


def _cache(num_pages, case, seed):
    g, shape = _gen(seed), (num_pages, case["Hkv"], case["page"], case["d"])
    return tuple(torch.randn(shape, generator=g, device=_DEV, dtype=_DT[case["dtype"]]) for _ in range(2))


def _axis(case):
    """Axis of each rotated pair: the pairs cut into one run for each axis, the first the shortest."""
    n, a = case["rot"] // 2, case["axes"]
    return [min(a - 1, i * (2 * a - 1) // max(1, 2 * n) if a > 1 else 0) for i in range(n)]


def prepare(case, seed):
    op, s = case["op"], {"case": case}
    B = case["B"]
    if op == "plan":
        ctx, new = _lengths(case)
        page, T = case["page"], sum(new)
        held = [_pages(c, page) for c in ctx]
        want = [_pages(c + n, page) for c, n in zip(ctx, new)]
        s["width"] = max(want)
        s["table"], s["held"], s["free"], s["free_count"] = _table(held, s["width"], sum(want) + 7, seed)
        s["ctx"], s["cu"], s["T"], s["max_new"] = _int(ctx), _cu(new), T, max(new)
        s["parent"] = _parents(new, seed) if case["tree"] else None
        s["words"] = _pages(s["max_new"], 64)
        s["seq_len"] = torch.zeros(B, dtype=torch.int32, device=_DEV)
        s["slot"], s["position"] = (torch.zeros(T, dtype=torch.int32, device=_DEV) for _ in range(2))
        s["mask"] = torch.zeros((T, s["words"]), dtype=torch.int64, device=_DEV) if case["tree"] else None
        return s
    if op == "rope":
        g, dt, n, d = _gen(seed), _DT[case["dtype"]], case["new"], case["d"]
        far = 200000 if case["axes"] == 1 else 4000
        s["positions"] = torch.randint(0, far, (case["axes"], B, n), generator=g, device=_DEV, dtype=torch.int32)
        exponent = torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"]
        s["inv_freq"] = (500000.0 ** -exponent).to(torch.float32).to(_DEV)
        s["axis"] = torch.tensor(_axis(case), dtype=torch.uint8, device=_DEV)
        if case["mode"] == "grad":
            s["dq"], s["dk"] = (torch.randn((B, h, n, d), generator=g, device=_DEV, dtype=dt)
                                for h in (case["Hq"], case["Hkv"]))
            s["dq_out"], s["dk_out"] = torch.empty_like(s["dq"]), torch.empty_like(s["dk"])
            return s
        # q, k and v as one projection leaves them: strided views of a packed tensor
        Hq, Hkv, T = case["Hq"], case["Hkv"], B * n
        packed = torch.randn((T, Hq + 2 * Hkv, d), generator=g, device=_DEV, dtype=dt)
        s["q"], s["k"], s["v"] = packed.split([Hq, Hkv, Hkv], dim=1)
        s["q_out"] = torch.empty((T, Hq, d), device=_DEV, dtype=dt)
        per = _pages(n, case["page"]) + 1
        s["cache"] = _cache(B * per, case, seed + 1)
        table, _, _, _ = _table([per] * B, per, B * per, seed)
        at = torch.arange(n, device=_DEV) + 3 % case["page"]  # the cache already holds a few rows
        s["slot"] = (table[:, at // case["page"]] * case["page"] + (at % case["page"]).to(torch.int32)).reshape(-1)
        return s
    if op == "commit":
        ctx, new = _lengths(case)
        page = case["page"]
        held = [_pages(c + n, page) for c, n in zip(ctx, new)]
        s["table"], _, _, _ = _table(held, max(held), sum(held), seed)
        s["cache"] = _cache(sum(held), case, seed)
        r = random.Random(seed)
        width = min(max(new), 12)
        count = [r.randint(1, min(n, width)) for n in new]
        rows = [sorted(r.sample(range(n), c)) + [-1] * (width - c) for n, c in zip(new, count)]
        s["ctx"], s["accepted"], s["count"] = _int(ctx), _int(rows), _int(count)
        s["new_len"] = torch.empty(B, dtype=torch.int32, device=_DEV)
        return s
    ctx, new = _lengths(case)
    page, T, dt = case["page"], sum(new), _DT[case["dtype"]]
    length = [c + n for c, n in zip(ctx, new)]
    held = [_pages(n, page) for n in length]
    s["table"], _, _, _ = _table(held, max(held), sum(held), seed)
    s["cache"] = _cache(sum(held), case, seed)
    s["q"] = torch.randn((T, case["Hq"], case["d"]), generator=_gen(seed + 5), device=_DEV, dtype=dt)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((T, case["Hq"]), dtype=torch.float32, device=_DEV)
    s["cu"], s["seq_len"], s["max_new"], s["max_len"] = _cu(new), _int(length), max(new), max(length)
    s["mask"] = None
    if case["tree"]:
        s["mask"] = _pack(_ancestors(_parents(new, seed), s["cu"], s["max_new"], T))
    if own:
        import io_aware_exact_19_b200 as fa
        s["workspace"] = torch.empty(
            fa.fa_tree_fwd_workspace_size(case["B"], T, s["max_new"], case["Hq"], case["Hkv"], case["d"]),
            dtype=torch.uint8, device=_DEV)
    return s


# --------------------------------------------------------------------------- plain forms

def _ragged(cu, T):
    """Request and index within the request of each of T packed tokens."""
    t = torch.arange(T, device=cu.device)
    b = (t[:, None] >= cu[None, 1:]).sum(1)
    return b, t - cu[b]


def _ancestors(parent, cu, max_new, T):
    """[T, max_new] truth values: whether the token's branch holds that token of its request (itself included)."""
    b, i = _ragged(cu, T)
    reach = torch.zeros((cu.numel() - 1, max_new, max_new), device=cu.device)
    reach[b, i, i] = 1.0
    reach[b[parent >= 0], i[parent >= 0], parent[parent >= 0].long()] = 1.0
    for _ in range(max(1, (max_new - 1).bit_length())):  # paths of twice the length each time
        reach = ((reach @ reach) > 0).float()
    return reach[b, i] > 0


def _pack(bits):
    """Truth values [T, n] in words of 64 bits, the lowest bit first."""
    T, n = bits.shape
    words = _pages(n, 64)
    wide = torch.nn.functional.pad(bits, (0, 64 * words - n)).view(T, words, 64).long()
    return (wide << torch.arange(64, device=bits.device)).sum(-1)


def _unpack(words, n):
    return ((words[:, :, None] >> torch.arange(64, device=words.device)) & 1).bool().reshape(words.shape[0], -1)[:, :n]


def _plan_plain(s):
    page, cu, T, ctx = s["case"]["page"], s["cu"], s["T"], s["ctx"]
    table, held, free = s["table"], s["held"], s["free"]
    new = cu[1:] - cu[:-1]
    want = (ctx + new + page - 1) // page
    column = torch.arange(s["width"], device=_DEV)[None, :]
    need = (want - held).clamp(min=0)
    upto = need.cumsum(0)
    granted = (need == 0) | (upto <= s["free_count"])
    # pages come off the end of the free list, in the order of the requests
    taken = (column >= held[:, None]) & (column < want[:, None]) & granted[:, None]
    rank = (upto - need)[:, None] + column - held[:, None]
    source = (s["free_count"] - 1 - rank).clamp(min=0)
    table.copy_(torch.where(taken, free[source], table))
    s["free_count"] -= taken.sum().to(torch.int32)
    held.copy_(torch.where(granted, want, held))
    s["seq_len"].copy_(torch.where(granted, ctx + new, torch.zeros_like(ctx)))
    b, i = _ragged(cu, T)
    at = ctx[b] + i
    slot = table[b, at // page] * page + at % page
    s["slot"].copy_(torch.where(granted[b], slot, -1))
    if s["parent"] is None:
        s["position"].copy_(at)
    else:
        bits = _ancestors(s["parent"], cu, s["max_new"], T)
        s["position"].copy_(ctx[b] + bits.sum(1) - 1)
        s["mask"].copy_(_pack(bits))


def _rotated(x, positions, s, sign):
    """x [..., n, d] rotated; positions [axes, ..., n] without the heads' dimension."""
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    angle = positions.double().movedim(0, -1)[..., s["axis"].long()] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), sign * angle.sin().float()
    y = x.float()
    if case["pairs"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _rope_plain(s):
    case, positions = s["case"], s["positions"]
    if case["mode"] == "grad":
        return tuple(_rotated(s[n], positions[:, :, None], s, -1.0) for n in ("dq", "dk"))
    flat = positions.flatten(1)[:, :, None]
    k_cache, v_cache = s["cache"]
    page, slot = case["page"], s["slot"].long()
    k_cache[slot // page, :, slot % page] = _rotated(s["k"], flat, s, 1.0)
    v_cache[slot // page, :, slot % page] = s["v"]
    return _rotated(s["q"], flat, s, 1.0), k_cache, v_cache


def _attend_plain(s):
    case, cu = s["case"], s["cu"]
    T, Hq, d = s["q"].shape
    Hkv, page, L, n = case["Hkv"], case["page"], s["max_len"], s["max_new"]
    at = torch.arange(L, device=_DEV)
    pages = s["table"][:, at // page].clamp(min=0).long()
    k, v = (c[pages, :, (at % page)[None, :]].float().permute(0, 2, 1, 3) for c in s["cache"])  # [B, Hkv, L, d]
    b, i = _ragged(cu, T)
    q = torch.zeros((case["B"], n, Hq, d), device=_DEV)
    q[b, i] = s["q"].float()
    q = q.view(-1, n, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(-1, Hkv, Hq // Hkv * n, d)
    score = (q @ k.transpose(-1, -2)).view(-1, Hkv, Hq // Hkv, n, L) / math.sqrt(d)
    ctx = (s["seq_len"] - (cu[1:] - cu[:-1]))[:, None, None]
    own_key = at[None, None, :] - ctx  # index of the key among the request's new tokens
    if s["mask"] is None:
        seen = own_key <= torch.arange(n, device=_DEV)[None, :, None]
    else:
        bits = torch.zeros((case["B"], n, n), dtype=torch.bool, device=_DEV)
        bits[b, i] = _unpack(s["mask"], n)
        index = own_key.clamp(0, n - 1).expand(-1, n, -1)
        seen = (own_key < 0) | bits.gather(2, index)
    seen = seen & (at[None, None, :] < s["seq_len"][:, None, None])
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    e = (score - top).exp()
    total = e.sum(-1, keepdim=True)
    o = ((e / total.clamp(min=1e-30)).view(-1, Hkv, Hq // Hkv * n, L) @ v).view(-1, Hkv, Hq // Hkv, n, d)
    lse = (top + total.log()).squeeze(-1)
    back = lambda x: x.movedim(3, 1).flatten(2, 3)[b, i]  # noqa: E731  [B, Hkv, G, n, ...] -> [T, Hq, ...]
    return back(o).to(s["q"].dtype), back(lse)


def _commit_plain(s):
    page, ctx, count, rows = s["case"]["page"], s["ctx"], s["count"], s["accepted"]
    step = torch.arange(rows.shape[1], device=_DEV)[None, :]
    b, j = torch.nonzero(step < count[:, None], as_tuple=True)
    source, target = ctx[b] + rows[b, j], ctx[b] + j
    where = lambda at: (s["table"][b, at // page].long(), slice(None), at % page)  # noqa: E731
    for c in s["cache"]:
        c[where(target)] = c[where(source)]
    s["new_len"].copy_(ctx + count)


# --------------------------------------------------------------------------- one pass

def _own(s):
    import io_aware_exact_19_b200 as fa
    case = s["case"]
    if case["op"] == "plan":
        fa.fa_cache_plan(s["ctx"], s["cu"], s["table"], s["held"], s["free"], s["free_count"], s["seq_len"],
                         s["slot"], s["position"], page_size=case["page"], max_new=s["max_new"], parent=s["parent"],
                         tree_mask=s["mask"])
    elif case["op"] == "rope" and case["mode"] == "grad":
        for x, out in ((s["dq"], s["dq_out"]), (s["dk"], s["dk_out"])):
            fa.fa_rope(x, out, s["positions"], s["inv_freq"], s["axis"], inverse=True, pairs=case["pairs"])
        return s["dq_out"], s["dk_out"]
    elif case["op"] == "rope":
        fa.fa_rope_append(s["q"], s["k"], s["v"], s["q_out"], *s["cache"], s["slot"], s["positions"].flatten(1),
                          s["inv_freq"], s["axis"], pairs=case["pairs"])
        return (s["q_out"], *s["cache"])
    elif case["op"] == "commit":
        fa.fa_cache_commit(*s["cache"], s["table"], s["ctx"], s["accepted"], s["count"], s["new_len"])
    else:
        fa.fa_tree_fwd(s["q"], *s["cache"], s["table"], s["seq_len"], s["cu"], s["o"], s["lse"], s["workspace"],
                       max_q=s["max_new"], tree_mask=s["mask"])
        return s["o"], s["lse"]


def run(state):
    op = state["case"]["op"]
    if own:
        out = _own(state)
    else:
        out = {"plan": _plan_plain, "rope": _rope_plain, "attend": _attend_plain, "commit": _commit_plain}[op](state)
    if op == "plan":
        return {k: state[k] for k in ("table", "held", "free_count", "seq_len", "slot", "position", "mask")
                if state[k] is not None}
    if op == "commit":
        return (*state["cache"], state["new_len"])
    return out


def work(case):
    op, B = case["op"], case["B"]
    if op == "rope":
        rows = B * case["new"]
        heads = case["Hq"] + case["Hkv"]
        moved = heads if case["mode"] == "grad" else heads + case["Hkv"]
        return {"bytes": rows * (4 * moved * case["d"] + 4 * case["axes"] + (4 if case["mode"] == "append" else 0)),
                "flops": 3 * rows * heads * case["rot"]}
    ctx, new = _lengths(case)
    if op == "plan":
        T, words = sum(new), _pages(max(new), 64) if case["tree"] else 0
        return {"bytes": 24 * B + T * (8 + 8 * words + (4 if case["tree"] else 0)), "flops": 0}
    if op == "commit":
        width = min(max(new), 12)  # about half of it is accepted
        return {"bytes": B * (8 + 4 * width) + sum(1 + min(n, width) for n in new) * 4 * case["Hkv"] * case["d"],
                "flops": 0}
    d, Hq, Hkv = case["d"], case["Hq"], case["Hkv"]
    keys = sum(c + n for c, n in zip(ctx, new))
    # a tree's token sees the context and its branch, a chain's all tokens before it
    pairs = sum(n * c + (n if case["tree"] else n * (n + 1) // 2) for c, n in zip(ctx, new))
    return {"bytes": 4 * keys * Hkv * d + sum(new) * Hq * (4 * d + 4) + 4 * _pages(keys, case["page"]),
            "flops": 4 * pairs * Hq * d}


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """What `run` returns, request by request in 64 bits; None where all of it is whole numbers."""
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rope_exact(s)
    if case["op"] == "commit":
        k, v = (c.double() for c in s["cache"])
        table, page = s["table"].tolist(), case["page"]
        for b, (c, rows, n) in enumerate(zip(s["ctx"].tolist(), s["accepted"].tolist(), s["count"].tolist())):
            for j, r in enumerate(rows[:n]):  # in order: a row is read before anything is written over it
                (p, i), (P, I) = divmod(c + r, page), divmod(c + j, page)
                for x in (k, v):
                    x[table[b][P], :, I] = x[table[b][p], :, i]
        return k, v, None
    return _attend_exact(s)


def _turn_exact(x, where, s, sign):
    """One token's heads [H, d], its position on each axis."""
    rot, y = s["case"]["rot"], x.double().clone()
    n = torch.arange(rot // 2, device=_DEV)
    first, second = (2 * n, 2 * n + 1) if s["case"]["pairs"] else (n, n + rot // 2)
    z = torch.polar(torch.ones(rot // 2, dtype=torch.float64, device=_DEV),
                    sign * where.double()[..., s["axis"].long()] * s["inv_freq"].double())
    w = torch.complex(y[..., first], y[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _rope_exact(s):
    case = s["case"]
    if case["mode"] == "grad":
        where = s["positions"].permute(1, 2, 0)[:, None]  # [B, 1, n, axes]
        return _turn_exact(s["dq"], where, s, -1.0), _turn_exact(s["dk"], where, s, -1.0)
    where = s["positions"].flatten(1).t()[:, None]  # [T, 1, axes]
    k, v = (c.double() for c in s["cache"])
    page, slot = case["page"], s["slot"].long()
    # the cache as rows of one page after the other
    for c, x in ((k, _turn_exact(s["k"], where, s, 1.0)), (v, s["v"].double())):
        rows = c.permute(0, 2, 1, 3).reshape(-1, case["Hkv"], case["d"]).clone()
        rows.index_copy_(0, slot, x)
        c.copy_(rows.view(-1, page, case["Hkv"], case["d"]).permute(0, 2, 1, 3))
    return _turn_exact(s["q"], where, s, 1.0), k, v


def _attend_exact(s):
    case = s["case"]
    T, Hq, d = s["q"].shape
    Hkv, page = case["Hkv"], case["page"]
    if 4.0 * T * Hq * d * s["max_len"] > 3e12:
        return None
    o = torch.zeros((T, Hq, d), dtype=torch.float64, device=_DEV)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=_DEV)
    cu, length = s["cu"].tolist(), s["seq_len"].tolist()
    for b in range(case["B"]):
        t0, n, L = cu[b], cu[b + 1] - cu[b], length[b]
        held = s["table"][b, : _pages(L, page)].long()
        k, v = (c[held].double().transpose(0, 1).reshape(Hkv, -1, d)[:, :L] for c in s["cache"])
        seen = torch.ones((n, L), dtype=torch.bool, device=_DEV)
        if s["mask"] is None:
            seen = torch.tril(seen, diagonal=L - n)
        else:
            seen[:, L - n:] = _unpack(s["mask"][t0:t0 + n], n)
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            x = (s["q"][t0:t0 + n, h].double() @ k[kv].t()) * d ** -0.5
            x[~seen] = -math.inf
            z = torch.logsumexp(x, 1, keepdim=True)
            o[t0:t0 + n, h] = torch.exp(x - z).nan_to_num(0.0) @ v[kv]
            lse[t0:t0 + n, h] = z[:, 0]
    return o, lse
