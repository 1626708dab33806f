"""fa_rope and fa_rope_append against the float64 oracle."""
import numpy as np
import pytest
import torch

import io_aware_exact_19_b200 as fa
from oracle import cache as C
from tests.cache_cases import DT, f64, ints

pytestmark = pytest.mark.gpu


def tables(rot, axes, base=500000.0):
    half = rot // 2
    inv = (base ** (-2.0 * np.arange(half) / rot)).astype(np.float32)
    axis = (np.arange(half) * axes // half).astype(np.uint8)
    return inv, axis, torch.from_numpy(inv).cuda(), torch.from_numpy(axis).cuda()


def assert_rotated(got, want, x, fmt):
    """One rounding to the type (half a step), and in 32 bits: the reduced angle (2 pi 2^-25), sincospif (2 ulp
    each) and three operations, all relative to |x| + |y| of the pair, which is at most 2 max|x| here."""
    u = torch.finfo(DT[fmt]).eps / 2
    tiny = 2.0 ** -25 if fmt == "fp16" else 0.0
    size = np.abs(x).max(-1, keepdims=True)
    lim = u * np.abs(want) * 1.01 + 2 * size * (2 * np.pi * 2.0 ** -25 + 8 * 2.0 ** -24) + tiny
    assert (np.abs(f64(got) - want) <= lim).all()


@pytest.mark.parametrize("B,H,N,d,rot,axes,fmt,pairs", [
    (1, 1, 1, 32, 32, 1, "bf16", False), (2, 3, 17, 64, 64, 3, "fp16", True), (2, 5, 33, 128, 128, 3, "bf16", False),
    (1, 2, 100, 96, 48, 2, "fp16", False), (3, 1, 7, 256, 256, 4, "bf16", True), (1, 4, 300, 128, 16, 8, "bf16", False),
    (1, 40, 5, 64, 32, 1, "fp16", True),
])
def test_rope_both_ways(B, H, N, d, rot, axes, fmt, pairs):
    rng = np.random.default_rng(N + d)
    x = torch.from_numpy(rng.standard_normal((B, H, N, d))).to(DT[fmt]).cuda()
    inv, axis, inv_d, axis_d = tables(rot, axes)
    pos = rng.integers(0, 100000, (axes, B, N))
    pos[0, 0, 0] = 2 ** 31 - 1  # the farthest position
    for inverse in (False, True):
        out = torch.full_like(x, float("nan"))
        fa.fa_rope(x, out, ints(pos), inv_d, axis_d, inverse=inverse, pairs=pairs)
        torch.cuda.synchronize()
        assert_rotated(out, C.rope(f64(x), pos[:, :, None], inv, axis, inverse, pairs), f64(x), fmt)
    assert torch.equal(out[..., rot:], x[..., rot:])


def test_rope_in_place_strided_and_broadcast():
    rng = np.random.default_rng(1)
    inv, axis, inv_d, axis_d = tables(64, 2)
    packed = torch.from_numpy(rng.standard_normal((2, 9, 5, 64))).to(torch.bfloat16).cuda()  # [B, N, heads, d]
    x = packed[:, :, 1:4].transpose(1, 2)  # a [B, H, N, d] view
    pos = rng.integers(0, 5000, (2, 9))
    before, others = f64(x), f64(packed[:, :, [0, 4]])
    fa.fa_rope(x, x, ints(pos), inv_d, axis_d)
    torch.cuda.synchronize()
    assert_rotated(x, C.rope(before, pos[:, None, None], inv, axis), before, "bf16")
    assert np.array_equal(f64(packed[:, :, [0, 4]]), others)


def test_rope_axis_out_of_range_is_left():
    inv, axis, inv_d, axis_d = tables(32, 2)
    axis_d[3] = 200
    x = torch.randn((1, 2, 6, 32), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(x)
    fa.fa_rope(x, out, ints(np.full((2, 6), 3)), inv_d, axis_d)
    torch.cuda.synchronize()
    assert torch.equal(out[..., [3, 19]], x[..., [3, 19]]) and not torch.equal(out, x)


def test_rope_gradient_by_differences():
    # <rope(x + e) - rope(x - e), g> = <2e, rope^-1(g)>; the oracle's rotation is pinned the same way.
    g = torch.Generator(device="cuda").manual_seed(0)
    x, e, w = (torch.randn((2, 3, 20, 64), generator=g, device="cuda").to(torch.float16) for _ in range(3))
    inv, axis, inv_d, axis_d = tables(64, 3)
    pos = torch.randint(0, 3000, (3, 2, 20), generator=g, device="cuda", dtype=torch.int32)
    f = lambda t, inverse=False: (lambda o: (fa.fa_rope(t, o, pos, inv_d, axis_d, inverse=inverse), o)[1])(
        torch.empty_like(t)).double()
    left = ((f(x + e) - f(x - e)) * w.double()).sum().item()
    right = (((x + e).double() - (x - e).double()) * f(w, True)).sum().item()
    # every value is rounded once (2^-11): independent errors of 3 terms over 7680 products of size about 2
    assert abs(left - right) < 6 * 3 * 2.0 ** -11 * 2 * 2 * np.sqrt(x.numel())


@pytest.mark.parametrize("T,Hq,H_kv,d,rot,axes,page,fmt,layout,pairs", [
    (1, 1, 1, 64, 64, 1, 16, "bf16", "hnd", False), (7, 8, 2, 128, 128, 3, 16, "bf16", "hnd", False),
    (50, 5, 5, 96, 32, 2, 8, "fp16", "nhd", True), (33, 4, 1, 256, 256, 1, 64, "bf16", "slice", False),
    (200, 3, 3, 32, 0, 1, 32, "fp16", "hnd", False),
])
def test_append(T, Hq, H_kv, d, rot, axes, page, fmt, layout, pairs):
    rng = np.random.default_rng(T)
    P = -(-T // page) + 3
    shape = {"hnd": (P, H_kv, page, d), "nhd": (P, page, H_kv, d), "slice": (P, 2, H_kv, page, d)}[layout]
    caches = []
    for _ in range(2):
        c = torch.full(shape, 7.0, dtype=DT[fmt], device="cuda")
        caches.append(c.transpose(1, 2) if layout == "nhd" else c[:, 0] if layout == "slice" else c)
    slot = rng.permutation(P * page)[:T]
    slot[T // 2] = -1 if T > 1 else slot[T // 2]
    if T > 3:
        slot[1], slot[2] = P * page, 2 ** 31 - 1  # outside the cache
    packed = torch.from_numpy(rng.standard_normal((T, Hq + 2 * H_kv, d))).to(DT[fmt]).cuda()
    q, k, v = packed.split([Hq, H_kv, H_kv], 1)
    q_out = torch.full((T, Hq, d), float("nan"), dtype=DT[fmt], device="cuda")
    args, qf, kf = {}, f64(q), f64(k)
    if rot:
        inv, axis, inv_d, axis_d = tables(rot, axes)
        pos = rng.integers(0, 4000, (axes, T))
        args = dict(positions=ints(pos), inv_freq=inv_d, axis=axis_d, pairs=pairs)
        qf, kf = (C.rope(x, pos[:, :, None], inv, axis, pairs=pairs) for x in (qf, kf))
    fa.fa_rope_append(q, k, v, q_out, *caches, ints(slot), **args)
    torch.cuda.synchronize()
    assert_rotated(q_out, qf, f64(q), fmt)
    got = [f64(c).transpose(0, 2, 1, 3).reshape(P * page, H_kv, d) for c in caches]
    inside = [t for t in range(T) if 0 <= slot[t] < P * page]
    assert_rotated(torch.from_numpy(got[0][slot[inside]]), kf[inside], f64(k)[inside], fmt)
    assert np.array_equal(got[1][slot[inside]], f64(v)[inside])
    rest = np.setdiff1d(np.arange(P * page), slot[inside])
    assert (got[0][rest] == 7).all() and (got[1][rest] == 7).all()
    if layout == "slice":
        assert (caches[0]._base[:, 1] == 7).all()


def test_append_without_queries_and_in_place():
    rng = np.random.default_rng(9)
    x = torch.from_numpy(rng.standard_normal((4, 3, 64))).to(torch.bfloat16).cuda()
    ck, cv = (torch.zeros((2, 3, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fa.fa_rope_append(None, x, x, None, ck, cv, ints([0, 17, 5, 31]))
    torch.cuda.synchronize()
    for t, (p, r) in enumerate([(0, 0), (1, 1), (0, 5), (1, 15)]):
        assert torch.equal(ck[p, :, r], x[t]) and torch.equal(cv[p, :, r], x[t])
    inv, axis, inv_d, axis_d = tables(64, 1)
    pos = np.array([[3, 9, 27, 81]])
    q = x.clone()
    fa.fa_rope_append(q, x, x, q, ck, cv, ints([0, 17, 5, 31]), ints(pos), inv_d, axis_d)
    torch.cuda.synchronize()
    assert_rotated(q, C.rope(f64(x), pos[:, :, None], inv, axis), f64(x), "bf16")
    assert torch.equal(ck[1, :, 1], q[1])


def test_flags_without_a_truth_value_are_refused():
    x = torch.zeros((1, 1, 2, 32), dtype=torch.float16, device="cuda")
    _, _, inv_d, axis_d = tables(32, 1)
    with pytest.raises(RuntimeError, match="ambiguous"):
        fa.fa_rope(x, x, ints([[0, 1]]), inv_d, axis_d, inverse=torch.zeros(2))
