"""Norms, rotation and the cache's new entries (qk_norm_rope) against 64 bits (needs an MI355X).

Tolerances: the norm is a sum of D squares, a division and a root in fp32, then two products: off by
(D/2 + 6) half steps of fp32 at most; sine and cosine by 2 ulps of 1 (4 half steps, the angle's reduction in 64
bits adds less); the rotation two products and a sum.  Relative to |a| + |b| that is (D/2 + 16) EPS32; then one
rounding to bf16, or of value / scale to e4m3 (whose steps below 2^-6 are 2^-9)."""
from __future__ import annotations

import pytest
import torch

import fp8_block_scaled_a8w8_amd as g
from attention_util import BF16, E4M3, EPS32, rotate64

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def projection(T, Hq, Hkv, D, gated, seed):
    gen = torch.Generator().manual_seed(seed)
    w = 2 if gated else 1
    rows = torch.randn(T, (w * Hq + 2 * Hkv) * D, generator=gen).to(torch.bfloat16)
    return rows, split(rows, Hq, Hkv, D, w)


def split(rows, Hq, Hkv, D, w):
    T = len(rows)
    q, k, v = rows.split((w * Hq * D, Hkv * D, Hkv * D), 1)
    return q.view(T, Hq, w * D)[..., :D], k.view(T, Hkv, D), v.view(T, Hkv, D)


def near(got, want, mag, D, what):
    tol = (D / 2 + 16) * EPS32 * mag
    bad = (got.double().cpu() - want).abs() > tol + BF16 * (want.abs() + tol) + 1e-38
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist())


CASES = [
    # T, Hq, Hkv, D, R, layout, axes, dtype, page, gated, norm, pad
    (1, 24, 4, 256, 64, "halves", 1, "bf16", 64, True, True, 0),
    (1, 1, 1, 64, 64, "pairs", 1, "fp8", 1, False, True, 0),
    (7, 3, 1, 64, 16, "halves", 3, "bf16", 16, False, True, 2),
    (33, 32, 8, 128, 128, "pairs", 1, "fp8", 16, False, True, 3),
    (33, 12, 2, 128, 96, "halves", 2, "fp8", 32, True, True, 0),
    (61, 6, 6, 256, 256, "halves", 4, "bf16", 128, False, True, 5),
    (130, 5, 1, 256, 80, "halves", 1, "bf16", 64, True, False, 0),
    (2000, 4, 2, 128, 48, "pairs", 3, "bf16", 16, False, True, 100),
    (5, 40, 40, 64, 0, "halves", 1, "bf16", 16, False, True, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_against_64_bits(case):
    T, Hq, Hkv, D, R, layout, axes, dtype, page, gated, norm, pad = case
    say("rope", case)
    rows, _ = projection(T, Hq, Hkv, D, gated, seed=T + D)
    gen = torch.Generator().manual_seed(3)
    wq, wk = ((1 + 0.3 * torch.randn(D, generator=gen)) if norm else None for _ in range(2))
    inv = (1e6 ** (-torch.arange(0, R, 2).double() / max(R, 1))).float() if R else None
    ax = torch.randint(-1, axes + 1, (R // 2,), generator=gen).int() if R and axes > 1 else None
    pos = torch.randint(0, 1 << 20, (axes, T), generator=gen).int()
    if T > 1:
        pos[:, 0] = 0
        pos[:, 1] = (1 << 31) - 1
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=gen)[:T].int()
    if pad:
        slots[-pad:] = -1
        slots[-1] = pages * page                     # outside as well
    kinds = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
    scales = [None, None] if dtype == "bf16" else [torch.rand(Hkv, generator=gen) / 100 + 0.003 for _ in range(2)]
    fill = torch.randint(0, 120, (2, pages, page, Hkv, D * (2 if dtype == "bf16" else 1)), generator=gen).to(torch.uint8)
    kc, vc = (fill[i].to(DEV).view(kinds[dtype]) for i in range(2))
    cache = g.KvCache(kc, vc, *(None if s is None else s.to(DEV) for s in scales))
    q, k, v = split(rows.to(DEV), Hq, Hkv, D, 2 if gated else 1)
    rope = g.Rope(inv.to(DEV), axes=None if ax is None else ax.to(DEV), layout=layout) if R else None
    args = dict(q_weight=None if wq is None else wq.to(DEV), k_weight=None if wk is None else wk.to(DEV), eps=1e-5)
    p = pos.to(DEV) if axes > 1 else pos[0].to(DEV)
    qo, none = g.qk_norm_rope(q, k, rope, p, v=v, cache=cache, slots=slots.to(DEV), **args)
    assert none is None
    q64, qm = rotate64(q.cpu(), wq, 1e-5, pos, inv, ax, layout)
    k64, km = rotate64(k.cpu(), wk, 1e-5, pos, inv, ax, layout)
    near(qo, q64, qm, D, "q")
    kept = torch.nonzero((slots >= 0) & (slots < pages * page))[:, 0]
    at = slots[kept].long()
    for name, c, old, x, m, s in (("k", kc, fill[0], k64, km, scales[0]), ("v", vc, fill[1], v.cpu().double(), v.cpu().double().abs(), scales[1])):
        got = c.cpu().view(-1, Hkv, D)
        if s is None:
            near(got[at], x[kept], m[kept], D, name)
        else:
            want = x[kept] / s.double()[:, None]
            tol = ((D / 2 + 17) * EPS32 * m[kept]) / s.double()[:, None]
            err = (got[at].double() - want.clamp(-448, 448)).abs()
            assert bool((err <= tol + torch.maximum(E4M3 * (want.abs() + tol), torch.tensor(2.0 ** -10).double())).all()), name
        # every other slot as it was
        other = torch.ones(pages * page, dtype=torch.bool)
        other[at] = False
        raw = c.view(torch.uint8).cpu().view(pages * page, -1)
        assert torch.equal(raw[other], old.view(pages * page, -1)[other]), name
    # without a cache the keys come back, from the same arithmetic
    q2, k2 = g.qk_norm_rope(q, k, rope, p, **args)
    assert torch.equal(q2.view(torch.int16), qo.view(torch.int16))
    near(k2, k64, km, D, "k_out")


def test_far_positions_keep_their_phase():
    """A frequency of 1 turns position 2^31 - 1 by an angle that fp32 cannot hold."""
    D, T = 64, 4
    pos = torch.tensor([(1 << 31) - 1, 1 << 24, 16777217, 1], dtype=torch.int32)
    inv = torch.cat([torch.ones(8), torch.full((8,), 0.777), torch.full((16,), 1e-3)])
    x = torch.zeros(T, 1, D, dtype=torch.bfloat16)
    x[..., :32] = 1.0
    k = x.clone()
    q, _ = g.qk_norm_rope(x.to(DEV), k.to(DEV), g.Rope(inv.to(DEV)), pos.to(DEV))
    want, mag = rotate64(x, None, 0.0, pos, inv, None, "halves")
    near(q, want, mag, D, "q")


def test_nan_stays_with_its_head_and_large_values_saturate():
    D, T, H = 128, 6, 2
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(T, H, D, generator=gen).to(torch.bfloat16) for _ in range(3))
    k[1, 0, 5] = float("nan")
    q[2, 1, 7] = float("inf")
    v[3, 1] = 1e30
    v[4, 0, 3], v[4, 0, 4] = float("inf"), -float("inf")
    v[5, 1, 9] = float("nan")
    cache = g.KvCache.empty(2, 16, H, D, dtype=torch.float8_e4m3fn, device=DEV)
    w = torch.ones(D, device=DEV)
    qo, _ = g.qk_norm_rope(q.to(DEV), k.to(DEV), None, None, q_weight=w, k_weight=w, v=v.to(DEV), cache=cache,
                           slots=torch.arange(T, dtype=torch.int32, device=DEV))
    kk, vv = cache.k.float().cpu().view(-1, H, D)[:T], cache.v.float().cpu().view(-1, H, D)[:T]
    assert bool(torch.isnan(kk[1, 0]).all()) and not torch.isnan(kk[1, 1]).any() and not torch.isnan(kk[0]).any()
    assert bool((vv[3, 1] == 448).all()) and vv[4, 0, 3] == 448 and vv[4, 0, 4] == -448
    assert torch.isnan(vv[5, 1, 9]) and int(torch.isnan(vv).sum()) == 1
    bad = ~torch.isfinite(qo.float().cpu())
    assert bool(bad[2, 1, 7]) and not bad[:2].any() and not bad[3:].any() and not bad[2, 0].any()


def test_captured_and_replayed():
    T, Hq, Hkv, D = 9, 4, 2, 128
    rows, _ = projection(T, Hq, Hkv, D, False, 5)
    rows = rows.to(DEV)
    q, k, v = split(rows, Hq, Hkv, D, 1)
    cache, other = (g.KvCache.empty(2, 16, Hkv, D, device=DEV) for _ in range(2))
    slots, pos = torch.arange(T, dtype=torch.int32, device=DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    rope = g.Rope(torch.logspace(0, -4, 64, device=DEV))
    w = torch.ones(D, device=DEV)
    call = lambda c: g.qk_norm_rope(q, k, rope, pos, q_weight=w, k_weight=w, v=v, cache=c, slots=slots)[0]  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(cache)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = call(cache)
    for i in range(3):
        rows.copy_(torch.randn(rows.shape, device=DEV).to(torch.bfloat16))
        pos.add_(1000 * i)
        graph.replay()
        torch.cuda.synchronize()
        eager = call(other)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), i
        assert torch.equal(cache.k.view(torch.int16), other.k.view(torch.int16)), i
        assert torch.equal(cache.v.view(torch.int16), other.v.view(torch.int16)), i


def test_more_tokens_than_a_launch_has_workgroups():
    """2^24 tokens and a few more, the heads of all of them one row in memory: token t is what its position makes of it,
    bit by bit the token of a short call at that position."""
    D, few = 64, 1 << 10
    T = (1 << 24) + 5
    say("rope", T)
    gen = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(1, 1, D, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(3))
    rope = g.Rope(torch.logspace(0, -4, 32, device=DEV))
    w = torch.rand(D, generator=gen).to(DEV)
    pos = torch.arange(few, dtype=torch.int32, device=DEV)
    want = g.qk_norm_rope(q.expand(few, 1, D), k.expand(few, 1, D), rope, pos, q_weight=w)
    long = pos.repeat(T // few + 1)[:T]
    got = g.qk_norm_rope(q.expand(T, 1, D), k.expand(T, 1, D), rope, long, q_weight=w)
    for x, y in zip(got, want):
        y = y.view(torch.int16)
        x = x.view(torch.int16)
        assert torch.equal(x[:T - 5].view(-1, few, D), y.view(1, few, D).expand(T // few, few, D))
        assert torch.equal(x[T - 5:], y[:5])
    # into a cache, whose slots are as many
    cache = g.KvCache.empty(T // 64 + 1, 64, 1, D, dtype=torch.float8_e4m3fn, device=DEV)
    slots = torch.arange(T, dtype=torch.int32, device=DEV).flip(0)
    g.qk_norm_rope(q.expand(T, 1, D), k.expand(T, 1, D), rope, long, q_weight=w, v=v.expand(T, 1, D), cache=cache, slots=slots)
    codes = want[1].float().clamp(-448, 448).view(few, D)
    kept = cache.k.view(torch.uint8).view(-1, D)[:T]
    for t in (0, 1, few + 7, (1 << 23) - 1, 1 << 23, (1 << 24) - 1, 1 << 24, T - 1):
        row = kept[T - 1 - t].view(torch.float8_e4m3fn).float()
        # e4m3 from fp32 against e4m3 from the bf16 key: half a step and the bf16 rounding
        assert bool(((row - codes[t % few]).abs() <= codes[t % few].abs() * (E4M3 + BF16) + 2.0 ** -9).all()), t
    values = cache.v.view(torch.uint8).view(-1, D)[:T]
    assert torch.equal(values, values[:1].expand(T, D)) and bool(values.any())
