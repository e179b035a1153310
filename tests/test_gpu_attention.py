"""Attention over a paged cache (paged_attention) against 64 bits (needs an MI355X); tolerances are derived in
attention_util.attend_tolerance."""
from __future__ import annotations

import math

import pytest
import torch

import fp8_block_scaled_a8w8_amd as g
from attention_util import Cache, attend64, attend_tolerance, values

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def heads(T, Hq, D, seed, strided=False, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = (std * torch.randn(T, Hq, (2 if strided else 1) * D, generator=gen)).to(torch.bfloat16)
    return x[..., :D] if strided else x


def check(got, q, c, q_start, lens, news, scale, window=0, sinks=0, gate=None, what="", kv=None):
    """Every sequence's rows of `got` within tolerance of the definition; returns the 64-bit result."""
    k, v = kv or (values(c.k, c.ks), values(c.v, c.vs))
    D, G = q.shape[2], q.shape[1] // c.k.shape[2]
    want, mag, most = attend64(q, k, v, c.table, c.page, q_start, lens, scale, window, sinks, gate)
    got = got.double().cpu()
    for b, n in enumerate(news):
        r = slice(q_start[b], q_start[b] + n)
        tol = attend_tolerance(want[r], mag[r], most[r], D, n * G, max(1, lens[b]))
        same = torch.isnan(want[r]) & torch.isnan(got[r]) | (want[r] == got[r])
        bad = ~(((got[r] - want[r]).abs() <= tol) | same)
        assert not bad.any(), (what, b, int(bad.sum()), bad.nonzero()[:3].tolist(), got[r][bad][:3], want[r][bad][:3])
    return want


def starts(news, first=0):
    s = [first]
    for n in news:
        s.append(s[-1] + n)
    return s


def call(q, c, q_start, lens, ws=None, **kw):
    cache = c.to(DEV)
    if ws is None:
        ws = g.Workspace(g.paged_attention_workspace_bytes(len(q), len(lens), q.shape[1], cache))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return g.paged_attention(q, cache, c.table.to(DEV), i32(q_start), i32(lens), ws, **kw)


CASES = [
    # D, Hkv, G, page, dtype, [(new, length)], window, sinks, gated
    (64, 1, 1, 16, "bf16", [(1, 1)], 0, 0, False),
    (128, 2, 4, 16, "bf16", [(1, 1), (1, 2), (1, 15), (1, 16), (1, 17), (1, 33), (1, 200)], 0, 0, True),
    (128, 2, 4, 16, "fp8", [(1, 1), (1, 31), (1, 129), (1, 1000)], 0, 0, False),
    (256, 4, 6, 64, "bf16", [(1, 501), (1, 64), (1, 2049)], 0, 0, True),
    (256, 1, 16, 32, "fp8", [(1, 700), (1, 5)], 0, 0, True),
    (64, 2, 8, 1, "bf16", [(1, 77), (1, 130)], 0, 0, False),
    (64, 1, 3, 128, "fp8", [(5, 300), (2, 2), (1, 513)], 0, 0, False),
    (128, 1, 1, 16, "bf16", [(16, 16), (16, 90), (17, 90)], 0, 0, False),
    (128, 2, 5, 32, "bf16", [(40, 40), (1, 300), (33, 150), (0, 20)], 0, 0, True),
    (256, 1, 2, 16, "bf16", [(130, 200)], 0, 0, False),
    (256, 2, 6, 64, "fp8", [(70, 70), (9, 400)], 0, 0, True),
    (64, 1, 12, 64, "fp8", [(100, 333)], 0, 0, False),
    (128, 1, 40, 16, "bf16", [(1, 99), (7, 120)], 0, 0, False),
    # windows: shorter than a tile, longer than the sequence, with and without sinks
    (64, 2, 8, 64, "bf16", [(1, 700), (1, 20), (1, 65)], 64, 4, False),
    (128, 1, 4, 16, "bf16", [(1, 900), (3, 500), (150, 400)], 100, 0, False),
    (128, 1, 2, 16, "fp8", [(140, 140), (1, 64)], 1, 0, False),
    (256, 1, 6, 32, "bf16", [(60, 300), (1, 290)], 33, 40, True),
    (128, 1, 1, 16, "bf16", [(200, 600)], 7, 3, False),
    (64, 1, 1, 16, "bf16", [(300, 300)], 1000, 4, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_against_64_bits(case):
    D, Hkv, G, page, dtype, seqs, window, sinks, gated = case
    say("attention", case)
    news, lens = [n for n, _ in seqs], [m for _, m in seqs]
    T, Hq = sum(news) + 3, Hkv * G
    q = heads(T, Hq, D, 1, strided=gated, std=1.5)
    gate = heads(T, Hq, D, 2, strided=True) if gated else None
    c = Cache(lens, Hkv, D, page, dtype, seed=len(seqs))
    qs = starts(news, 1)                             # a row before the first sequence, two behind the last
    sentinel = heads(T, Hq, D, 9)
    for hint in (0, max(news)):
        out = sentinel.to(DEV)
        dq = q.to(DEV) if not gated else torch.cat([q, q], 2).to(DEV)[..., :D]
        dg = None if gate is None else torch.cat([gate, gate], 2).to(DEV)[..., :D]
        r = call(dq, c, qs, lens, window=window, sinks=sinks, gate=dg, max_new=hint, out=out)
        torch.cuda.synchronize()
        assert r is out
        check(out, q, c, qs, lens, news, D ** -0.5, window, sinks, gate, what=f"hint {hint}")
        for t in (0, T - 2, T - 1):
            assert torch.equal(out[t].cpu().view(torch.int16), sentinel[t].view(torch.int16)), t


@pytest.mark.parametrize("D,dtype,hint", [(64, "bf16", 1), (128, "fp8", 0), (256, "bf16", 0)])
def test_long_decode_is_split(D, dtype, hint):
    """Long caches, few rows: the keys are split over many workgroups; ragged lengths beside them."""
    say("long", D, dtype)
    lens, Hkv, G = [20011, 3, 5000], 2, 3
    q = heads(3, Hkv * G, D, 4, std=2.0)
    c = Cache(lens, Hkv, D, 64, dtype, seed=8)
    out = call(q.to(DEV), c, [0, 1, 2, 3], lens, max_new=hint)
    check(out, q, c, [0, 1, 2, 3], lens, [1, 1, 1], D ** -0.5)


@pytest.mark.parametrize("D,dtype", [(64, "fp8"), (128, "bf16"), (256, "bf16")])
def test_chunk_over_long_cache_is_split(D, dtype):
    say("long chunk", D, dtype)
    lens, news, Hkv, G = [6000, 70], [30, 20], 1, 5
    q = heads(50, Hkv * G, D, 4, std=2.0)
    c = Cache(lens, Hkv, D, 32, dtype, seed=9)
    out = call(q.to(DEV), c, [0, 30, 50], lens)
    check(out, q, c, [0, 30, 50], lens, news, D ** -0.5)


@pytest.mark.parametrize("D,dtype,window", [(64, "bf16", 0), (128, "fp8", 0), (256, "bf16", 0), (128, "bf16", 2500)])
def test_few_tiles_with_long_and_short_items(D, dtype, window):
    """The whole call has fewer blocks than would fill the card: runs are longer than an equal share."""
    say("few tiles", D, dtype, window)
    lens, news, Hkv, G = [8453, 300, 41, 2000, 900], [70, 290, 41, 21, 1], 1, 8
    q_start = starts(news)
    q = heads(q_start[-1], Hkv * G, D, 14, std=2.0)
    c = Cache(lens, Hkv, D, 32, dtype, seed=19)
    out = call(q.to(DEV), c, q_start, lens, window=window, sinks=3 if window else 0)
    check(out, q, c, q_start, lens, news, D ** -0.5, window, 3 if window else 0)


@pytest.mark.parametrize("n,G", [(5, 2), (40, 4)])
def test_rows_that_see_nothing_are_zero(n, G):
    """A length shorter than the new rows (the first rows stand before the sequence), empty and negative lengths."""
    D, lens, news = 128, [3, 0, -7, 12], [n, n, n, n]
    q = heads(4 * n, G, D, 5)
    c = Cache(lens, 1, D, 16, "bf16", seed=2)
    out = call(q.to(DEV), c, starts(news), lens)
    want = check(out, q, c, starts(news), lens, news, D ** -0.5)
    assert not out.float().cpu()[n:3 * n].any() and not out.float().cpu()[:n - 3].any()
    assert not want[:n - 3].any()


@pytest.mark.parametrize("n", [1, 50])
def test_bad_pages_and_skipped_sequences(n):
    """Keys in pages outside the cache are not seen; a length past the table ends there; sequences whose rows do not lie
    inside the call are skipped."""
    D, G = 64, 4
    lens = [200, 160, 100]
    c = Cache(lens, 1, D, 16, "bf16", seed=3)
    c.table[0, 2], c.table[0, 5] = -5, len(c.k)
    c.table[1, :] = -1
    c.table = c.table[:, :8].contiguous()             # 128 keys at most
    q = heads(3 * n, G, D, 6)
    out = call(q.to(DEV), c, [0, n, 2 * n, 3 * n], lens)
    check(out, q, c, [0, n, 2 * n, 3 * n], lens, [n, n, n], D ** -0.5)
    assert not out.float().cpu()[n:2 * n].any()
    for bad in ([-1, n, 2 * n, 3 * n], [0, n, 2 * n, 3 * n + 1], [2 * n, n, 2 * n, 3 * n]):
        sentinel = heads(3 * n, G, D, 7)
        out = sentinel.to(DEV)
        call(q.to(DEV), c, bad, lens, out=out)
        want, _, _ = attend64(q, values(c.k, None), values(c.v, None), c.table, 16, bad, lens, D ** -0.5, out=sentinel)
        skipped = [b for b in range(3) if bad[b] < 0 or bad[b + 1] > 3 * n or bad[b + 1] < bad[b]]
        assert len(skipped) == 1
        r = slice(0, n) if skipped[0] == 0 else slice(2 * n, 3 * n)
        assert torch.equal(out[r].cpu().view(torch.int16), sentinel[r].view(torch.int16)), bad
        assert float((out.double().cpu() - want).abs().max()) < 0.05


@pytest.mark.parametrize("D,n,G,window,sinks", [(64, 3, 4, 0, 0), (128, 60, 2, 0, 0), (256, 50, 3, 0, 0),
                                                (128, 60, 2, 20, 2), (128, 3, 4, 40, 2)])
def test_infinities_and_nan_reach_only_rows_that_see_them(D, n, G, window, sinks):
    lens = [130]
    c = Cache(lens, 1, D, 16, "bf16", seed=4)

    def put(x, j, d, value):
        x[int(c.table[0, j // 16]), j % 16, 0, d] = value

    last = lens[0] - 1
    put(c.v, last, 3, math.inf)                       # seen by the last row only
    put(c.v, last - 1, 5, math.nan)                   # by the last two
    put(c.v, last - 1, 6, -math.inf)
    put(c.v, last - n + 1, 7, math.inf)               # by all rows (a window lets go of it)
    put(c.v, last - n + 1, 8, -math.inf)
    put(c.v, last, 8, math.inf)                       # the last row sees both signs (without a window)
    put(c.k, last, 0, math.nan)                       # the last row's softmax is NaN, no other's
    q = heads(n, G, D, 8)
    out = call(q.to(DEV), c, [0, n], lens, window=window, sinks=sinks)
    want = check(out, q, c, [0, n], lens, [n], D ** -0.5, window, sinks)
    finite = torch.isfinite(want)
    assert torch.equal(torch.isfinite(out.float().cpu()), finite)
    assert not finite[-1].any() and finite[0].sum() >= G * (D - 2)


def test_equal_and_extreme_scores():
    """Scores all equal; scores so far apart that one key takes all; scale 0 and a negative scale."""
    D, G, lens = 128, 2, [333]
    c = Cache(lens, 1, D, 16, "bf16", seed=5)
    for std, scale in ((0.0, None), (60.0, None), (1.0, 0.0), (1.0, -0.3), (1.0, 1e-30)):
        for n in (1, 30):
            q = heads(n, G, D, 3, std=std)
            out = call(q.to(DEV), c, [0, n], lens, scale=scale)
            check(out, q, c, [0, n], lens, [n], D ** -0.5 if scale is None else scale, what=(std, scale))


def test_large_cache_offsets_pass_32_bits():
    """A cache of more than 4 GiB per side, the sequence in its last pages."""
    Hkv, D, page, G = 8, 128, 64, 2
    pages = (4 << 30) // (page * Hkv * D * 2) + 3
    k, v = (torch.zeros(pages, page, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    gen = torch.Generator().manual_seed(6)
    small = [torch.randn(2, page, Hkv, D, generator=gen).to(torch.bfloat16) for _ in range(2)]
    k[-2:], v[-2:] = small[0].to(DEV), small[1].to(DEV)
    cache = g.KvCache(k, v)
    for n in (1, 40):
        q = heads(n, Hkv * G, D, 7)
        ws = g.Workspace(g.paged_attention_workspace_bytes(n, 1, Hkv * G, cache))
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        out = g.paged_attention(q.to(DEV), cache, i32([[pages - 2, pages - 1]]), i32([0, n]), i32([100]), ws)
        want, mag, most = attend64(q, small[0].double(), small[1].double(), torch.tensor([[0, 1]]), page, [0, n], [100], D ** -0.5)
        assert bool(((out.double().cpu() - want).abs() <= attend_tolerance(want, mag, most, D, n * G, 100)).all())


def test_same_call_same_bits_and_shared_workspace():
    """Bitwise the same again, on another stream, and after other calls on the workspace."""
    D, lens, news = 128, [9000, 300, 4000], [1, 60, 1]
    q = heads(62, 8, D, 8).to(DEV)
    c = Cache(lens, 2, D, 16, "fp8", seed=6)
    cache = c.to(DEV)
    ws = g.Workspace(g.paged_attention_workspace_bytes(62, 3, 8, cache))
    first = call(q, c, starts(news), lens, ws)
    call(q[:1], c, [0, 1, 1, 1], [40, 0, 0], ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = call(q, c, starts(news), lens, ws)
    s.synchronize()
    assert torch.equal(first.view(torch.int16), second.view(torch.int16))


@pytest.mark.parametrize("hint", [1, 0])
def test_captured_and_replayed_with_other_lengths(hint):
    """The lengths are read on the device: a captured step replays with longer sequences."""
    D, Hkv, G, B = 128, 2, 4, 3
    q = torch.zeros(B, Hkv * G, D, dtype=torch.bfloat16, device=DEV)
    c = Cache([3000, 2000, 700], Hkv, D, 16, "bf16", seed=7)
    cache, table = c.to(DEV), c.table.to(DEV)
    ws, ws2 = (g.Workspace(g.paged_attention_workspace_bytes(B, B, Hkv * G, cache)) for _ in range(2))
    qs = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    lens = torch.tensor([10, 1, 5], dtype=torch.int32, device=DEV)
    run = lambda w: g.paged_attention(q, cache, table, qs, lens, w, max_new=hint)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run(ws)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = run(ws)
    for i, ln in enumerate(([3000, 2000, 700], [17, 400, 0], [2999, 16, 33])):
        host = heads(B, Hkv * G, D, 20 + i)
        q.copy_(host.to(DEV))
        lens.copy_(torch.tensor(ln, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        eager = run(ws2)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), i
        check(out, host, c, [0, 1, 2, 3], ln, [1, 1, 1], D ** -0.5)


def test_two_streams_with_their_own_workspaces():
    D, lens = 128, [6000, 5000]
    c = Cache(lens, 2, D, 64, "bf16", seed=10)
    q = heads(2, 8, D, 11).to(DEV)
    cache = c.to(DEV)
    ws = [g.Workspace(g.paged_attention_workspace_bytes(2, 2, 8, cache)) for _ in range(2)]
    want = call(q, c, [0, 1, 2], lens, ws[0], max_new=1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for i in range(4):
        for s, w, o in zip(streams, ws, outs):
            with torch.cuda.stream(s):
                o.append(call(q, c, [0, 1, 2], lens, w, max_new=1))
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        assert torch.equal(o.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("D,G,n,window", [(128, 1, 700, 100), (64, 2, 400, 50), (256, 1, 300, 0)])
def test_infinities_in_several_tiles(D, G, n, window):
    """Infinite values in many blocks that only part of a tile's rows sees, over several tiles of rows."""
    lens = [n + 40]
    c = Cache(lens, 1, D, 16, "bf16", seed=12)
    for j in range(5, lens[0], 37):
        c.v[int(c.table[0, j // 16]), j % 16, 0, j % D] = math.inf if j % 2 else -math.inf
    q = heads(n, G, D, 9)
    out = call(q.to(DEV), c, [0, n], lens, window=window)
    want = check(out, q, c, [0, n], lens, [n], D ** -0.5, window)
    assert torch.equal(torch.isfinite(out.float().cpu()), torch.isfinite(want))


@pytest.mark.parametrize("D,dtype,hint", [(64, "bf16", 1), (128, "fp8", 5), (256, "bf16", 2)])
def test_hint_smaller_than_the_rows(D, dtype, hint):
    """max_new is a hint: sequences with more rows are served all the same."""
    lens, news, G = [150, 90, 40], [45, 1, 17], 3
    q = heads(63, 2 * G, D, 13)
    c = Cache(lens, 2, D, 32, dtype, seed=13)
    out = call(q.to(DEV), c, starts(news), lens, max_new=hint, window=70, sinks=3)
    # (few rows at a time: the numerators of all sequences are two terms; the bound for one holds)
    check(out, q, c, starts(news), lens, news, D ** -0.5, 70, 3)


@pytest.mark.parametrize("B,hint", [(64, 1), (65, 1), (300, 1), (2048, 1), (130, 0)])
def test_many_sequences(B, hint):
    """Sequences of mixed lengths, empty ones among them; with hint 0 some have chunks."""
    say("sequences", B, hint)
    gen = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 40, (B,), generator=gen).tolist()
    lens[0], lens[B - 1], lens[B // 2] = 700, 650, 300
    news = [1 if n else 0 for n in lens]
    if hint == 0:
        for b in (0, 7, B // 2, B - 1):
            news[b] = min(max(lens[b], 1), 35)
            lens[b] = max(lens[b], news[b])
    q = heads(sum(news), 4, 64, 14)
    c = Cache(lens, 1, 64, 16, "bf16", seed=14)
    out = call(q.to(DEV), c, starts(news), lens, max_new=hint)
    check(out, q, c, starts(news), lens, news, 64 ** -0.5)


def test_more_tiles_than_threads():
    """A prompt of more row tiles than a workgroup has threads (the search for a run goes in several rounds)."""
    D, G, n, page = 64, 64, 900, 64
    for w in (0, 33):
        gen = torch.Generator(device=DEV).manual_seed(15)
        k, v = (torch.randn(15, page, 1, D, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2))
        q = torch.randn(n, G, D, generator=gen, device=DEV).to(torch.bfloat16)
        cache = g.KvCache(k, v)
        ws = g.Workspace(g.paged_attention_workspace_bytes(n, 1, G, cache))
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        out = g.paged_attention(q, cache, i32([list(range(15))]), i32([0, n]), i32([n]), ws, window=w)
        kk, vv = k.view(-1, D)[:n].double(), v.view(-1, D)[:n].double()
        s = (q.double().view(-1, D) @ kk.t()).view(n, G, n) * D ** -0.5
        i, j = torch.arange(n, device=DEV)[:, None], torch.arange(n, device=DEV)[None]
        hidden = (j > i) | ((j <= i - w) if w else torch.zeros_like(j > i))
        p = torch.softmax(s.masked_fill(hidden[:, None], -math.inf), 2)
        want, mag = p @ vv, p @ vv.abs()
        most = (q.double().abs().view(-1, D) @ kk.abs().t()).view(n, G, n).amax(2) * D ** -0.5
        assert bool(((out.double() - want).abs() <= attend_tolerance(want, mag, most, D, n * G, n)).all()), w


@pytest.mark.parametrize("n", [1, 30])
def test_window_behind_the_end_of_the_table(n):
    """Lengths far past the table: the window lies behind every key that can be read; only sinks are seen, or nothing."""
    D, G = 128, 2
    c = Cache([64, 64], 1, D, 16, "bf16", seed=16)
    c.table = c.table[:, :4].contiguous()
    q = heads(2 * n, G, D, 16)
    for sinks in (0, 3):
        out = call(q.to(DEV), c, [0, n, 2 * n], [5000, 2 ** 31 - 1], window=100, sinks=sinks)
        check(out, q, c, [0, n, 2 * n], [5000, 2 ** 31 - 1], [n, n], D ** -0.5, 100, sinks)
        assert bool((out == 0).all()) == (sinks == 0)
