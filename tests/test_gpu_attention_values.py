"""Attention over a paged cache: scales, gates and cached values at the ends of what a call may hold (needs an MI355X).
The definition and the tolerances are those of attention_util."""
from __future__ import annotations

import math

import pytest
import torch

import fp8_block_scaled_a8w8_amd as g
from attention_util import Cache
from test_gpu_attention import call, check, heads, starts

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [None, -0.2])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [2, 45])
def test_head_scales_of_any_sign_and_none(D, n, scale):
    """Keys are code times the head's scale, whatever its sign: a negative one turns the order of the scores, zero makes them
    equal, NaN and infinity leave NaN in every row that sees a key and nothing in those that see none."""
    say("head scales", D, n, scale)
    lens, news, G = [170, 0, 33], [n, n, n], 2
    c = Cache(lens, 6, D, 16, "fp8", seed=21)
    c.ks *= torch.tensor([1.0, -1.0, 0.0, math.nan, math.inf, -1.0])
    c.vs *= torch.tensor([1.0, 1.0, -1.0, 1.0, 1.0, math.nan])
    q = heads(3 * n, 6 * G, D, 22, std=2.0)
    out = call(q.to(DEV), c, starts(news), lens, scale=scale)
    want = check(out, q, c, starts(news), lens, news, D ** -0.5 if scale is None else scale)
    seen = torch.tensor([t < n or (t >= 2 * n and 33 - 3 * n + t >= 0) for t in range(3 * n)])
    finite = torch.isfinite(out.float().cpu()).view(3 * n, 6, G, D)
    assert bool(finite[:, :3].all()) and bool(finite[~seen].all()) and not finite[seen][:, 3:].any()
    assert float(want[:n].nan_to_num().abs().max()) > 0.1


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp8"), (256, "bf16")])
@pytest.mark.parametrize("n", [2, 45])
def test_gates_of_any_value(D, dtype, n):
    """Gates far out, infinite and NaN: only their own elements follow, and a row that sees no key gets zeros all the same."""
    say("gates", D, dtype, n)
    lens, news, G = [170, 0, 2], [n, n, n], 3
    c = Cache(lens, 2, D, 16, dtype, seed=23)
    q, gate = heads(3 * n, 2 * G, D, 24), heads(3 * n, 2 * G, D, 25)
    gate[..., 5], gate[..., 6], gate[..., 7] = math.nan, math.inf, -math.inf
    gate[..., 8], gate[..., 9], gate[..., 10] = 60.0, -60.0, -3.0e38
    out = call(q.to(DEV), c, starts(news), lens, gate=gate.to(DEV))
    check(out, q, c, starts(news), lens, news, D ** -0.5, gate=gate)
    assert not out.float().cpu()[n:2 * n].any() and not out.float().cpu()[2 * n:3 * n - 2].any()
    nan = torch.isnan(out.float().cpu())
    assert bool(nan[:n, :, 5].all()) and int(nan.sum()) == (n + 2) * 2 * G


def test_handles_follow_their_tensors_memory():
    """A tensor of a handle that got other memory (a cache parked and brought back) is read and written where it is now."""
    D, G = 64, 2
    c = Cache([40], 1, D, 16, "bf16", seed=26)
    cache, rope = c.to(DEV), g.Rope(torch.logspace(0, -3, 16, device=DEV))
    q = heads(1, G, D, 27).to(DEV)
    ws = g.Workspace(g.paged_attention_workspace_bytes(1, 1, G, cache))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    args = (c.table.to(DEV), i32([0, 1]), i32([40]), ws)
    want = g.paged_attention(q, cache, *args)
    turned, _ = g.qk_norm_rope(q, q[:, :1], rope, i32([5]))
    old = [t.detach() for t in (cache.k, cache.v, rope.inv_freq)]     # (the old memory stays allocated)
    for t in (cache.k, cache.v, rope.inv_freq):
        t.data = t.detach().clone()
    for t in old:
        t.zero_()
    assert torch.equal(g.paged_attention(q, cache, *args), want)
    assert torch.equal(g.qk_norm_rope(q, q[:, :1], rope, i32([5]))[0], turned)
    g.qk_norm_rope(q, q[:, :1], rope, i32([5]), v=q[:, 1:], cache=cache, slots=i32([3]))
    assert not any(t.any() for t in old) and torch.equal(cache.v.view(-1, 1, D)[3], q[0, 1:])


def put_nan(c, j, d, sign):
    """The 8-bit type's NaN, either sign, at key j of sequence 0."""
    c.v.view(torch.uint8)[int(c.table[0, j // c.page]), j % c.page, 0, d] = 0xff if sign else 0x7f


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,G,window,sinks", [(3, 4, 0, 0), (3, 4, 40, 2), (60, 2, 0, 0), (60, 3, 20, 2), (300, 1, 100, 5)])
def test_nan_codes_reach_only_rows_that_see_them(D, n, G, window, sinks):
    """NaN codes among the values (and one among the keys) of an 8-bit cache, at keys that only part of a tile's rows sees."""
    say("nan codes", D, n, G, window)
    lens = [n + 90]
    c = Cache(lens, 1, D, 16, "fp8", seed=31)
    last = lens[0] - 1
    put_nan(c, last, 3, 0)                            # seen by the last row only
    put_nan(c, last - 1, 5, 1)                        # by the last two
    put_nan(c, last - n + 1, 7, 0)                    # by all rows (a window lets go of it)
    put_nan(c, 1, 11, 1)                              # a sink, if there are any
    for i, j in enumerate(range(40, last - 4, 29)):   # (many tiles: in blocks that rows begin and end to see)
        put_nan(c, j, 16 + i % (D - 16), i % 2)
    c.k.view(torch.uint8)[int(c.table[0, last // 16]), last % 16, 0, 0] = 0x7f       # the last row's softmax is NaN, no other's
    q = heads(n, G, D, 32)
    out = call(q.to(DEV), c, [0, n], lens, window=window, sinks=sinks)
    want = check(out, q, c, [0, n], lens, [n], D ** -0.5, window, sinks)
    finite = torch.isfinite(want)
    assert torch.equal(torch.isfinite(out.float().cpu()), finite)
    assert not finite[-1].any() and finite[0].any() and not finite[0].all()


@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3)])
@pytest.mark.parametrize("D,dtype,page", [(64, "bf16", 1), (64, "bf16", 2), (64, "bf16", 4), (128, "bf16", 1), (128, "bf16", 2),
                                          (256, "bf16", 1), (64, "fp8", 1), (64, "fp8", 8), (128, "fp8", 4), (256, "fp8", 2)])
def test_prompts_over_pages_smaller_than_a_copy(D, dtype, page, window, sinks):
    """Pages of fewer keys than a copy of the kernel of many rows has rows: each key's page is looked up by itself."""
    say("small pages", D, dtype, page, window)
    lens, news, G = [333, 70], [97, 70], 2
    q = heads(167, 2 * G, D, 33, std=1.5)
    c = Cache(lens, 2, D, page, dtype, seed=33)
    c.table[0, 100 // page] = -1                      # (and one that is not there)
    out = call(q.to(DEV), c, starts(news), lens, window=window, sinks=sinks)
    check(out, q, c, starts(news), lens, news, D ** -0.5, window, sinks)


@pytest.mark.parametrize("n", [2, 20])
def test_queries_and_gates_whose_rows_lie_far_apart(n):
    """Row offsets of queries and gates past 2^31 elements."""
    D, G, lens = 64, 2, [40]
    row = (2 ** 31 + 64) // (n - 1) // 8 * 8 + 8
    c = Cache(lens, 1, D, 16, "bf16", seed=34)
    host = [heads(n, G, D, s) for s in (35, 36)]
    base = torch.empty((n - 1) * row + 2 * G * D, dtype=torch.bfloat16, device=DEV)
    q, gate = (base[i * G * D:].as_strided((n, G, D), (row, D, 1)) for i in range(2))
    for there, here in zip((q, gate), host):
        there.copy_(here.to(DEV))
    assert (n - 1) * row > 2 ** 31
    out = call(q, c, [0, n], lens, gate=gate)
    check(out, host[0], c, [0, n], lens, [n], D ** -0.5, gate=host[1])
    turned, _ = g.qk_norm_rope(q, gate[:, :1], None, None, q_weight=torch.ones(D, device=DEV))
    again, _ = g.qk_norm_rope(host[0].to(DEV), host[1].to(DEV)[:, :1], None, None, q_weight=torch.ones(D, device=DEV))
    assert torch.equal(turned, again)
