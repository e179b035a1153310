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
