"""Attention over a paged cache: scales, gates and cached values at the ends of what a call may hold (needs an MI355X).
The definition and the tolerances are those of attention_util."""
from __future__ import annotations

import math

import pytest
import torch

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
