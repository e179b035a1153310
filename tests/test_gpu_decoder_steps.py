"""Steps of the decoder block over a growing cache, each part against 64 bits from what the part before it left (needs an
MI355X)."""
from __future__ import annotations

import pytest
import torch

import fp8_block_scaled_a8w8_amd as g
from attention_util import BF16, E4M3, EPS32, attend64, attend_tolerance, rotate64, values
from fp8_block_scaled_a8w8_amd.serving_block import page_batch
from test_gpu_decoder_block import block

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[], [20, 0]])
def test_a_step_of_no_tokens(lens):
    """A step whose sequences bring nothing: empty results, the cache as it was."""
    say("no tokens", lens)
    b = block()
    b.cache.k.fill_(1.5)
    x = torch.zeros(0, 256, dtype=torch.bfloat16, device=DEV)
    batch = page_batch(lens, [0] * len(lens), 16)
    assert tuple(b.attend(x, *batch).shape) == (0, b.q_heads * b.head_dim)
    out, logits = b.layer(x, torch.zeros(0, dtype=torch.int32, device=DEV), *batch)
    assert tuple(out.shape) == (0, 256) and tuple(logits.shape) == (0, 8)
    assert bool((b.cache.k == 1.5).all()) and not b.cache.v.any()


@pytest.mark.parametrize("dtype,sizes", [(torch.bfloat16, {}), (torch.float8_e4m3fn, {}),
                                         (torch.float8_e4m3fn, dict(q_heads=8, kv_heads=1, head_dim=128, rotary_dim=128)),
                                         (torch.bfloat16, dict(q_heads=2, kv_heads=2, head_dim=256, rotary_dim=64))])
def test_each_part_against_64_bits(dtype, sizes):
    """Prompts, a chunk beside decoded tokens, decoded tokens alone, past the ends of pages.  The new entries of the cache are
    the rounded 64-bit values of the block's own projection (tolerances as in the rotation's tests), every other entry is
    as it was, and the output is attention over the cache's entries as they are: the bound is the attention's own."""
    b = block(dtype, **sizes)
    D, H, page, room = b.head_dim, b.kv_heads, 16, 100
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    inv, scales = b.rope.inv_freq.cpu(), (b.cache.k_scale, b.cache.v_scale)
    lens = [0, 0, 0]
    for new in ([40, 1, 17], [1, 30, 14], [1, 1, 1], [0, 1, 1], [1, 1, 1], [37, 2, 1]):
        lens = [n + m for n, m in zip(lens, new)]
        say("decoder step", new, lens)
        x = torch.randn(sum(new), 256, generator=gen, device=DEV).to(torch.bfloat16)
        batch = page_batch(lens, new, page, room=room)
        positions, slots, table, starts, _ = (t.cpu() for t in batch)
        q, gate, k, v = b.qkv(x)
        before = [c.view(torch.uint8).clone() for c in (b.cache.k, b.cache.v)]
        out = b.attend(x, *batch, max_new=max(new)).double().cpu().view(sum(new), -1, D)
        k64, kmag = rotate64(k.cpu(), b.k_weight.cpu(), 1e-6, positions, inv, None, "halves")
        kept = slots.long()
        for cache, old, want, mag, s in ((b.cache.k, before[0], k64, kmag, scales[0]),
                                         (b.cache.v, before[1], v.cpu().double(), torch.zeros(sum(new), H, D), scales[1])):
            got = values(cache, s).view(-1, H, D)[kept]
            near = (D / 2 + 17) * EPS32 * mag
            # (steps of the 8-bit type below 2^-6 of the scale are 2^-9 of it)
            half = BF16 * (want.abs() + near) if s is None else torch.maximum(E4M3 * (want.abs() + near), 2.0 ** -10 * s.cpu().double()[:, None])
            assert bool(((got - want).abs() <= near + half + 1e-37).all())
            other = torch.ones(len(old) * page, dtype=torch.bool, device=DEV)
            other[kept.to(DEV)] = False
            assert torch.equal(cache.view(torch.uint8).view(len(other), -1)[other], old.view(len(other), -1)[other])
        turned, _ = g.qk_norm_rope(q, k, b.rope, batch[0], q_weight=b.q_weight, k_weight=b.k_weight)
        q64, qmag = rotate64(q.cpu(), b.q_weight.cpu(), 1e-6, positions, inv, None, "halves")
        near = (D / 2 + 16) * EPS32 * qmag
        assert bool(((turned.double().cpu() - q64).abs() <= near + BF16 * (q64.abs() + near) + 1e-37).all())
        want, mag, most = attend64(turned, values(b.cache.k, scales[0]), values(b.cache.v, scales[1]), table, page, starts, lens,
                                   D ** -0.5, gate=gate)
        for i, m in enumerate(new):
            r = slice(int(starts[i]), int(starts[i + 1]))
            tol = attend_tolerance(want[r], mag[r], most[r], D, m * b.q_heads // H, max(1, lens[i]))
            assert bool(((out[r] - want[r]).abs() <= tol).all()), (new, i)
