"""Steps of the decoder block over a growing cache, each part against 64 bits from what the part before it left (needs an
MI355X)."""
from __future__ import annotations

import pytest
import torch

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
