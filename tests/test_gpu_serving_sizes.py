"""The serving block at every batch size that it is made for (needs an MI355X)."""
from __future__ import annotations

import pytest
import torch

from fp8_block_scaled_a8w8_amd.serving_block import ServingBlock

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most,sizes", [(600, (600, 513, 512, 300, 40, 1)), (192, (192, 191, 17, 2))])
def test_fewer_tokens_than_the_most(most, sizes):
    """One workspace, sized for the most tokens, serves every smaller batch; rows do not depend on what it held."""
    b = ServingBlock(hidden=1024, width=512, experts=32, inter=768, topk=1, adapters=5, rank=16, max_tokens=most)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(most)
    for T in sizes:
        say("serving block", most, T)
        att = torch.randn(T, 512, generator=gen, device=DEV).to(torch.bfloat16)
        res = torch.randn(T, 1024, generator=gen, device=DEV).to(torch.bfloat16)
        ids = torch.randint(-1, 5, (T,), generator=gen, device=DEV).to(torch.int32)
        out, logits = b.step(att, res, ids)
        # x and the layer are each rounded to bf16, 2^-9 of the norm at most on average (as for the block's own check)
        assert b.error(att, res, ids, out, logits) <= 3 * 2.0 ** -9, T
