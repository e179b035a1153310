"""The serving block at every batch size that it is made for (needs an MI355X)."""
from __future__ import annotations

import pytest
import torch

import fp8_block_scaled_a8w8_amd as a8w8
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


@pytest.mark.parametrize("T", [3, 40, 200])
def test_the_experts_part_by_itself(T):
    """Expert weights scaled up until the layer's part outweighs x, so that an error of that part shows.  Its
    bound: h, the layer's row and out are rounded to bf16 once each, 2^-9 of the layer's norm at most on average."""
    b = ServingBlock(hidden=512, width=768, experts=12, inter=256, topk=3, adapters=5, rank=16, max_tokens=T)
    b.experts.w2_scale *= 256.0
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T)
    att = torch.randn(T, 768, generator=gen, device=DEV).to(torch.bfloat16)
    res = torch.randn(T, 512, generator=gen, device=DEV).to(torch.bfloat16)
    ids = torch.randint(-1, 5, (T,), generator=gen, device=DEV).to(torch.int32)
    out, logits = b.step(att, res, ids)
    x = res + a8w8.gemm_a8w8_blockscale_lora(att, b.W, b.w_scale, b.adapters, ids, b.workspace)   # the step's own x
    torch.cuda.synchronize()

    def weights(codes, s):
        return codes.double() * s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)

    e, m = b.experts, torch.zeros(T, 512, dtype=torch.float64, device=DEV)
    chosen = torch.sort(logits.double(), dim=1, descending=True, stable=True)
    w = torch.softmax(chosen.values[:, :3], 1)
    for i in range(12):
        gate, up = (x.double() @ weights(e.W13[i], e.w13_scale[i]).t()).chunk(2, 1)
        share = torch.where(chosen.indices[:, :3] == i, w, 0.0).sum(1, keepdim=True)
        m += share * ((gate * torch.sigmoid(gate) * up) @ weights(e.W2[i], e.w2_scale[i]).t())
    assert float(m.norm() / x.double().norm()) > 2.0
    assert float((out.double() - x.double() - m).norm() / m.norm()) <= 3 * 2.0 ** -9
