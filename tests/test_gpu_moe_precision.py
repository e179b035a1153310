"""How near the mixture-of-experts layer for few slots per expert comes to 64 bits (needs an MI355X).

The hidden rows are carried as two bf16 terms (2^-17 of a value each), so the output's own rounding to
bf16 is all that may be seen: fp32 sums of at most 2^13 terms move a row by about 2^-24 * 2^6.5 of the norm
of its terms, so the error is within a twentieth of the rounding's."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_block_scaled_a8w8_amd as g

from gpu_util import DEV, say
from test_gpu_moe import experts_inputs, layer_ref, make_handle

pytestmark = pytest.mark.gpu


# One token (routed inside the up product), a few, and batches whose experts have up to three slots each on
# average; hidden sizes that fill and that end inside a unit of four K blocks.
@pytest.mark.parametrize("T,E,k,H,I,packed", [(1, 8, 1, 512, 256, False), (1, 8, 1, 2048, 640, True), (1, 16, 8, 1024, 384, False),
                                              (2, 8, 1, 1024, 128, False), (5, 32, 4, 640, 512, True), (8, 64, 2, 512, 256, False),
                                              (20, 64, 2, 512, 256, False), (20, 64, 4, 512, 384, True), (33, 32, 2, 384, 256, False),
                                              (61, 64, 3, 384, 640, True)])
def test_only_the_outputs_rounding_is_seen(T, E, k, H, I, packed):
    say("moe layer precision", T, E, k, H, I, packed)
    weights = experts_inputs(E, H, I, seed=7)
    gen = torch.Generator().manual_seed(T + E)
    X = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen)
    ex = make_handle(weights, packed)
    y = g.moe_layer_a16w8_blockscale(X.to(DEV), logits.to(DEV), ex, k, g.Workspace(g.moe_workspace_bytes(T, k, ex)))
    ref = layer_ref(X.double().numpy(), logits.numpy(), weights, k)
    own = np.linalg.norm(torch.from_numpy(ref).to(torch.bfloat16).double().numpy() - ref)
    assert np.linalg.norm(y.double().cpu().numpy() - ref) <= 1.05 * own


def test_infinite_hidden_values_stay_infinite():
    """No second term beside an infinity (infinity minus infinity): the output is infinite, not NaN."""
    T, E, k, H, I = 1, 8, 1, 128, 128
    w13 = torch.full((E, 2 * I, H), 0x38, dtype=torch.uint8, device=DEV)                 # 1.0
    w2 = torch.full((E, H, I), 0x38, dtype=torch.uint8, device=DEV)
    ex = g.MoeExperts(w13, torch.full((E, 2, 1), 2.0 ** 66, device=DEV), w2, torch.ones(E, 1, 1, device=DEV))
    X = torch.ones(T, H, dtype=torch.bfloat16, device=DEV)
    y = g.moe_layer_a16w8_blockscale(X, torch.zeros(T, E, device=DEV), ex, k, g.Workspace(g.moe_workspace_bytes(T, k, ex)))
    assert bool(torch.isposinf(y.float()).all())
