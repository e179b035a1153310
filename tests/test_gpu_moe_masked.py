"""Batches of the mixture-of-experts layer that reach few experts or none (needs an MI355X).

The expected rows are exact: a token whose logits are all masked gets a row of zeros, whatever
its activations, the weights and the workspace hold."""
from __future__ import annotations

import pytest
import torch

import fp8_block_scaled_a8w8_amd as g

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def handle(E, H, I, gen, packed=False):
    """Expert weights of random finite codes; the scales are infinite, so that no product of theirs is a zero."""
    w13, w2 = (torch.randint(0, 127, s, generator=gen, device=DEV, dtype=torch.uint8) for s in ((E, 2 * I, H), (E, H, I)))
    s13, s2 = (torch.full(s, float("inf"), device=DEV) for s in ((E, 2 * I // 128, H // 128), (E, H // 128, I // 128)))
    return g.MoeExperts(w13, s13, w2, s2, packed=packed)


def adapters_call(space, gen):
    """A call of another layer on the same workspace: 64 rows of 256 fp8 codes land where the layer keeps its plan."""
    M, N, K = 64, 256, 4096
    ad = g.LoraAdapters(torch.randn(2, 8, K, generator=gen, device=DEV).to(torch.bfloat16),
                        torch.randn(2, N, 8, generator=gen, device=DEV).to(torch.bfloat16), torch.ones(2, device=DEV))
    X = torch.randn(M, K, generator=gen, device=DEV).to(torch.bfloat16)
    W = torch.randint(0, 127, (N, K), generator=gen, device=DEV, dtype=torch.uint8)
    ws = torch.ones(N // 128, K // 128, device=DEV)
    need = g.lora_workspace_bytes(M, N, K, ad)
    assert need <= space.nbytes
    return g.gemm_a8w8_blockscale_lora(X, W, ws, ad, torch.zeros(M, dtype=torch.int32, device=DEV), space)


# T = 3 routes inside the up product, T = 20 in a launch of its own; a narrow H splits the down product's
# units over several workgroups, a wide one does not; I = 640 ends inside a unit of four K blocks.
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("H,I", [(128, 1024), (128, 640), (8192, 128)])
@pytest.mark.parametrize("T,k", [(3, 2), (3, 8), (20, 2), (20, 8)])
def test_no_token_reaches_an_expert(T, k, H, I, packed):
    say("moe layer, all masked", T, k, H, I, packed)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T + H + I)
    E = 64
    ex = handle(E, H, I, gen, packed)
    space = g.Workspace(max(g.moe_workspace_bytes(T, k, ex), 8 << 20))
    X = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    for masked in (float("-inf"), float("nan")):
        adapters_call(space, gen)
        out = torch.full((T, H), 7.0, dtype=torch.bfloat16, device=DEV)
        g.moe_layer_a16w8_blockscale(X, torch.full((T, E), masked, device=DEV), ex, k, space, out=out)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), torch.zeros_like(out).view(torch.int16))


@pytest.mark.parametrize("T", [3, 20])
def test_one_token_reaches_the_last_expert(T):
    """The last expert's last blocks: the unit of the last weights, scales and hidden rows of every buffer."""
    E, k, H, I = 64, 2, 128, 640
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T)
    ex = handle(E, H, I, gen)
    ex.w13_scale.fill_(2.0 ** -12)
    ex.w2_scale.fill_(2.0 ** -12)
    space = g.Workspace(max(g.moe_workspace_bytes(T, k, ex), 8 << 20))
    adapters_call(space, gen)
    X = torch.randn(T, H, generator=gen, device=DEV).to(torch.bfloat16)
    logits = torch.full((T, E), float("-inf"), device=DEV)
    logits[T - 1, E - 1] = 0.0
    y = g.moe_layer_a16w8_blockscale(X, logits, ex, k, space)
    torch.cuda.synchronize()
    assert torch.count_nonzero(y[:T - 1]).item() == 0
    w13 = ex.W13[E - 1].view(torch.float8_e4m3fn).double() * 2.0 ** -12
    w2 = ex.W2[E - 1].view(torch.float8_e4m3fn).double() * 2.0 ** -12
    gate, up = (w13 @ X[T - 1].double()).chunk(2)
    ref = w2 @ (gate * torch.sigmoid(gate) * up)
    # one rounding of h and one of Y to bf16, 2^-8 of the norm at most each
    assert float((y[T - 1].double() - ref).norm() / ref.norm()) <= 2 * 2.0 ** -8


# 8 tokens route inside the up product; 20 and 60 take the down product for few slots, 100 the one for many.
@pytest.mark.parametrize("T,pads", [(8, 3), (20, 5), (60, 9), (100, 30)])
def test_padding_rows_do_not_matter(T, pads):
    """Wherever the padding rows of a batch lie and whatever they hold, the other rows keep their bits (the
    same experts are reached, by the same tokens in the same order), and the batch without them gives the same
    rows up to the order of the sums and the roundings of h and Y (2^-8 of the norm)."""
    E, k, H, I = 16, 2, 256, 384
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T)
    ex = handle(E, H, I, gen)
    ex.w13_scale.fill_(2.0 ** -12)
    ex.w2_scale.fill_(2.0 ** -12)
    space = g.Workspace(g.moe_workspace_bytes(T, k, ex))
    X = torch.randn(T - pads, H, generator=gen, device=DEV).to(torch.bfloat16)
    logits = torch.randn(T - pads, E, generator=gen, device=DEV)
    alone = g.moe_layer_a16w8_blockscale(X, logits, ex, k, space)
    first = None
    for value, spread in ((0.0, False), (float("nan"), False), (float("inf"), True), (1.0, True)):
        live = torch.ones(T, dtype=torch.bool, device=DEV)
        live[(torch.arange(pads, device=DEV) * (T // pads)) if spread else torch.arange(T - pads, T, device=DEV)] = False
        Xp = torch.full((T, H), value, dtype=torch.bfloat16, device=DEV)
        lp = torch.full((T, E), float("-inf"), device=DEV)
        Xp[live], lp[live] = X, logits
        y = g.moe_layer_a16w8_blockscale(Xp, lp, ex, k, space)
        torch.cuda.synchronize()
        assert torch.count_nonzero(y[~live]).item() == 0
        first = y[live] if first is None else first
        assert torch.equal(y[live].view(torch.int16), first.view(torch.int16)), (value, spread)
    assert float((first.double() - alone.double()).norm() / alone.double().norm()) <= 2.0 ** -8
