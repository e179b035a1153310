"""The decoder block: qkv projection, norms and rotation into the paged cache, attention over it, and the weight half,
run together as a serving program runs them (needs an MI355X).

The attention is checked against 64 bits from the block's own projections (the GEMM has tests of its own) over several
steps -- prompts, a chunk beside decoded tokens, decoded tokens alone.  The cache holds k after norm and rotation, and v,
rounded once: relative to the 64-bit history that is BF16 (E4M3 for the 8-bit cache) of each cached value.  Scores are
off by that times sum |q||k| / sqrt(D), which is taken as the weights' relative error twice (numerator and
denominator); values add their own rounding times the weights; q's rounding adds BF16 to the scores; the result's own
rounding and the numerators' BF16 each."""
from __future__ import annotations

import pytest
import torch

import fp8_block_scaled_a8w8_amd as g
from attention_util import BF16, E4M3, rotate64
from fp8_block_scaled_a8w8_amd.serving_block import DecoderBlock, page_batch

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def block(dtype=torch.bfloat16, **kw):
    f = dict(hidden=256, q_heads=6, kv_heads=2, head_dim=64, rotary_dim=32, pages=64, page_size=16, max_tokens=128, max_seqs=4,
             cache_dtype=dtype, experts=8, inter=128, topk=2, adapters=3, rank=8)
    f.update(kw)
    return DecoderBlock(**f)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_steps_against_64_bits(dtype):
    b = block(dtype)
    D, H, G = b.head_dim, b.q_heads, b.q_heads // b.kv_heads
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    step_eps = BF16 if dtype == torch.bfloat16 else E4M3
    keys, vals = [[], [], []], [[], [], []]
    lens = [0, 0, 0]
    for new in ([40, 1, 17], [1, 30, 1], [1, 1, 1], [1, 1, 1]):
        lens = [a + n for a, n in zip(lens, new)]
        say("decoder step", new, lens)
        x = torch.randn(sum(new), 256, generator=gen, device=DEV).to(torch.bfloat16)
        # sequences grow: pages are laid out for the longest they get
        batch = page_batch([64] * 3, new, 16)
        pos = torch.tensor([p for n, m in zip(lens, new) for p in range(n - m, n)], dtype=torch.int32)
        slots = torch.tensor([64 * i + p for i, (n, m) in enumerate(zip(lens, new)) for p in range(n - m, n)], dtype=torch.int32)
        args = (pos.to(DEV), slots.to(DEV), batch[2], batch[3], torch.tensor(lens, dtype=torch.int32, device=DEV))
        att = b.attend(x, *args, max_new=max(new)).double().cpu().view(-1, H, D)
        q, gate, k, v = (t.cpu() for t in b.qkv(x))
        inv = b.rope.inv_freq.cpu()
        q64, _ = rotate64(q, b.q_weight.cpu(), 1e-6, pos, inv, None, "halves")
        k64, _ = rotate64(k, b.k_weight.cpu(), 1e-6, pos, inv, None, "halves")
        t = 0
        for i, m in enumerate(new):
            for j in range(m):
                keys[i].append(k64[t + j])
                vals[i].append(v[t + j].double())
            kk, vv = torch.stack(keys[i]), torch.stack(vals[i])
            for j in range(m):
                n = lens[i] - m + j + 1
                for h in range(H):
                    s = kk[:n, h // G] @ q64[t, h] * D ** -0.5
                    w = torch.softmax(s, 0)
                    sig = torch.sigmoid(gate[t, h].double())
                    want = w @ vv[:n, h // G] * sig
                    mag = w @ vv[:n, h // G].abs() * sig
                    ds = (step_eps + BF16 * 1.01) * float((kk[:n, h // G].abs() @ q64[t, h].abs()).max()) * D ** -0.5
                    # (8 bits: values below 2^-6 of a step of 1/32 round by half a step of 2^-9 / 32)
                    tol = mag * (2 * ds + step_eps + BF16) * 1.05 + want.abs() * BF16 + 2.0 ** -15
                    assert bool(((att[t, h] - want).abs() <= tol).all()), (i, j, h)
                t += 1
    out, logits = b.layer(x, torch.zeros(len(x), dtype=torch.int32, device=DEV), *args, max_new=1)
    again, _ = b.step(b.attend(x, *args, max_new=1), x, torch.zeros(len(x), dtype=torch.int32, device=DEV))
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and tuple(logits.shape) == (3, 8)


def test_replayed_graph_equals_eager():
    """A captured decode step replays with new tokens, positions, slots and lengths."""
    b = block(pages=64, max_seqs=3)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    for side in (b.cache.k, b.cache.v):
        side.copy_(torch.randn(side.shape, generator=gen, device=DEV))
    x = torch.randn(3, 256, generator=gen, device=DEV).to(torch.bfloat16)
    ids = torch.tensor([0, -1, 2], dtype=torch.int32, device=DEV)
    table = page_batch([160, 320, 320], [1, 1, 1], 16)[2]
    starts = torch.arange(4, dtype=torch.int32, device=DEV)
    pos, slots, lens = (torch.zeros(3, dtype=torch.int32, device=DEV) for _ in range(3))

    def place(n):
        p = torch.tensor(n, dtype=torch.int32, device=DEV) - 1
        pos.copy_(p)
        slots.copy_(table.gather(1, (p // 16)[:, None].long())[:, 0] * 16 + p % 16)
        lens.copy_(p + 1)

    run = lambda: b.layer(x, ids, pos, slots, table, starts, lens, max_new=1)[0]  # noqa: E731
    place([100, 300, 7])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = run()
    for i, n in enumerate(([100, 300, 7], [101, 17, 8], [160, 320, 1])):
        x.copy_(torch.randn(3, 256, generator=gen, device=DEV).to(torch.bfloat16))
        place(n)
        graph.replay()
        torch.cuda.synchronize()
        eager = run()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), i


def test_workspace_serves_both_halves():
    b = block()
    assert b.workspace.nbytes >= g.paged_attention_workspace_bytes(128, 4, 6, b.cache)
