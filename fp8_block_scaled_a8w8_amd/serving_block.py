"""A decoder block in serving, on fp8 block-scaled weights.

``ServingBlock`` is the weight half: one step takes the attention's output and the residual stream of a batch of tokens -- each
token of its own request, with its own low-rank adapter or none -- through

    x   = residual + projection(attention output) with the token's adapter
    out = x + mixture of experts(x), routed by x's logits

with the library's calls in the order and on the buffers that a serving program keeps:
handles for the adapters and the experts' weights, one workspace for the stream, and no
allocation in the step that a HIP graph could not replay.  ``DecoderBlock`` puts the attention
half before it:

    q, gate, k, v = qkv projection(x)
    q, k  = norms and rotation; k, v into the paged cache
    attention output = attention of the new tokens over the cache * sigmoid(gate)

    python -m fp8_block_scaled_a8w8_amd.serving_block [--tokens 16] [--steps 50]

runs both on synthetic weights, eagerly and as a replayed graph, and prints the time per
step and the experts' load.
"""
from __future__ import annotations

import argparse

import torch

import fp8_block_scaled_a8w8_amd as a8w8


def quantise_weights(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """Weights [..., N, K] (N and K multiples of 128) as e4m3fn codes and one fp32 scale per 128x128 block."""
    *lead, N, K = w.shape
    blocks = w.float().view(*lead, N // 128, 128, K // 128, 128)
    s = blocks.abs().amax(dim=(-3, -1)).clamp(min=1e-12) / 448.0
    codes = (blocks / s[..., :, None, :, None]).to(torch.float8_e4m3fn).view(*lead, N, K)
    return codes, s.contiguous()


class ServingBlock:
    """Weights, handles and workspace of one block, for up to ``max_tokens`` tokens a step."""

    def __init__(self, hidden: int, width: int, experts: int, inter: int, topk: int, adapters: int, rank: int,
                 max_tokens: int, seed: int = 0, device: str = "cuda"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(*shape, generator=gen, device=device) * std

        self.topk = topk
        self.W, self.w_scale = quantise_weights(normal(hidden, width, std=0.02))
        self.adapters = a8w8.LoraAdapters(normal(adapters, rank, width, std=width ** -0.5).to(torch.bfloat16),
                                          normal(adapters, hidden, rank, std=0.05).to(torch.bfloat16),
                                          torch.ones(adapters, device=device))
        self.gate = normal(experts, hidden, std=hidden ** -0.5)
        self.experts = a8w8.MoeExperts(*quantise_weights(normal(experts, 2 * inter, hidden, std=0.02)),
                                       *quantise_weights(normal(experts, hidden, inter, std=0.02)))
        # calls of one stream share a workspace
        self.workspace = a8w8.Workspace(max(a8w8.lora_workspace_bytes(max_tokens, hidden, width, self.adapters),
                                            a8w8.moe_workspace_bytes(max_tokens, topk, self.experts)), device=device)

    def step(self, attention: torch.Tensor, residual: torch.Tensor, adapter_ids: torch.Tensor) -> tuple:
        """(out bf16 [T,hidden], logits float32 [T,experts]) of T tokens; adapter_ids int32 [T], -1: none."""
        y = a8w8.gemm_a8w8_blockscale_lora(attention, self.W, self.w_scale, self.adapters, adapter_ids, self.workspace)
        x = residual + y
        logits = x.float() @ self.gate.t()
        return x + a8w8.moe_layer_a16w8_blockscale(x, logits, self.experts, self.topk, self.workspace), logits

    def error(self, attention, residual, adapter_ids, out, logits) -> float:
        """Relative 2-norm distance of a step's output from the same step in fp32 torch operations, row by row."""
        def weights(w, s):
            return w.float() * s.repeat_interleave(128, -2).repeat_interleave(128, -1)

        codes, scales = a8w8.quantize_1x128(attention)
        y = (codes.float() * scales.repeat_interleave(128, 1)) @ weights(self.W, self.w_scale).t()
        A, B, scaling = self.adapters.A.float(), self.adapters.B.float(), self.adapters.scaling
        for t, a in enumerate(adapter_ids.tolist()):
            if a >= 0:
                y[t] += scaling[a] * (B[a] @ (A[a] @ attention[t].float()))
        x = (residual + y.to(torch.bfloat16)).float()
        e, ref = self.experts, x.clone()
        for t, (row, ids) in enumerate(zip(*a8w8.moe_route(logits, self.topk))):
            for w, i in zip(row, ids.tolist()):
                gate, up = (weights(e.W13[i], e.w13_scale[i]) @ x[t]).chunk(2)
                ref[t] += w * (weights(e.W2[i], e.w2_scale[i]) @ (torch.nn.functional.silu(gate) * up))
        return float((out.float() - ref).norm() / ref.norm())

    def load(self, logits: torch.Tensor) -> torch.Tensor:
        """Tokens per expert, from the same routing (what a serving program watches)."""
        _, ids = a8w8.moe_route(logits, self.topk)
        return torch.bincount(ids[ids >= 0].long(), minlength=self.experts.E)


class DecoderBlock(ServingBlock):
    """A whole decoder block: gated attention of ``q_heads`` heads of ``head_dim`` over a paged cache of ``pages`` pages, then
    the weight half.  Serves up to ``max_tokens`` new tokens of up to ``max_seqs`` sequences a step."""

    def __init__(self, hidden: int, q_heads: int, kv_heads: int, head_dim: int, rotary_dim: int, pages: int, page_size: int,
                 max_tokens: int, max_seqs: int, cache_dtype=torch.bfloat16, theta: float = 1e6, seed: int = 0,
                 device: str = "cuda", **weight_half):
        super().__init__(hidden, q_heads * head_dim, max_tokens=max_tokens, seed=seed, device=device, **weight_half)
        gen = torch.Generator(device=device)
        gen.manual_seed(seed + 1)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        rows = (2 * q_heads + 2 * kv_heads) * head_dim          # each query head with its gate behind it, keys, values
        self.Wqkv, self.wqkv_scale = quantise_weights(torch.randn(rows, hidden, generator=gen, device=device) * 0.02)
        self.q_weight, self.k_weight = (1.0 + 0.1 * torch.randn(head_dim, generator=gen, device=device) for _ in "qk")
        freq = theta ** (-torch.arange(0, rotary_dim, 2, device=device).double() / rotary_dim)
        self.rope = a8w8.Rope(freq.float())
        scale = torch.full((kv_heads,), 1 / 32, device=device) if cache_dtype == torch.float8_e4m3fn else None
        self.cache = a8w8.KvCache.empty(pages, page_size, kv_heads, head_dim, cache_dtype, scale, scale, device=device)
        need = a8w8.paged_attention_workspace_bytes(max_tokens, max_seqs, q_heads, self.cache)
        if need > self.workspace.nbytes:
            self.workspace = a8w8.Workspace(need, device=device)

    def qkv(self, x: torch.Tensor) -> tuple:
        """(q, gate, k, v) of bf16 x [T,hidden]: views into the projection's rows."""
        rows = a8w8.gemm_a8w8_blockscale(*a8w8.quantize_1x128(x), self.Wqkv, self.wqkv_scale, workspace=self.workspace)
        q, k, v = rows.split((2 * self.q_heads * self.head_dim, *(self.kv_heads * self.head_dim,) * 2), 1)
        q = q.view(len(x), self.q_heads, 2 * self.head_dim)
        k, v = (t.view(len(x), self.kv_heads, self.head_dim) for t in (k, v))
        return q[..., :self.head_dim], q[..., self.head_dim:], k, v

    def attend(self, x, positions, slots, page_table, q_start, kv_lens, max_new: int = 0) -> torch.Tensor:
        """The attention's output bf16 [T,q_heads*head_dim] of the new tokens x [T,hidden] (int32 positions and cache slots
        [T]; page table, first rows and lengths of the sequences as paged_attention takes them)."""
        q, gate, k, v = self.qkv(x)
        q, _ = a8w8.qk_norm_rope(q, k, self.rope, positions, q_weight=self.q_weight, k_weight=self.k_weight, v=v,
                                 cache=self.cache, slots=slots)
        out = a8w8.paged_attention(q, self.cache, page_table, q_start, kv_lens, self.workspace, gate=gate, max_new=max_new)
        return out.flatten(1)

    def layer(self, x, adapter_ids, positions, slots, page_table, q_start, kv_lens, max_new: int = 0) -> tuple:
        """(out bf16 [T,hidden], logits) of the whole block."""
        attention = self.attend(x, positions, slots, page_table, q_start, kv_lens, max_new)
        return self.step(attention, x, adapter_ids)


def page_batch(lens, new, page_size: int, device: str = "cuda", room=None) -> tuple:
    """(positions, slots, page table, q_start, kv_lens) of sequences of ``lens`` tokens, the last ``new`` of each new, on
    pages one sequence after another from page 0 on.  Each sequence gets the pages of ``room`` tokens (a number or one
    each; None: of its ``lens``).  A batch of the same sequences grown longer finds their cache only where both calls
    have the same ``room``."""
    room = list(lens) if room is None else [room] * len(lens) if isinstance(room, int) else list(room)
    if not len(lens) == len(new) == len(room) or any(not 0 <= m <= n <= r for n, m, r in zip(lens, new, room)):
        raise ValueError(f"each sequence needs 0 <= new <= tokens <= room, got {list(new)} {list(lens)} {room}")
    per = [-(-r // page_size) for r in room]
    first = [sum(per[:b]) for b in range(len(per))]
    table = torch.full((len(lens), max(per, default=0)), -1, dtype=torch.int32)
    positions, slots, starts = [], [], [0]
    for b, (n, m) in enumerate(zip(lens, new)):
        table[b, :per[b]] = torch.arange(first[b], first[b] + per[b])
        positions += range(n - m, n)
        slots += range(first[b] * page_size + n - m, first[b] * page_size + n)
        starts.append(starts[-1] + m)
    return tuple(torch.as_tensor(t, dtype=torch.int32).to(device) for t in (positions, slots, table, starts, lens))


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--steps", type=int, default=50)
    args = ap.parse_args(argv)
    T = args.tokens
    block = ServingBlock(hidden=2048, width=4096, experts=64, inter=768, topk=8, adapters=32, rank=16, max_tokens=T)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    attention = torch.randn(T, 4096, generator=gen, device="cuda").to(torch.bfloat16)
    residual = torch.randn(T, 2048, generator=gen, device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, 32, (T,), generator=gen, device="cuda").to(torch.int32)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        out, logits = block.step(attention, residual, ids)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        block.step(attention, residual, ids)

    def timed(run) -> float:
        for _ in range(3):
            run()
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        for _ in range(args.steps):
            run()
        t1.record()
        t1.synchronize()
        return t0.elapsed_time(t1) * 1e3 / args.steps

    eager, replay = timed(lambda: block.step(attention, residual, ids)), timed(graph.replay)
    load = block.load(logits)
    print(f"{T} tokens: {eager:.1f} us a step, {replay:.1f} us replayed; {int((load > 0).sum())} of {len(load)} experts "
          f"reached, the busiest by {int(load.max())} tokens; |out| mean {out.float().abs().mean().item():.3f}")

    # the whole block: each token the next one of a request of its own, 1000 to 2000 tokens long
    lens = [1000 + 1000 * t // max(1, T - 1) for t in range(T)]
    layer = DecoderBlock(hidden=2048, q_heads=16, kv_heads=2, head_dim=256, rotary_dim=64, pages=32 * T, page_size=64,
                         max_tokens=T, max_seqs=T, experts=64, inter=768, topk=8, adapters=32, rank=16)
    for side in (layer.cache.k, layer.cache.v):
        side.copy_(torch.randn(side.shape, generator=gen, device="cuda"))
    batch = page_batch(lens, [1] * T, 64)
    with torch.cuda.stream(stream):
        stream.wait_stream(torch.cuda.default_stream())
        out, _ = layer.layer(residual, ids, *batch, max_new=1)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer.layer(residual, ids, *batch, max_new=1)
    eager, replay = timed(lambda: layer.layer(residual, ids, *batch, max_new=1)), timed(graph.replay)
    print(f"whole block over {sum(lens)} cached tokens: {eager:.1f} us a step, {replay:.1f} us replayed; |out| mean "
          f"{out.float().abs().mean().item():.3f}")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
