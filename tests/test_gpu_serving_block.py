"""The serving block: the projection with adapters, the routing and the experts run together (needs an MI355X).

The block is checked against the same steps in 64 bits from its own intermediate x and logits (both are
outputs that a step fixes: x is bf16, and routing is compared on the logits it used).  Tolerances: x and the
layer are each rounded to bf16 (twice along the way, 2^-9 at most each): rel-L2 below 3 * 2^-9 = 5.9e-3."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_block_scaled_a8w8_amd as g
from fp8_block_scaled_a8w8_amd import serving_block
from fp8_block_scaled_a8w8_amd.serving_block import ServingBlock

from gpu_util import DEV, say
from test_gpu_lora import quantise

pytestmark = pytest.mark.gpu


def rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


def dequant(codes, s):
    return codes.double() * s.double().repeat_interleave(128, -2).repeat_interleave(128, -1)


@pytest.mark.parametrize("T", [1, 7, 40])
def test_step_against_64_bits(T):
    say("serving block", T)
    b = ServingBlock(hidden=512, width=768, experts=12, inter=256, topk=3, adapters=5, rank=16, max_tokens=64)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T)
    att = torch.randn(T, 768, generator=gen, device=DEV).to(torch.bfloat16)
    res = torch.randn(T, 512, generator=gen, device=DEV).to(torch.bfloat16)
    ids = torch.randint(-1, 5, (T,), generator=gen, device=DEV).to(torch.int32)
    out, logits = b.step(att, res, ids)
    torch.cuda.synchronize()
    # the projection
    q, s = quantise(att.cpu())
    xq = torch.from_numpy(q).view(torch.float8_e4m3fn).double() * torch.from_numpy(s).double().repeat_interleave(128, 1)
    y = xq @ dequant(b.W, b.w_scale).cpu().t()
    for t in range(T):
        a = int(ids[t])
        if a >= 0:
            y[t] += b.adapters.B[a].double().cpu() @ (b.adapters.A[a].double().cpu() @ att[t].double().cpu())
    x = (res.double().cpu() + y.to(torch.bfloat16).double()).to(torch.bfloat16)
    # the experts, from the step's own logits (x is the same up to roundings of single values)
    w, e = g.moe_route(logits, 3)
    m = torch.zeros(T, 512, dtype=torch.float64)
    for t in range(T):
        for j in range(3):
            gu = dequant(b.experts.W13[e[t, j]], b.experts.w13_scale[e[t, j]]).cpu() @ x[t].double()
            h = gu[:256] * torch.sigmoid(gu[:256]) * gu[256:]
            m[t] += float(w[t, j]) * (dequant(b.experts.W2[e[t, j]], b.experts.w2_scale[e[t, j]]).cpu() @ h)
    assert rel(out.double().cpu().numpy(), (x.double() + m).numpy()) <= 3 * 2.0 ** -9
    load = b.load(logits)
    assert int(load.sum()) == 3 * T and len(load) == 12


def test_replayed_graph_equals_eager():
    T = 9
    b = ServingBlock(hidden=512, width=768, experts=12, inter=256, topk=3, adapters=5, rank=16, max_tokens=16)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    att = torch.randn(T, 768, generator=gen, device=DEV).to(torch.bfloat16)
    res = torch.randn(T, 512, generator=gen, device=DEV).to(torch.bfloat16)
    ids = torch.randint(-1, 5, (T,), generator=gen, device=DEV).to(torch.int32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.step(att, res, ids)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, _ = b.step(att, res, ids)
    for i in range(3):
        att.copy_(torch.randn(T, 768, generator=gen, device=DEV).to(torch.bfloat16))
        ids.copy_(torch.randint(-1, 5, (T,), generator=gen, device=DEV).to(torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        eager, _ = b.step(att, res, ids)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager.view(torch.int16)), i


def test_command_runs(capsys):
    assert serving_block.main(["--tokens", "5", "--steps", "3"]) == 0
    assert "us a step" in capsys.readouterr().out
