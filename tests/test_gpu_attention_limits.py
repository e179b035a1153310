"""Attention over a paged cache at the ends of its sizes, from several threads, and as a process's first call (needs an
MI355X)."""
from __future__ import annotations

import subprocess
import sys
import threading

import pytest
import torch

import fp8_block_scaled_a8w8_amd as g
from attention_util import Cache, attend64, attend_tolerance, values
from conftest import ROOT
from test_gpu_attention import call, check, heads, starts

from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_the_most_rows():
    """2^22 rows of one sequence whose tokens are the last few: those are as in a short call, all before them see nothing."""
    T, D, n = 1 << 22, 64, 200
    c = Cache([n], 1, D, 16, "bf16", seed=41)
    cache = c.to(DEV)
    q = torch.zeros(T, 1, D, dtype=torch.bfloat16, device=DEV)
    q[-n:] = heads(n, 1, D, 42).to(DEV)
    ws = g.Workspace(g.paged_attention_workspace_bytes(T, 1, 1, cache))
    out = g.paged_attention(q, cache, c.table.to(DEV), i32([0, T]), i32([n]), ws)
    check(out[-n:], q[-n:].cpu(), c, [0, n], [n], [n], D ** -0.5)
    assert not out[:-n].any()


@pytest.mark.parametrize("Hq,Hkv,D,n", [(1024, 1024, 64, 1), (1024, 1024, 64, 20), (1024, 16, 128, 2), (64, 1, 256, 1)])
def test_the_most_heads(Hq, Hkv, D, n):
    say("heads", Hq, Hkv, D, n)
    lens = [37, n]
    c = Cache(lens, Hkv, D, 16, "bf16", seed=43)
    q = heads(2 * n, Hq, D, 44)
    out = call(q.to(DEV), c, [0, n, 2 * n], lens)
    check(out, q, c, [0, n, 2 * n], lens, [n, n], D ** -0.5)


@pytest.mark.parametrize("n", [1, 40])
def test_the_largest_pages(n):
    """Pages of 65536 tokens, a sequence that ends in its second one, keys with a window and sinks far apart."""
    D, G, page, length = 64, 2, 65536, 65536 + 300
    gen = torch.Generator(device=DEV).manual_seed(45)
    k, v = (torch.randn(3, page, 1, D, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2))
    cache, q = g.KvCache(k, v), heads(n, G, D, 46)
    ws = g.Workspace(g.paged_attention_workspace_bytes(n, 1, G, cache))
    table = torch.tensor([[2, 0]], dtype=torch.int32)
    for window, sinks in ((0, 0), (500, 70)):
        out = g.paged_attention(q.to(DEV), cache, table.to(DEV), i32([0, n]), i32([length]), ws, window=window, sinks=sinks)
        want, mag, most = attend64(q, values(k, None), values(v, None), table, page, [0, n], [length], D ** -0.5, window, sinks)
        tol = attend_tolerance(want, mag, most, D, n * G, length)
        assert bool(((out.double().cpu() - want).abs() <= tol).all()), window


@pytest.mark.parametrize("news", [[1, 1, 1], [30, 1, 25]])
def test_sequences_share_pages(news):
    """A prefix whose pages several sequences name, one page named twice by one sequence."""
    D, G, page = 128, 4, 16
    lens = [100, 90, 64]
    c = Cache([100, 0, 0], 1, D, page, "bf16", seed=47)
    c.table = c.table[:1].repeat(3, 1)
    c.table[1, 5] = c.table[0, 1]
    c.table[2, 2] = c.table[2, 1]
    q = heads(sum(news), G, D, 48)
    out = call(q.to(DEV), c, starts(news), lens)
    check(out, q, c, starts(news), lens, news, D ** -0.5)


def test_two_threads_at_once():
    """Calls of two threads, each with its stream and workspace."""
    D, G, lens, news = 128, 4, [3000, 500], [1, 40]
    c = Cache(lens, 2, D, 16, "bf16", seed=49)
    cache, table, qs, ls = c.to(DEV), c.table.to(DEV), i32(starts(news)), i32(lens)
    q = heads(41, 2 * G, D, 50).to(DEV)
    make = lambda: g.Workspace(g.paged_attention_workspace_bytes(41, 2, 2 * G, cache))  # noqa: E731
    want = g.paged_attention(q, cache, table, qs, ls, make())
    torch.cuda.synchronize()
    outs, errors = [[], []], []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                ws = make()
                for _ in range(30):
                    outs[i].append(g.paged_attention(q, cache, table, qs, ls, ws))
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and all(torch.equal(o, want) for o in outs[0] + outs[1]) and len(outs[0]) == len(outs[1]) == 30


FIRST = """
import torch, sys
import fp8_block_scaled_a8w8_amd as g
dev = "cuda:0"
gen = torch.Generator(device=dev).manual_seed(1)
k, v = (torch.randn(8, 16, 1, 64, generator=gen, device=dev).to(torch.bfloat16) for _ in range(2))
q = torch.randn(40, 2, 64, generator=gen, device=dev).to(torch.bfloat16)
cache, rope = g.KvCache(k, v), g.Rope(torch.ones(16, device=dev))
ws = g.Workspace(g.paged_attention_workspace_bytes(40, 2, 2, cache))
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
table, starts, lens, pos = i32([[0, 1, 2, 3], [4, 5, 6, 7]]), i32([0, 39, 40]), i32([60, 50]), i32(list(range(40)))
torch.cuda.synchronize()
def step():
    t, _ = g.qk_norm_rope(q, q[:, :1], rope, pos)
    return g.paged_attention(t, cache, table, starts, lens, ws)
graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(graph, stream=stream):
    out = step()
for i in range(3):
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    again = step()
    torch.cuda.synchronize()
    assert torch.equal(out, again) and bool(out.any()), i
    q.mul_(0.5)
print("captured first")
"""


def test_the_first_call_of_a_process_is_captured():
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]
