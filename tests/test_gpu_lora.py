"""Low-rank adapters beside a shared projection against the definition in 64 bits (needs an MI355X).

Tolerances (derived): the projection is the GEMM's (fp32 sums, bf16 once: rel-L2 bar 3e-3 and the
per-element rule of parity_util); the adapters' part is bf16 x bf16 in fp32 with inner values of 16
bits, an error of 2^-16 of that part, far below the one bf16 rounding of the sum.  Outputs of fewer
than 4096 elements: the worst case of one rounding, 2^-8 = 3.9e-3.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_block_scaled_a8w8_amd as g
import inputgen
import oracle

from gpu_util import DEV, say, variant_by_name, variant_names
from parity_util import compare

pytestmark = pytest.mark.gpu


def make(M, N, K, R, L, seed, how):
    gen = torch.Generator().manual_seed(seed)
    W, ws = inputgen.make_weights(N, K, seed=seed)
    X = torch.randn(M, K, generator=gen).to(torch.bfloat16)
    A = (torch.randn(L, R, K, generator=gen) / K ** 0.5).to(torch.bfloat16)
    B = (torch.randn(L, N, R, generator=gen) * 0.2).to(torch.bfloat16)
    sc = torch.rand(L, generator=gen) + 0.5
    if how == "random":
        ids = torch.randint(-1, L, (M,), generator=gen)
    elif how == "none":
        ids = torch.full((M,), -1)
    elif how == "one":
        ids = torch.full((M,), L - 1)
    else:                                     # runs of one adapter, cut at odd places
        ids = (torch.arange(M) // 37 * 5 + 1) % (L + 1) - 1
    return W, ws, X, A, B, sc, ids.to(torch.int32)


def quantise(X):
    """The operator's codes and scales: the e4m3fn rounding (torch's cast) of x / s with s = fp32(amax * fp32(1/448))."""
    x = X.float().numpy().reshape(X.shape[0], -1, 128)
    s = np.abs(x).max(axis=2) * (np.float32(1) / np.float32(448))
    assert s.dtype == np.float32
    q = np.divide(x, s[:, :, None], out=np.zeros_like(x), where=s[:, :, None] > 0)
    codes = torch.from_numpy(np.clip(q, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return np.ascontiguousarray(codes.reshape(X.shape)), s


def reference(W, ws, X, A, B, sc, ids):
    q, s = quantise(X)
    y = oracle.gemm(q, s, W, ws)
    x, ids = X.double().numpy(), ids.numpy()
    L = A.shape[0]
    for a in np.unique(ids[(ids >= 0) & (ids < L)]):
        t = ids == a
        y[t] += float(sc[a]) * ((x[t] @ A[a].double().numpy().T) @ B[a].double().numpy().T)
    return y


def run(W, ws, X, A, B, sc, ids, packed=False, variant=None, out=None):
    dW = torch.from_numpy(W).to(DEV)
    N = W.shape[0]
    if packed:
        dW = g.prepack_weights(dW)
    ad = g.LoraAdapters(A.to(DEV), B.to(DEV), sc.to(DEV))
    space = g.Workspace(g.lora_workspace_bytes(X.shape[0], N, X.shape[1], ad))
    y = g.gemm_a8w8_blockscale_lora(X.to(DEV), dW, torch.from_numpy(ws).to(DEV), ad, ids.to(DEV), space,
                                    packed_n=N if packed else None, variant=variant, out=out)
    torch.cuda.synchronize()
    return y


def assert_close(y, ref, what):
    st = compare(y, ref)
    bar = 3e-3 if ref.size >= 4096 else 3.9e-3
    assert st["finite"] and st["rel_l2"] <= bar and st["failing_count"] == 0, (what, st)


CASES = [  # M, N, K, R, L, ids, packed
    (1, 512, 1024, 8, 1, "one", False), (1, 5120, 256, 16, 3, "random", True), (2, 130, 128, 24, 2, "random", False),
    (3, 257, 384, 128, 5, "random", False), (7, 1, 256, 16, 2, "random", False), (15, 512, 1024, 64, 20, "random", True),
    (16, 2048, 640, 16, 16, "random", False), (16, 333, 256, 256, 3, "random", False), (16, 512, 512, 32, 4, "none", False),
    (17, 512, 512, 16, 4, "random", False), (40, 96, 256, 40, 8, "random", True), (65, 640, 384, 16, 70, "random", False),
    (128, 512, 256, 32, 3, "runs", False), (133, 1000, 512, 64, 9, "random", False), (300, 514, 384, 8, 6, "runs", True),
    (512, 1024, 256, 16, 5, "one", False), (1000, 768, 256, 16, 7, "runs", False), (33, 31, 256, 16, 4, "random", False),
    (4100, 300, 128, 16, 40, "random", False),
]


@pytest.mark.parametrize("M,N,K,R,L,how,packed", CASES)
def test_lora(M, N, K, R, L, how, packed):
    say("lora", M, N, K, R, L, how, packed)
    case = make(M, N, K, R, L, 3 * M + N, how)
    y = run(*case, packed=packed)
    again = run(*case, packed=packed)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    assert_close(y, reference(*case), (M, N, K, R, L, how, packed))


@pytest.mark.parametrize("M,N,K,R,L", [(133, 640, 768, 64, 24), (100, 130, 384, 64, 4), (257, 257, 1664, 40, 40), (300, 512, 256, 40, 3),
                                       (512, 384, 512, 16, 1), (512, 256, 128, 256, 33), (511, 128, 256, 8, 300),
                                       (700, 256, 384, 16, 60), (1100, 128, 256, 72, 5), (2100, 128, 128, 256, 7)])
@pytest.mark.parametrize("order", ["random", "runs", "tail"])
def test_lora_many_rows_of_an_adapter(M, N, K, R, L, order):
    """Decode batches whose rows share adapters: groups that fill up, cross the rows' chunks or begin late."""
    say("lora groups", M, N, K, R, L, order)
    W, ws, X, A, B, sc, ids = make(M, N, K, R, L, M + R, "random")
    if order == "runs":
        ids = torch.sort(ids).values
    elif order == "tail":                     # one adapter nearly everywhere; the others, or none, in the last rows
        ids[:M - 20] = 0
        ids[M - 20:M - 15] = -1
        ids[5], ids[M - 1] = 2 ** 31 - 1, L
    assert_close(run(W, ws, X, A, B, sc, ids), reference(W, ws, X, A, B, sc, ids), (M, N, K, R, L, order))


def test_tall_projection_for_one_token():
    """N = 34816 (more rows than the row-range instances take): the plan's other family."""
    case = make(2, 34816, 256, 16, 3, 5, "random")
    assert_close(run(*case), reference(*case), "tall")


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("name", [n for n in variant_names(kinds=("tile", "ptile", "rskinny"), splits=False)])
def test_every_instance(name, few):
    """Every instance with adapters: ragged tiles, mixed and missing adapters, both weight layouts, with the
    adapters' part formed beforehand (few rows) and in the epilogue."""
    v = variant_by_name(name)
    skinny = v["kernel_name"] == "rskinny"
    M = (13 if few else 2) if skinny else v["bm"] + 37 if few else 549
    N = 1000 if skinny else 2 * v["bn"] + 21
    say("lora instance", name, M, N)
    case = make(M, N, 640, 24, 5, 17, "random")
    if v["bm"] > 128:                         # 256-row tiles have no form with adapters
        with pytest.raises(g.A8W8Error) as e:
            run(*case, variant=v["variant"])
        assert e.value.status == g.A8W8_ERR_PLAN
        return
    ref = reference(*case)
    a = run(*case, variant=v["variant"])
    b = run(*case, variant=v["variant"], packed=True)
    assert_close(a, ref, name)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_without_adapters_it_is_the_projection():
    """No row has an adapter: bitwise the GEMM of the same instance on the quantised rows."""
    for M, N, K in ((5, 5120, 1024), (200, 640, 512)):
        W, ws, X, A, B, sc, ids = make(M, N, K, 16, 2, M, "none")
        q, s = (torch.from_numpy(t).to(DEV) for t in quantise(X))
        dW, dws = torch.from_numpy(W).to(DEV), torch.from_numpy(ws).to(DEV)
        for v in g.variants():
            if (v["kernel_name"] in ("rskinny", "ptile") and v["splits"] == 1 and v["bm"] <= 128
                    and (M <= 16) == (v["kernel_name"] == "rskinny")):
                y = run(W, ws, X, A, B, sc, ids, variant=v["variant"])
                base = g.gemm_a8w8_blockscale_run_variant(v["variant"], q, s, dW, dws)
                assert torch.equal(y.view(torch.int16), base.view(torch.int16)), v["name"]


def test_ids_out_of_range_and_rows_of_others_do_not_matter():
    """Ids outside the stack add nothing; an adapter of NaN reaches its own rows only."""
    M, N, K, R, L = 50, 512, 256, 16, 4
    W, ws, X, A, B, sc, ids = make(M, N, K, R, L, 8, "random")
    ids[3], ids[20], ids[49] = 2 ** 31 - 1, L, -2 ** 31
    assert_close(run(W, ws, X, A, B, sc, ids), reference(W, ws, X, A, B, sc, ids), "out of range")
    A2 = A.clone()
    A2[2] = float("nan")
    y, y2 = run(W, ws, X, A, B, sc, ids), run(W, ws, X, A2, B, sc, ids)
    mine = ids == 2
    assert bool(torch.isnan(y2[mine.to(DEV)]).all())
    assert torch.equal(y[~mine.to(DEV)].view(torch.int16), y2[~mine.to(DEV)].view(torch.int16))


def test_unaligned_out_other_stream_and_graph():
    M, N, K, R, L = 9, 512, 256, 16, 3
    W, ws, X, A, B, sc, ids = make(M, N, K, R, L, 2, "random")
    y = run(W, ws, X, A, B, sc, ids)
    buf = torch.full((M * N + 40,), 3.0, dtype=torch.bfloat16, device=DEV)
    run(W, ws, X, A, B, sc, ids, out=buf[17:17 + M * N].view(M, N))
    assert torch.equal(buf[17:17 + M * N].view(M, N), y)
    assert bool((buf[:17] == 3).all()) and bool((buf[17 + M * N:] == 3).all())
    dW, dws, dX, dids = (t.to(DEV) for t in (torch.from_numpy(W), torch.from_numpy(ws), X, ids))
    ad = g.LoraAdapters(A.to(DEV), B.to(DEV), sc.to(DEV))
    space = g.Workspace(g.lora_workspace_bytes(M, N, K, ad))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ys = g.gemm_a8w8_blockscale_lora(dX, dW, dws, ad, dids, space)
    s.synchronize()
    assert torch.equal(ys, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        yc = g.gemm_a8w8_blockscale_lora(dX, dW, dws, ad, dids, space)
    gen = torch.Generator().manual_seed(5)
    for i in range(3):
        dX.copy_(torch.randn(M, K, generator=gen).to(torch.bfloat16))
        dids.copy_(torch.randint(-1, L, (M,), generator=gen).to(torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        eager = g.gemm_a8w8_blockscale_lora(dX, dW, dws, ad, dids, space)
        torch.cuda.synchronize()
        assert torch.equal(yc.view(torch.int16), eager.view(torch.int16)), i


def test_refusals():
    M, N, K, R, L = 4, 256, 256, 16, 2
    W, ws, X, A, B, sc, ids = make(M, N, K, R, L, 2, "random")
    dW, dws, dX, dids, dA, dB, dsc = (t.to(DEV) for t in (torch.from_numpy(W), torch.from_numpy(ws), X, ids, A, B, sc))
    ad = g.LoraAdapters(dA, dB, dsc)
    space = g.Workspace(g.lora_workspace_bytes(M, N, K, ad))
    f = g.gemm_a8w8_blockscale_lora
    with pytest.raises(g.A8W8Error) as e:
        f(dX, dW, dws, ad, dids, g.Workspace(65536))
    assert e.value.status == g.A8W8_ERR_WORKSPACE
    split = next(v["variant"] for v in g.variants() if v["splits"] > 1)
    with pytest.raises(g.A8W8Error) as e:
        f(dX, dW, dws, ad, dids, space, variant=split)
    assert e.value.status == g.A8W8_ERR_PLAN
    with pytest.raises(ValueError):
        f(dX.float(), dW, dws, ad, dids, space)
    with pytest.raises(ValueError):
        f(dX, dW, dws, ad, dids.long(), space)
    with pytest.raises(ValueError):
        f(dX, dW, dws, ad, dids[:2], space)
    with pytest.raises(ValueError):
        f(dX, dW[:128], dws[:1], ad, dids, space)
    with pytest.raises(ValueError):
        g.LoraAdapters(dA[:, :12].contiguous(), dB[:, :, :12].contiguous(), dsc)
    with pytest.raises(ValueError):
        g.LoraAdapters(dA, dB, dsc[:1])
    with pytest.raises(TypeError):
        g.LoraAdapters(dA.float(), dB, dsc)
    assert f(dX[:0], dW, dws, ad, dids[:0], space).shape == (0, N)
