"""Expert routing and the mixture-of-experts layer against the definitions in 64 bits (needs an MI355X).

Tolerances (derived, not fitted):

* ids are whole numbers and must be equal;
* routing weights: fp32 exponentials (a few ulp each; the argument's rounding adds at most
  |x| 2^-24, |x| < 20 here, wherever the weight counts), a sum of at most 1024 of them and one
  division: relative error below 64 * 2^-24 = 4e-6 of the row's largest weight;
* the layer: Y is rounded to bf16 once and h once (each at most 2^-9 relative, about 1.7e-3 in
  2-norm over many elements, independent: 2.4e-3 together); everything else is fp32.  rel-L2 bar
  3e-3 as for the GEMM, per element 2e-2 of the row set's rms or a bf16 neighbour (parity_util).
  With few elements the 2-norms of roundings scatter around their means but stay below the worst
  case 2^-8 = 3.9e-3, the bar for outputs of fewer than 4096 elements.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_block_scaled_a8w8_amd as g
import inputgen

from gpu_util import DEV, say
from parity_util import compare

pytestmark = pytest.mark.gpu

F32_MAX = float(np.finfo(np.float32).max)


def route_ref(logits, k, score, renorm, scale=1.0):
    x = np.asarray(logits, dtype=np.float64).copy()
    x[np.isnan(x)] = -np.inf
    x = np.minimum(x, F32_MAX)
    T, E = x.shape
    ids = np.full((T, k), -1, dtype=np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        order = sorted((e for e in range(E) if x[t, e] > -np.inf), key=lambda e: (-x[t, e], e))[:k]
        ids[t, :len(order)] = order
        if not order:
            continue
        v = x[t, order]
        if score == "softmax":
            p = np.exp(v - v[0])
            total = p.sum() if renorm else np.exp(x[t][x[t] > -np.inf] - v[0]).sum()
        else:
            log_p = np.where(v > 0, -np.log1p(np.exp(-np.abs(v))), v - np.log1p(np.exp(-np.abs(v))))
            p = np.exp(log_p - log_p[0]) if renorm else np.exp(log_p)
            total = p.sum() if renorm else 1.0
        if total > 0:
            w[t, :len(order)] = p / total * scale
    return w, ids


def check_route(logits, k, score="softmax", renorm=True, scale=1.0):
    w, ids = g.moe_route(logits, k, score=score, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    rw, rids = route_ref(logits.float().cpu().numpy(), k, score, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), rids)
    got = w.cpu().numpy().astype(np.float64)
    bound = 4e-6 * np.maximum(np.abs(rw).max(axis=1, keepdims=True), 1e-30)
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - rw) <= bound), np.abs(got - rw).max()
    return w, ids


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (3, 17, 5), (5, 63, 1), (7, 64, 16), (9, 65, 16), (33, 128, 8),
                                   (6, 160, 6), (61, 256, 8), (4, 257, 3), (2, 511, 16), (2, 513, 9), (3, 1024, 16),
                                   (2053, 60, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route(T, E, k, dtype):
    x = (torch.randn(T, E, generator=torch.Generator().manual_seed(T + E)) * 2).to(dtype).to(DEV)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            say("route", T, E, k, dtype, score, renorm)
            check_route(x, k, score, renorm, 1.0 if renorm else 2.5)


@pytest.mark.parametrize("E,k", [(1, 1), (17, 5), (60, 4), (100, 8), (129, 1), (256, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_many_tokens(E, k, dtype):
    # Random rows; rows of few distinct values (ties among more logits than any list holds); masked ones.
    T = 4099
    gen = torch.Generator().manual_seed(E)
    x = torch.randn(T, E, generator=gen) * 2
    x[1000:1100] = x[1000:1100].round()
    x[1100:1150] = (x[1100:1150] * 0.25).round()
    x[2000:2020] = 0.0
    x[2001] = -0.0
    x[2030:2034] = float("-inf")
    x[2040:2060, 1:] = float("-inf")
    x[2060:2080, E // 2:] = float("nan")
    x[2080:2090, ::2] = float("inf")
    x[2090:2100, ::3] = -F32_MAX
    x[4098, : E // 2] = float("-inf")
    x = x.to(dtype).to(DEV)
    for score, renorm in (("softmax", False), ("softmax", True), ("sigmoid", True)):
        say("route", T, E, k, dtype, score, renorm)
        check_route(x, k, score, renorm, 1.5)


def test_route_ties_masks_and_extremes():
    E, k = 70, 4
    inf, low = float("inf"), -F32_MAX
    rows = [torch.zeros(E),                                             # all equal: 0, 1, 2, 3
            torch.full((E,), -inf),                                     # nothing left
            torch.full((E,), low),                                      # the type's lowest value is no mask
            torch.full((E,), float("nan")),
            torch.cat([torch.full((E - 2,), -inf), torch.tensor([1.0, 2.0])]),   # fewer than k
            torch.cat([torch.tensor([inf, inf]), torch.randn(E - 2)]),
            torch.cat([torch.tensor([float("nan"), F32_MAX, low, -inf]), torch.randn(E - 4)]),
            torch.cat([torch.full((E - 1,), -200.0), torch.tensor([-201.0])]),   # sigmoids underflow
            torch.arange(E).float().flip(0), (torch.arange(E) // 9).float()]
    x = torch.stack(rows).to(DEV)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check_route(x, k, score, renorm)
    check_route(x.to(torch.bfloat16), k)


def test_route_outputs_given_stream_and_determinism():
    x = torch.randn(37, 96, generator=torch.Generator().manual_seed(3)).to(DEV)
    w, ids = check_route(x, 6)
    wo = torch.full((37, 6), 7.0, device=DEV)
    io = torch.full((37, 6), 7, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g.moe_route(x, 6, weights_out=wo, ids_out=io, stream=s)
    s.synchronize()
    assert torch.equal(wo, w) and torch.equal(io, ids)


def test_route_refusals():
    x = torch.zeros(4, 8, device=DEV)
    for bad in (0, 9, 17):
        with pytest.raises(g.A8W8Error):
            g.moe_route(x, bad)
    with pytest.raises(g.A8W8Error):
        g.moe_route(torch.zeros(2, 1025, device=DEV), 2)
    with pytest.raises(ValueError):
        g.moe_route(x, 2, score="tanh")
    with pytest.raises(ValueError):
        g.moe_route(x.half(), 2)
    with pytest.raises(ValueError):
        g.moe_route(x.t(), 2)
    with pytest.raises(ValueError):
        g.moe_route(x, 2, ids_out=torch.zeros(4, 2, device=DEV))
    assert g.moe_route(torch.zeros(0, 8, device=DEV), 2)[0].shape == (0, 2)


# ---------------------------------------------------------------------------

def experts_inputs(E, H, I, seed):
    """Expert weights (codes and block scales, host) from the seeded GEMM weight generator."""
    w13, s13, w2, s2 = [], [], [], []
    for e in range(E):
        a, b = inputgen.make_weights(2 * I, H, seed=seed + 2 * e)
        c, d = inputgen.make_weights(H, I, seed=seed + 2 * e + 1)
        w13.append(a), s13.append(b), w2.append(c), s2.append(d)
    return [np.stack(v) for v in (w13, s13, w2, s2)]


def dequant(codes, s):
    w = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    N, K = w.shape
    return w * np.repeat(np.repeat(s.astype(np.float64), 128, 0)[:N], 128, 1)[:, :K]


def layer_ref(X, logits, weights, k, score="softmax", renorm=True, scale=1.0):
    w13, s13, w2, s2 = weights
    w, ids = route_ref(logits, k, score, renorm, scale)
    I = w2.shape[2]
    y = np.zeros((X.shape[0], X.shape[1]))
    for e in np.unique(ids[ids >= 0]):
        t, j = np.nonzero(ids == e)
        gu = X[t] @ dequant(w13[e], s13[e]).T
        h = gu[:, :I] / (1.0 + np.exp(-gu[:, :I])) * gu[:, I:]
        y[t] += w[t, j][:, None] * (h @ dequant(w2[e], s2[e]).T)
    return y


def make_handle(weights, packed):
    dev = [torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for v in weights]
    return g.MoeExperts.pack(*dev) if packed else g.MoeExperts(*dev)


def assert_layer(y, ref, what):
    st = compare(y, ref)
    bar = 3e-3 if ref.size >= 4096 else 3.9e-3
    assert st["finite"] and st["rel_l2"] <= bar and st["failing_count"] == 0, (what, st)


CASES = [  # T, E, k, H, I, packed
    (1, 8, 2, 128, 128, False), (1, 4, 4, 640, 256, True), (2, 8, 8, 256, 384, False), (5, 16, 3, 1152, 128, False),
    (16, 8, 2, 512, 256, True), (17, 8, 2, 512, 256, False), (33, 4, 4, 384, 384, False), (64, 8, 1, 256, 128, True),
    (100, 3, 3, 256, 640, False), (255, 16, 4, 256, 256, False), (256, 5, 2, 128, 256, True), (257, 8, 2, 256, 128, False),
    (600, 6, 2, 256, 128, False), (7, 1, 1, 256, 128, False), (40, 130, 8, 128, 128, False),
]


@pytest.mark.parametrize("T,E,k,H,I,packed", CASES)
def test_layer(T, E, k, H, I, packed):
    say("moe layer", T, E, k, H, I, packed)
    weights = experts_inputs(E, H, I, seed=11)
    gen = torch.Generator().manual_seed(T * 7 + E)
    X = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen)
    ex = make_handle(weights, packed)
    ws = g.Workspace(g.moe_workspace_bytes(T, k, ex))
    y = g.moe_layer_a16w8_blockscale(X.to(DEV), logits.to(DEV), ex, k, ws)
    again = g.moe_layer_a16w8_blockscale(X.to(DEV), logits.to(DEV), ex, k, ws)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    assert_layer(y, layer_ref(X.double().numpy(), logits.numpy(), weights, k), (T, E, k, H, I, packed))


@pytest.mark.parametrize("packed", [False, True])
def test_layer_scores_masks_padding_and_skew(packed):
    T, E, k, H, I = 48, 12, 4, 384, 256
    weights = experts_inputs(E, H, I, seed=5)
    gen = torch.Generator().manual_seed(1)
    X = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen)
    logits[:, 3] += 50.0                                    # every live token reaches expert 3
    logits[5:9] = float("-inf")                             # padding rows, with values no one may read
    X[5:9] = float("nan")
    logits[10, 2:] = float("-inf")                          # two experts left
    logits[11, :] = -F32_MAX
    ex = make_handle(weights, packed)
    ws = g.Workspace(g.moe_workspace_bytes(T, k, ex))
    live = X.clone()
    live[5:9] = 0
    for score, renorm, scale, dtype in (("softmax", True, 1.0, torch.float32), ("softmax", False, 2.5, torch.bfloat16),
                                        ("sigmoid", True, 1.0, torch.bfloat16), ("sigmoid", False, 0.5, torch.float32)):
        lg = logits.to(dtype)
        y = g.moe_layer_a16w8_blockscale(X.to(DEV), lg.to(DEV), ex, k, ws, score=score, renormalize=renorm, scale=scale)
        ref = layer_ref(live.double().numpy(), lg.float().numpy(), weights, k, score, renorm, scale)
        assert torch.count_nonzero(y[5:9]).item() == 0
        assert_layer(y, ref, (score, renorm, scale, dtype))
    # nothing routed at all
    y = g.moe_layer_a16w8_blockscale(X.to(DEV), torch.full((T, E), float("-inf"), device=DEV), ex, k, ws)
    assert torch.count_nonzero(y).item() == 0


def test_packed_equals_row_major_and_padding_does_not_matter():
    """The two weight layouts give the same bits, and a token's row does not depend on padding rows."""
    T, E, k, H, I = 12, 9, 3, 640, 384
    weights = experts_inputs(E, H, I, seed=23)
    X = torch.randn(T, H, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(4)).to(DEV)
    row, pk = make_handle(weights, False), make_handle(weights, True)
    ws = g.Workspace(g.moe_workspace_bytes(T, k, row))
    a = g.moe_layer_a16w8_blockscale(X, logits, row, k, ws)
    b = g.moe_layer_a16w8_blockscale(X, logits, pk, k, ws)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_layer_unaligned_out_guard_band_and_graph():
    """An out tensor at an odd element offset, its surroundings untouched; a captured call replays."""
    T, E, k, H, I = 5, 8, 2, 256, 128
    weights = experts_inputs(E, H, I, seed=31)
    ex = make_handle(weights, False)
    ws = g.Workspace(g.moe_workspace_bytes(T, k, ex))
    gen = torch.Generator().manual_seed(9)
    X = torch.randn(T, H, generator=gen).to(torch.bfloat16).to(DEV)
    logits = torch.randn(T, E, generator=gen).to(DEV)
    y = g.moe_layer_a16w8_blockscale(X, logits, ex, k, ws)
    buf = torch.full((T * H + 64,), 3.0, dtype=torch.bfloat16, device=DEV)
    out = buf[33:33 + T * H].view(T, H)
    g.moe_layer_a16w8_blockscale(X, logits, ex, k, ws, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, y) and bool((buf[:33] == 3).all()) and bool((buf[33 + T * H:] == 3).all())
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g.moe_layer_a16w8_blockscale(X, logits, ex, k, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        yc = g.moe_layer_a16w8_blockscale(X, logits, ex, k, ws)
    for i in range(3):
        X.copy_(torch.randn(T, H, generator=gen).to(torch.bfloat16))
        logits.copy_(torch.randn(T, E, generator=gen))
        graph.replay()
        torch.cuda.synchronize()
        eager = g.moe_layer_a16w8_blockscale(X, logits, ex, k, ws)
        torch.cuda.synchronize()
        assert torch.equal(yc.view(torch.int16), eager.view(torch.int16)), i


def test_layer_refusals():
    E, H, I, T = 4, 256, 128, 3
    weights = experts_inputs(E, H, I, seed=1)
    dev = [torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for v in weights]
    ex = g.MoeExperts(*dev)
    X = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    lg = torch.zeros(T, E, device=DEV)
    ws = g.Workspace(g.moe_workspace_bytes(T, 2, ex))
    with pytest.raises(g.A8W8Error) as e:
        g.moe_layer_a16w8_blockscale(X, lg, ex, 2, g.Workspace(65536))
    assert e.value.status == g.A8W8_ERR_WORKSPACE
    for bad in (0, 5):
        with pytest.raises(g.A8W8Error):
            g.moe_layer_a16w8_blockscale(X, lg, ex, bad, ws)
    with pytest.raises(ValueError):
        g.moe_layer_a16w8_blockscale(X[:, :128].contiguous(), lg, ex, 2, ws)
    with pytest.raises(ValueError):
        g.moe_layer_a16w8_blockscale(X.float(), lg, ex, 2, ws)
    with pytest.raises(ValueError):
        g.moe_layer_a16w8_blockscale(X, lg[:, :2], ex, 2, ws)
    with pytest.raises(ValueError):
        g.MoeExperts(dev[0], dev[1], dev[2][:, :, :64].contiguous(), dev[3])
    with pytest.raises(ValueError):
        g.MoeExperts(dev[0], dev[1][:, :1].contiguous(), dev[2], dev[3])
    with pytest.raises(TypeError):
        g.MoeExperts(dev[0].float(), *dev[1:])
    assert g.moe_layer_a16w8_blockscale(X[:0], lg[:0], ex, 2, ws).shape == (0, H)


@pytest.mark.parametrize("packed", [False, True])
def test_layer_many_slots_on_many_experts(packed):
    # Enough workgroups of 128 weight rows for every CU, one and two passes of 32 slots, and tokens
    # that reach fewer experts than they may, or none.
    T, E, k, H, I = 253, 110, 10, 256, 128
    say("moe layer", T, E, k, H, I, packed)
    weights = experts_inputs(E, H, I, seed=3)
    gen = torch.Generator().manual_seed(8)
    X = torch.randn(T, H, generator=gen).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=gen)
    logits[:70, 109] += 50.0
    logits[100:103] = float("-inf")
    logits[200, 3:] = float("-inf")
    ex = make_handle(weights, packed)
    ws = g.Workspace(g.moe_workspace_bytes(T, k, ex))
    y = g.moe_layer_a16w8_blockscale(X.to(DEV), logits.to(DEV), ex, k, ws)
    torch.cuda.synchronize()
    assert torch.equal(y[100:103], torch.zeros_like(y[100:103]))
    assert_layer(y, layer_ref(X.double().numpy(), logits.numpy(), weights, k), (T, E, k, H, I, packed))
