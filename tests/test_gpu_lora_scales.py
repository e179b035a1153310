"""The projection with adapters on the library's own quantisation (needs an MI355X).

With ``scales="quotient"`` a row without an adapter is the projection that quantize_1x128 and the GEMM
give, to the bit.  With adapters the bars are those of the other rounding's tests: one bf16 rounding of an
fp32 sum (rel-L2 3e-3, 3.9e-3 below 4096 elements, per element parity_util's rule)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import fp8_block_scaled_a8w8_amd as g
import oracle

from gpu_util import DEV, say
from test_gpu_lora import assert_close, make, quantise

pytestmark = pytest.mark.gpu


def run(W, ws, X, A, B, sc, ids, packed=False, **kw):
    dW = torch.from_numpy(W).to(DEV)
    N = W.shape[0]
    if packed:
        dW = g.prepack_weights(dW)
    ad = g.LoraAdapters(A.to(DEV), B.to(DEV), sc.to(DEV))
    space = g.Workspace(g.lora_workspace_bytes(X.shape[0], N, X.shape[1], ad))
    y = g.gemm_a8w8_blockscale_lora(X.to(DEV), dW, torch.from_numpy(ws).to(DEV), ad, ids.to(DEV), space,
                                    packed_n=N if packed else None, **kw)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("M,N,K", [(5, 5120, 1024), (200, 640, 512), (600, 300, 256)])
def test_without_adapters_it_is_the_librarys_projection(M, N, K):
    say("lora scales, no adapter", M, N, K)
    W, ws, X, A, B, sc, ids = make(M, N, K, 16, 2, M, "none")
    q, s = g.quantize_1x128(X.to(DEV))
    # (the two roundings of a scale differ in some of these groups, so the comparison tells them apart)
    assert not np.array_equal(s.cpu().numpy(), quantise(X)[1])
    dW, dws = torch.from_numpy(W).to(DEV), torch.from_numpy(ws).to(DEV)
    for v in g.variants():
        if (v["kernel_name"] in ("rskinny", "ptile") and v["splits"] == 1 and v["bm"] <= 128
                and (M <= 16) == (v["kernel_name"] == "rskinny")):
            y = run(W, ws, X, A, B, sc, ids, variant=v["variant"], scales="quotient")
            base = g.gemm_a8w8_blockscale_run_variant(v["variant"], q, s, dW, dws)
            assert torch.equal(y.view(torch.int16), base.view(torch.int16)), v["name"]


@pytest.mark.parametrize("M,N,K,R,L,how,packed", [(1, 512, 1024, 8, 1, "one", False), (16, 333, 256, 64, 20, "random", True),
                                                  (133, 640, 768, 64, 24, "random", False), (700, 256, 384, 16, 7, "runs", True)])
def test_against_64_bits(M, N, K, R, L, how, packed):
    say("lora scales", M, N, K, R, L, how, packed)
    W, ws, X, A, B, sc, ids = case = make(M, N, K, R, L, 3 * M + N, how)
    q, s = oracle.quantize_1x128(X.float().numpy())
    ref = oracle.gemm(q, s, W, ws)
    x = X.double().numpy()
    for a in range(L):
        t = ids.numpy() == a
        ref[t] += float(sc[a]) * ((x[t] @ A[a].double().numpy().T) @ B[a].double().numpy().T)
    assert_close(run(*case, packed=packed, scales="quotient"), ref, (M, N, K, R, L, how, packed))


def test_refusals():
    case = make(4, 256, 256, 16, 2, 2, "random")
    with pytest.raises(ValueError):
        run(*case, scales="exact")
    split = next(v["variant"] for v in g.variants() if v["splits"] > 1)
    with pytest.raises(g.A8W8Error) as e:
        run(*case, scales="quotient", variant=split)
    assert e.value.status == g.A8W8_ERR_PLAN
    assert g.lib().gemm_a8w8_blockscale_lora_quantize_1x128(None, None) == g.A8W8_ERR_NULL
