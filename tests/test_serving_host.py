"""Host-side checks of the routing, mixture-of-experts and adapter entries (no GPU): statuses of bad
arguments, reported before anything is enqueued, and the workspace sizes."""
from __future__ import annotations

import ctypes

import pytest

import fp8_block_scaled_a8w8_amd as g

P = 256                                     # an aligned, never dereferenced address


def route(logits=P, dtype=0, T=4, E=64, k=8, score=0, w=P, ids=P):
    return g.lib().a8w8_moe_route(logits, dtype, T, E, k, score, 1, 1.0, w, ids, None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=(1 << 30) + 1), dict(E=0), dict(E=1025, k=2), dict(k=0), dict(k=17),
                                dict(E=4, k=5), dict(dtype=2), dict(dtype=-1), dict(score=2)])
def test_route_bad_shapes(kw):
    assert route(**kw) == g.A8W8_ERR_SHAPE


def test_route_null_alignment_and_no_op():
    assert route(logits=None) == g.A8W8_ERR_NULL
    assert route(w=None) == g.A8W8_ERR_NULL and route(ids=None) == g.A8W8_ERR_NULL
    assert route(logits=P + 2) == g.A8W8_ERR_ALIGN
    assert route(logits=P + 1, dtype=1) == g.A8W8_ERR_ALIGN
    assert route(w=P + 2) == g.A8W8_ERR_ALIGN and route(ids=P + 1) == g.A8W8_ERR_ALIGN
    assert route(T=0, logits=None, w=None, ids=None) == g.A8W8_OK


def moe(**kw):
    f = dict(X=P, logits=P, W13=P, w13_scale=P, W2=P, w2_scale=P, Y=P, T=4, H=256, I=128, experts=8, topk=2,
             logits_dtype=0, score=0, renormalize=1, w_packed=0, scale=1.0, reserved=0, workspace=P, workspace_bytes=1 << 40)
    f.update(kw)
    return g.lib().a8w8_moe_layer(ctypes.byref(g.MoeDesc(**f)), None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(H=0), dict(H=130), dict(H=65536 + 128), dict(I=64), dict(I=0),
                                dict(I=65536 + 128), dict(H=65536, I=65536), dict(experts=0), dict(experts=1025),
                                dict(topk=0), dict(topk=9), dict(topk=17, experts=64), dict(w_packed=2),
                                dict(logits_dtype=3), dict(score=-1)])
def test_moe_bad_shapes(kw):
    assert moe(**kw) == g.A8W8_ERR_SHAPE


def test_moe_null_alignment_and_no_op():
    assert g.lib().a8w8_moe_layer(None, None) == g.A8W8_ERR_NULL
    for name in ("X", "logits", "W13", "w13_scale", "W2", "w2_scale", "Y"):
        assert moe(**{name: None}) == g.A8W8_ERR_NULL, name
        if name != "Y":
            assert moe(**{name: P + 2}) == g.A8W8_ERR_ALIGN, name
    assert moe(Y=P + 1) == g.A8W8_ERR_ALIGN and moe(workspace=P + 128) == g.A8W8_ERR_ALIGN
    assert moe(T=0, X=None, logits=None, Y=None, workspace=None, workspace_bytes=0) == g.A8W8_OK


def moe_bytes(T, k, E, H, I, cus=0):
    n = ctypes.c_int64(-1)
    rc = g.lib().a8w8_moe_workspace_bytes(T, k, E, H, I, cus, ctypes.byref(n))
    return rc, n.value


def test_moe_workspace_bytes():
    assert g.lib().a8w8_moe_workspace_bytes(1, 1, 8, 256, 128, 0, None) == g.A8W8_ERR_NULL
    assert moe_bytes(4, 2, 8, 250, 128)[0] == g.A8W8_ERR_SHAPE
    assert moe_bytes(0, 2, 8, 256, 128) == (g.A8W8_OK, 0)
    # counters, plan, and the hidden rows of every slot fit; more tokens than a chunk need no more
    rc, n = moe_bytes(256, 8, 128, 2048, 768)
    assert rc == g.A8W8_OK and n >= 65536 + 256 * 8 * 768 * 2
    assert moe_bytes(5000, 8, 128, 2048, 768) == (rc, n)
    assert moe_bytes(1, 8, 128, 2048, 768)[1] < n


def lora(**kw):
    f = dict(X=P, W=P, w_scale=P, A=P, B=P, scaling=P, ids=P, Y=P, M=4, N=256, K=256, adapters=2, rank=16, w_packed=0,
             variant=-1, workspace=P, workspace_bytes=1 << 40)
    f.update(kw)
    return g.lib().gemm_a8w8_blockscale_lora(ctypes.byref(g.LoraDesc(**f)), None)


@pytest.mark.parametrize("kw", [dict(M=-1), dict(N=0), dict(K=100), dict(K=0), dict(adapters=0), dict(adapters=(1 << 20) + 1),
                                dict(rank=0), dict(rank=12), dict(rank=264), dict(w_packed=-1), dict(N=(1 << 22) + 1),
                                dict(N=1 << 22, rank=256)])
def test_lora_bad_shapes(kw):
    assert lora(**kw) == g.A8W8_ERR_SHAPE


def test_lora_null_alignment_workspace_and_no_op():
    assert g.lib().gemm_a8w8_blockscale_lora(None, None) == g.A8W8_ERR_NULL
    for name in ("X", "W", "w_scale", "A", "B", "scaling", "ids", "Y"):
        assert lora(**{name: None}) == g.A8W8_ERR_NULL, name
        if name != "Y":
            assert lora(**{name: P + 2}) == g.A8W8_ERR_ALIGN, name
    assert lora(Y=P + 1) == g.A8W8_ERR_ALIGN and lora(workspace=P + 16) == g.A8W8_ERR_ALIGN
    assert lora(workspace=None) == g.A8W8_ERR_WORKSPACE and lora(workspace_bytes=65536) == g.A8W8_ERR_WORKSPACE
    assert lora(variant=g.gemm_a8w8_num_variants()) == g.A8W8_ERR_PLAN
    assert lora(M=0, X=None, ids=None, Y=None, workspace=None, workspace_bytes=0) == g.A8W8_OK


def test_lora_workspace_bytes():
    n = ctypes.c_int64(-1)
    f = g.lib().gemm_a8w8_blockscale_lora_workspace_bytes
    assert f(16, 512, 256, 2, 16, None) == g.A8W8_ERR_NULL
    assert f(16, 512, 256, 2, 10, ctypes.byref(n)) == g.A8W8_ERR_SHAPE
    assert f(0, 512, 256, 2, 16, ctypes.byref(n)) == g.A8W8_OK and n.value == 0
    assert f(2048, 512, 256, 2, 16, ctypes.byref(n)) == g.A8W8_OK
    assert n.value >= 65536 + 2048 * 256 + 2048 * 2 * 4 + 2048 * 2 * 16 * 2


def test_binding_refuses_host_tensors():
    import torch
    with pytest.raises(ValueError):
        g.moe_route(torch.zeros(2, 8), 2)
    with pytest.raises(ValueError):
        g.MoeExperts(torch.zeros(2, 256, 128, dtype=torch.uint8), torch.zeros(2, 2, 1), torch.zeros(2, 128, 128, dtype=torch.uint8),
                     torch.zeros(2, 1, 1))
    with pytest.raises(ValueError):
        g.LoraAdapters(torch.zeros(2, 16, 128, dtype=torch.bfloat16), torch.zeros(2, 64, 16, dtype=torch.bfloat16), torch.zeros(2))
