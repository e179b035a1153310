"""Limits and workspace sizes of the mixture-of-experts and adapter entries over whole ranges (no GPU)."""
from __future__ import annotations

import ctypes

import pytest

import fp8_block_scaled_a8w8_amd as g


def lora_bytes(M, N, K, L, R):
    n = ctypes.c_int64(-1)
    return g.lib().gemm_a8w8_blockscale_lora_workspace_bytes(M, N, K, L, R, ctypes.byref(n)), n.value


def test_adapters_rows_of_x_stay_within_32_bit_offsets():
    """256 rows of 2^22 bf16 values are 2 GiB: one row of them past what the kernels' offsets reach."""
    K = 1 << 22
    for M in (256, 257, 512, 5000):
        assert lora_bytes(M, 16, K, 2, 8)[0] == g.A8W8_ERR_SHAPE, M
        assert lora_bytes(M, 16, K - 128, 2, 8)[0] == g.A8W8_OK, M
    assert lora_bytes(255, 16, K, 2, 8)[0] == g.A8W8_OK


def moe_bytes(T, k, E, H, I, cus=0):
    n = ctypes.c_int64(-1)
    return g.lib().a8w8_moe_workspace_bytes(T, k, E, H, I, cus, ctypes.byref(n)), n.value


@pytest.mark.parametrize("N,K,R", [(14336, 5120, 32), (512, 8192, 8), (5120, 6144, 64), (1, 128, 256)])
def test_a_workspace_for_most_rows_serves_fewer(N, K, R):
    sizes = [lora_bytes(M, N, K, 16, R) for M in (*range(1, 700), 1024, 2048, 4096, 4097)]
    assert all(rc == g.A8W8_OK for rc, _ in sizes)
    assert sizes == sorted(sizes, key=lambda s: s[1])


@pytest.mark.parametrize("cus", [0, 32])
@pytest.mark.parametrize("k,E,H,I", [(1, 32, 1024, 768), (8, 128, 2048, 768), (4, 32, 5120, 1792), (8, 256, 2048, 512),
                                     (2, 8, 128, 2048), (2, 64, 8192, 128), (16, 1024, 256, 128)])
def test_a_workspace_for_most_tokens_serves_fewer(k, E, H, I, cus):
    sizes = [moe_bytes(T, k, E, H, I, cus) for T in (*range(1, 300), 5000)]
    assert all(rc == g.A8W8_OK for rc, _ in sizes)
    assert sizes == sorted(sizes, key=lambda s: s[1])
