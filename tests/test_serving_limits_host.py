"""Limits and workspace sizes of the mixture-of-experts and adapter entries over whole ranges (no GPU)."""
from __future__ import annotations

import ctypes

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
