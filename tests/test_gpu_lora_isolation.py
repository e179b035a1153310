"""An adapter reaches the rows of its own requests only, whatever its values are (needs an MI355X).

Bitwise comparisons: the other rows' sums have the same terms in the same order."""
from __future__ import annotations

import pytest
import torch

import fp8_block_scaled_a8w8_amd as g

from gpu_util import say, variant_by_name, variant_names
from test_gpu_lora import make, run

pytestmark = pytest.mark.gpu

NAMES = [n for n in variant_names(kinds=("tile", "ptile", "rskinny"), splits=False) if variant_by_name(n)["bm"] <= 128]


def check(M, N, K, R, L, bad, variant=None):
    W, ws, X, A, B, sc, ids = make(M, N, K, R, L, M + R, "random")
    ids[0], ids[1], ids[M - 1] = 2, -1, 1           # rows of others and of none beside the bad adapter's in one tile
    B2 = B.clone()
    B2[2, ::3, R - 1] = bad
    B2[2, 1::3, 0] = -bad
    y = run(W, ws, X, A, B, sc, ids, variant=variant)
    y2 = run(W, ws, X, A, B2, sc, ids, variant=variant)
    mine = (ids == 2).to(y.device)
    assert not bool(torch.isfinite(y2[mine][:, ::3]).any()) and not bool(torch.isfinite(y2[mine][:, 1::3]).any())
    assert torch.equal(y[~mine].view(torch.int16), y2[~mine].view(torch.int16))
    assert torch.equal(y[mine][:, 2::3].contiguous().view(torch.int16), y2[mine][:, 2::3].contiguous().view(torch.int16))


# A decode batch (the waves share the adapters out), few rows on tiles (the products formed beforehand), and more.
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("M,N,K,R,L", [(3, 512, 256, 16, 3), (13, 1000, 384, 40, 5), (16, 512, 256, 8, 16), (50, 300, 256, 72, 4),
                                       (133, 640, 384, 64, 24), (600, 514, 256, 24, 6)])
def test_infinite_elements_of_b(M, N, K, R, L, bad):
    say("lora isolation", M, N, K, R, L, bad)
    check(M, N, K, R, L, bad)


@pytest.mark.parametrize("name", NAMES)
def test_every_instance_keeps_adapters_apart(name):
    v = variant_by_name(name)
    M, N = (11, 1000) if v["kernel_name"] == "rskinny" else (549, 2 * v["bn"] + 21)
    say("lora isolation", name, M, N)
    check(M, N, 256, 40, 5, float("nan"), variant=v["variant"])
