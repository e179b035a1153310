"""Host-side parts of the decoder block (no GPU): where a batch's tokens lie in the cache."""
from __future__ import annotations

import pytest
import torch

from attention_util import Cache, attend64, attend_tolerance, values
from fp8_block_scaled_a8w8_amd.serving_block import page_batch


def place(batch, page, b, position):
    """The slot of a sequence's token by the page table."""
    return int(batch[2][b, position // page]) * page + position % page


@pytest.mark.parametrize("room", [80, [80, 40, 64]])
def test_grown_sequences_keep_their_pages(room):
    """Step after step, a sequence's earlier tokens lie where the steps before put them, and no two tokens share a slot."""
    page, lens, written = 16, [0, 0, 0], {}
    for new in ([15, 1, 30], [1, 16, 2], [17, 0, 1], [1, 1, 1]):
        lens = [n + m for n, m in zip(lens, new)]
        batch = page_batch(lens, new, page, "cpu", room=room)
        positions, slots, _, starts, kept = (t.tolist() for t in batch)
        assert kept == lens and starts[-1] == sum(new)
        for b in range(3):
            for p, s in zip(positions[starts[b]:starts[b + 1]], slots[starts[b]:starts[b + 1]]):
                written[b, p] = s
        for b in range(3):
            assert positions[starts[b]:starts[b + 1]] == list(range(lens[b] - new[b], lens[b]))
            for p in range(lens[b]):
                assert place(batch, page, b, p) == written[b, p], (b, p)
        assert len(set(written.values())) == len(written)


def test_pages_without_room_are_for_the_lengths():
    positions, slots, table, starts, lens = (t.tolist() for t in page_batch([40, 23, 0], [40, 1, 0], 16, "cpu"))
    assert table == [[0, 1, 2], [3, 4, -1], [-1, -1, -1]] and lens == [40, 23, 0] and starts == [0, 40, 41, 41]
    assert positions == [*range(40), 22] and slots == [*range(40), 3 * 16 + 22]
    assert tuple(page_batch([], [], 16, "cpu")[2].shape) == (0, 0)


@pytest.mark.parametrize("lens,new,room", [([3], [5], None), ([3], [-1], None), ([30], [1], 20), ([3, 4], [1], None),
                                           ([3, 4], [1, 1], [8])])
def test_what_does_not_fit_is_refused(lens, new, room):
    with pytest.raises(ValueError):
        page_batch(lens, new, 16, "cpu", room=room)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("D,G", [(64, 3), (128, 8), (256, 1)])
def test_the_bound_on_a_step_tells_wrong_results(dtype, D, G):
    """What the steps' test would let pass: no row may be zeros, half of itself, or without its newest key."""
    lens, news = [41, 1, 30, 57, 99], [1, 1, 30, 2, 37]
    starts = [0, 1, 2, 32, 34, 71]
    gen = torch.Generator().manual_seed(D)
    q, gate = (torch.randn(71, 2 * G, D, generator=gen).to(torch.bfloat16) for _ in range(2))
    c = Cache(lens, 2, D, 16, dtype, seed=1)
    k, v = values(c.k, c.ks), values(c.v, c.vs)
    want, mag, most = attend64(q, k, v, c.table, 16, starts, lens, D ** -0.5, gate=gate)
    late, _, _ = attend64(q, k, v, c.table, 16, starts, [n - 1 for n in lens], D ** -0.5, gate=gate)      # rows one key short
    for b, n in enumerate(news):
        r = slice(starts[b], starts[b + 1])
        tol = attend_tolerance(want[r], mag[r], most[r], D, n * G, lens[b])

        def passes(x):
            return ((x - want[r]).abs() <= tol).flatten(1).all(1)

        assert bool(passes(want[r].to(torch.bfloat16).double()).all())
        for what, x in (("zeros", 0 * want[r]), ("half", want[r] / 2), ("newest", late[r])):
            assert not passes(x).any(), (b, what)
