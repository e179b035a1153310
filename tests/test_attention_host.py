"""Host-side checks of the rotation and attention entries (no GPU): statuses of bad arguments, reported before
anything is enqueued, the workspace size, and what the binding refuses."""
from __future__ import annotations

import ctypes

import pytest
import torch

import fp8_block_scaled_a8w8_amd as g

P = 256                                     # an aligned, never dereferenced address


def rope(**kw):
    f = dict(q=P, k=P, v=P, q_row=1024, q_head=128, k_row=256, k_head=128, v_row=256, v_head=128, q_weight=P, k_weight=P,
             positions=P, inv_freq=P, axis_of=None, slots=P, q_out=P, k_out=None, k_cache=P, v_cache=P, k_scale=None,
             v_scale=None, T=4, cache_slots=64, q_heads=8, kv_heads=2, head_dim=128, rotary_dim=64, axes=1, layout=0,
             cache_dtype=0, eps=1e-6)
    f.update(kw)
    return g.lib().a8w8_qk_norm_rope(ctypes.byref(g.RopeDesc(**f)), None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=(1 << 30) + 1), dict(q_heads=0), dict(kv_heads=0), dict(q_heads=1025),
                                dict(kv_heads=1025), dict(head_dim=96), dict(head_dim=0), dict(rotary_dim=144), dict(rotary_dim=24),
                                dict(rotary_dim=-16), dict(axes=0), dict(axes=17), dict(layout=2), dict(layout=-1),
                                dict(cache_dtype=2), dict(eps=-1.0), dict(eps=float("nan")), dict(cache_slots=0),
                                dict(cache_slots=1 << 31), dict(q_row=1020), dict(q_head=-128), dict(k_head=4), dict(v_row=12)])
def test_rope_bad_shapes(kw):
    assert rope(**kw) == g.A8W8_ERR_SHAPE


def test_rope_null_alignment_and_no_op():
    assert g.lib().a8w8_qk_norm_rope(None, None) == g.A8W8_ERR_NULL
    for name in ("q", "k", "v", "positions", "inv_freq", "slots", "q_out", "k_cache", "v_cache"):
        assert rope(**{name: None}) == g.A8W8_ERR_NULL, name
    assert rope(k_out=P) == g.A8W8_ERR_NULL                              # cache and k_out at once
    assert rope(k_cache=None, v_cache=None) == g.A8W8_ERR_NULL           # neither
    for name in ("q", "k", "v", "q_out", "k_cache", "v_cache"):
        assert rope(**{name: P + 8}) == g.A8W8_ERR_ALIGN, name
    for name in ("q_weight", "k_weight", "positions", "inv_freq", "axis_of", "slots", "k_scale", "v_scale"):
        assert rope(**{name: P + 2}) == g.A8W8_ERR_ALIGN, name
    assert rope(cache_dtype=1, k_cache=P + 4) == g.A8W8_ERR_ALIGN
    assert rope(T=0, q=None, k=None, v=None, q_out=None) == g.A8W8_OK


def attention(**kw):
    f = dict(q=P, gate=None, q_row=1024, q_head=128, gate_row=0, gate_head=0, k_cache=P, v_cache=P, k_scale=None, v_scale=None,
             page_table=P, q_start=P, kv_lens=P, out=P, T=4, B=2, pages=8, table_pages=4, page_size=16, q_heads=8, kv_heads=2,
             head_dim=128, cache_dtype=0, window=0, sinks=0, max_new=0, scale=0.1, reserved=0, workspace=P,
             workspace_bytes=1 << 40)
    f.update(kw)
    return g.lib().a8w8_paged_attention(ctypes.byref(g.AttentionDesc(**f)), None)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(T=(1 << 22) + 1), dict(B=-1), dict(B=2049), dict(q_heads=0), dict(q_heads=7),
                                dict(kv_heads=0), dict(q_heads=1032), dict(q_heads=130, kv_heads=2), dict(head_dim=80),
                                dict(cache_dtype=-1), dict(pages=0), dict(table_pages=0), dict(page_size=0), dict(page_size=48),
                                dict(page_size=1 << 17), dict(pages=(1 << 27) + 1), dict(table_pages=(1 << 26) + 1),
                                dict(window=-1), dict(sinks=-1), dict(max_new=-1), dict(scale=float("nan")), dict(q_row=4),
                                dict(q_head=-8), dict(gate=P, gate_row=12), dict(gate=P, gate_row=8, gate_head=2)])
def test_attention_bad_shapes(kw):
    assert attention(**kw) == g.A8W8_ERR_SHAPE


def test_attention_null_alignment_workspace_and_no_op():
    assert g.lib().a8w8_paged_attention(None, None) == g.A8W8_ERR_NULL
    for name in ("q", "k_cache", "v_cache", "page_table", "q_start", "kv_lens", "out"):
        assert attention(**{name: None}) == g.A8W8_ERR_NULL, name
    for name in ("q", "gate", "k_cache", "v_cache", "out"):
        assert attention(**{name: P + 8}) == g.A8W8_ERR_ALIGN, name
    for name in ("k_scale", "v_scale", "page_table", "q_start", "kv_lens"):
        assert attention(**{name: P + 2}) == g.A8W8_ERR_ALIGN, name
    assert attention(workspace=P + 128) == g.A8W8_ERR_ALIGN
    assert attention(T=0, q=None, out=None, workspace=None) == g.A8W8_OK
    assert attention(B=0, page_table=None, kv_lens=None, workspace=None) == g.A8W8_OK


def workspace_bytes(*a):
    n = ctypes.c_int64(-1)
    return g.lib().a8w8_paged_attention_workspace_bytes(*a, ctypes.byref(n)), n.value


def test_attention_workspace_bytes():
    assert g.lib().a8w8_paged_attention_workspace_bytes(1, 1, 8, 2, 128, 0, 0, None) == g.A8W8_ERR_NULL
    assert workspace_bytes(4, 2, 8, 2, 100, 0, 0)[0] == g.A8W8_ERR_SHAPE
    assert workspace_bytes(0, 2, 8, 2, 128, 0, 0) == (g.A8W8_OK, 0)
    rc, one = workspace_bytes(1, 1, 8, 2, 128, 0, 0)
    assert rc == g.A8W8_OK and one >= 65536
    # more rows or sequences never need less (a workspace for the largest step serves every smaller one)
    for T in (1, 2, 7, 64, 300, 5000, 100000):
        for B in (1, 5, 64, 2048):
            rc, n = workspace_bytes(T, B, 32, 8, 128, 0, 0)
            assert rc == g.A8W8_OK and n >= 65536
            for t, b in ((max(1, T // 2), B), (T, max(1, B // 2))):
                assert workspace_bytes(t, b, 32, 8, 128, 0, 0)[1] <= n


def test_binding_refuses():
    cpu = torch.zeros(2, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        g.KvCache(cpu, cpu)                                              # host tensors
    with pytest.raises(TypeError):
        g.KvCache(cpu.float(), cpu.float())
    with pytest.raises(ValueError):
        g.KvCache(cpu, cpu[:1])
    with pytest.raises(ValueError):
        g.KvCache(cpu[:, :12], cpu[:, :12])                              # page size not a power of two
    with pytest.raises(ValueError):
        g.KvCache(cpu[..., :96], cpu[..., :96])
    with pytest.raises(ValueError):
        g.KvCache(cpu, cpu, torch.ones(2))                               # scales of a bf16 cache
    with pytest.raises(ValueError):
        g.Rope(torch.ones(12))
    with pytest.raises(ValueError):
        g.Rope(torch.ones(16), layout="thirds")
    with pytest.raises(ValueError):
        g.Rope(torch.ones(16), axes=torch.zeros(8, dtype=torch.int32))
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        g.qk_norm_rope(q, q)


def test_attention_slots_stay_below_32_bits():
    """Page numbers are compared in 32 bits: 2^31 pages of one slot would be a negative number of pages, none of them seen."""
    assert attention(page_size=1, pages=1 << 31) == g.A8W8_ERR_SHAPE
    assert attention(page_size=1, pages=1 << 32) == g.A8W8_ERR_SHAPE
    assert attention(page_size=16, pages=1 << 27) == g.A8W8_ERR_SHAPE
    assert attention(page_size=1, pages=(1 << 31) - 1, q=None) == g.A8W8_ERR_NULL
    assert attention(page_size=16, pages=(1 << 27) - 1, q=None) == g.A8W8_ERR_NULL


def test_attention_of_nothing_needs_no_table():
    assert attention(B=0, page_table=None, table_pages=0, q_start=None, kv_lens=None, workspace=None) == g.A8W8_OK
    assert attention(T=0, q=None, out=None, table_pages=0, page_table=None, workspace=None) == g.A8W8_OK
    assert attention(table_pages=0) == g.A8W8_ERR_SHAPE                  # rows, and nowhere to look for their keys
    assert attention(B=0, page_size=24) == g.A8W8_ERR_SHAPE


def test_handles_keep_what_was_checked(monkeypatch):
    """Another tensor in place of a checked one is refused, not taken for it."""
    monkeypatch.setattr(g, "_check_device", lambda named, device: None)
    k = torch.zeros(2, 16, 2, 128, dtype=torch.bfloat16)
    cache, rope = g.KvCache(k, k.clone()), g.Rope(torch.ones(16))
    for handle, names in ((cache, ("k", "v", "k_scale", "v_scale", "pages", "page_size", "kv_heads", "head_dim", "dtype")),
                          (rope, ("inv_freq", "axes", "layout", "rotary_dim"))):
        for name in names:
            before = getattr(handle, name)
            with pytest.raises(AttributeError):
                setattr(handle, name, torch.ones(16))
            assert getattr(handle, name) is before
    assert cache.operands() == (cache.k.data_ptr(), cache.v.data_ptr(), None, None)
    assert rope.operands() == (rope.inv_freq.data_ptr(), None, 32, 0)


class Reached(Exception):
    """The check before the descriptor is formed."""


@pytest.fixture
def on_host(monkeypatch):
    """A cache, queries and a table of host tensors, taken for those of a GPU up to the check of the current device."""
    def reached(index):
        raise Reached

    monkeypatch.setattr(g, "_check_device", lambda named, device: None)
    monkeypatch.setattr(g, "_check_heads", lambda name, x, shape, index: (x.shape, 0, 0, 0))
    monkeypatch.setattr(g, "_check_ints", lambda name, x, shape, index: 0)
    monkeypatch.setattr(g, "_check_current", reached)
    k = torch.zeros(2, 16, 2, 128, dtype=torch.bfloat16)
    ws = object.__new__(g.Workspace)
    ws.buf, ws.nbytes = torch.zeros(1), 1
    i32 = lambda *shape: torch.zeros(shape, dtype=torch.int32)  # noqa: E731
    return torch.zeros(1, 4, 128, dtype=torch.bfloat16), g.KvCache(k, k.clone()), i32(1, 2), i32(2), i32(1), ws


def test_counts_fit_their_fields(on_host):
    """2^32 + 1 is not taken for 1: a window of one key, an eager hint of one row."""
    with pytest.raises(Reached):
        g.paged_attention(*on_host, window=2 ** 31 - 1, sinks=2 ** 31 - 1, max_new=2 ** 31 - 1)
    for name in ("window", "sinks", "max_new"):
        for value in (-1, 2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 63):
            with pytest.raises(ValueError, match=name):
                g.paged_attention(*on_host, **{name: value})
    for kw in (dict(q_heads=2 ** 32 + 4), dict(q_heads=4, cu_count=2 ** 32 + 256)):
        with pytest.raises(ValueError):
            g.paged_attention_workspace_bytes(1, 1, cache=on_host[1], **kw)
