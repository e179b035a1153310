"""Timed cases of the attention half of a served decoder block, with their plain forms.

Two operators (formulas at each plain form below):

* rotate  norms of queries and keys for each head, the position rotation (one or several
          axes) and the paged cache's new entries in one pass: ``qk_norm_rope``;
* attend  attention of the new tokens of several sequences -- one each, or a chunk -- over a
          paged cache, with a sliding window and sink tokens: ``paged_attention``.

``own`` chooses what ``run`` calls: the plain forms here (elementary torch operations in 32
bits, rounded once at the end; angles in 64) or the library's operators.  ``exact`` gives the
same results from the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False
DEV = "cuda"
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # Rotation: one decoded token behind the qkv projection 14336 x 5120 (24 gated query heads, 4 key
        # heads of 256, a quarter of each head rotated): latency.
        dict(name="rotate 1 token gated 256", op="rotate", T=1, Hq=24, Hkv=4, D=256, R=64, layout="halves", axes=1,
             page=64, dtype="bf16", gated=True, pad=0),
        # A decode batch with padding rows, whole heads rotated in pairs, into an 8-bit cache.
        dict(name="rotate 61 tokens fp8 pairs", op="rotate", T=61, Hq=32, Hkv=8, D=128, R=128, layout="pairs", axes=1,
             page=16, dtype="fp8", gated=False, pad=3),
        # A prompt with images: positions of three axes; bandwidth.
        dict(name="rotate prompt 8191 3 axes", op="rotate", T=8191, Hq=24, Hkv=4, D=256, R=64, layout="halves", axes=3,
             page=64, dtype="bf16", gated=True, pad=0),
        # Attention: one request just after its prompt: latency.
        dict(name="decode 1 x 501", op="attend", dec=1, chunks=0, new=1, ctx=501, Hq=24, Hkv=4, D=256, page=64,
             dtype="bf16", window=0, sinks=0, gated=True, lens=1),
        # A ragged decode batch on small pages of an 8-bit cache.
        dict(name="decode 61 x 4000 fp8", op="attend", dec=61, chunks=0, new=1, ctx=4000, Hq=32, Hkv=8, D=128, page=16,
             dtype="fp8", window=0, sinks=0, gated=False, lens=2),
        # A decode batch of long requests on the gated heads.
        dict(name="decode 16 x 20000", op="attend", dec=16, chunks=0, new=1, ctx=20000, Hq=24, Hkv=4, D=256, page=64,
             dtype="bf16", window=0, sinks=0, gated=True, lens=3),
        # One very long request: few rows, the keys split over the whole card.
        dict(name="decode 1 x 131071", op="attend", dec=1, chunks=0, new=1, ctx=131071, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16", window=0, sinks=0, gated=False, lens=4),
        # Two chunks of long prompts, the earlier chunks in the cache.
        dict(name="chunks 2 x 2048 over 8000", op="attend", dec=0, chunks=2, new=2048, ctx=8000, Hq=24, Hkv=4, D=256,
             page=64, dtype="bf16", window=0, sinks=0, gated=True, lens=5),
        # A whole prompt at once.
        dict(name="prompt 8191", op="attend", dec=0, chunks=1, new=8191, ctx=0, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16", window=0, sinks=0, gated=False, lens=6),
        # A step of a serving program: one prompt chunk beside decoding requests, 8-bit cache.
        dict(name="mixed 1000 + 32 fp8", op="attend", dec=32, chunks=1, new=1000, ctx=6000, Hq=32, Hkv=8, D=128, page=16,
             dtype="fp8", window=0, sinks=0, gated=False, lens=7),
        # Sliding window with sink tokens: a decode batch far into long requests, and a prompt.
        dict(name="window decode 33 x 30000", op="attend", dec=33, chunks=0, new=1, ctx=30000, Hq=16, Hkv=2, D=64, page=64,
             dtype="bf16", window=1024, sinks=4, gated=False, lens=8),
        dict(name="window prompt 8000", op="attend", dec=0, chunks=1, new=8000, ctx=0, Hq=32, Hkv=8, D=128, page=64,
             dtype="bf16", window=1024, sinks=4, gated=False, lens=9),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


MOST_SQUARE = 32 * 8191 * 8191              # the largest listed set of scores
MOST_CACHE = 16 * 20000 * 4 * 256           # the largest listed cache, in elements of the keys


def draw(rng):
    Hkv, group, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 8, 12, 16]), rng.choice([64, 128, 128, 256])
    while Hkv * group > 64:
        group = rng.choice([1, 2, 3, 4, 5, 6, 8])
    heads = dict(Hq=Hkv * group, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "bf16", "fp8"]),
                 gated=rng.random() < 0.4)
    if rng.random() < 0.3:
        T = _log_int(rng, 1, min(16384, 8191 * 14336 // ((heads["Hq"] * (1 + heads["gated"]) + 2 * Hkv) * D)))
        return dict(op="rotate", T=T, R=rng.choice([D, D, D // 2, D // 4]), layout=rng.choice(["halves", "halves", "pairs"]),
                    axes=rng.choice([1, 1, 3]), pad=rng.choice([0, T // 16]), **heads)
    kind = rng.choice(["decode", "decode", "few", "chunks", "mixed"])
    while True:
        c = dict(op="attend", dec=0, chunks=0, new=1, ctx=0, window=0, sinks=0, lens=rng.randint(0, 999), **heads)
        if kind in ("decode", "mixed"):
            c["dec"] = _log_int(rng, 1, 128)
        if kind == "few":                    # several tokens a request, as where drafts are checked
            c["chunks"], c["new"] = _log_int(rng, 1, 64), rng.randint(2, 12)
        if kind in ("chunks", "mixed"):
            c["chunks"], c["new"] = rng.choice([1, 1, 2, 3]), _log_int(rng, 16, 8191)
        c["ctx"] = _log_int(rng, 16, 131071) if kind != "chunks" or rng.random() < 0.7 else 0
        if rng.random() < 0.3:
            c["window"], c["sinks"] = _log_int(rng, 64, 8192), rng.choice([0, 1, 4, 16])
        length = c["ctx"] + c["new"]
        if (c["dec"] + c["chunks"]) * length * Hkv * D <= MOST_CACHE and \
                c["chunks"] * c["new"] * length * c["Hq"] * max(1.0, D / 128) <= MOST_SQUARE:
            return c


def _lengths(case):
    """(new tokens, cached tokens before them) of each sequence: the chunks first, then the decoding ones;
    the first of each kind has the case's full sizes, the others are ragged."""
    rng = random.Random(case["lens"])
    seqs = []
    for i in range(case["chunks"]):
        seqs.append((case["new"], case["ctx"]) if i == 0 else
                    (rng.randint(max(1, case["new"] // 2), case["new"]), rng.randint(case["ctx"] // 4, case["ctx"])))
    for i in range(case["dec"]):
        seqs.append((1, case["ctx"] if i == 0 else rng.randint(case["ctx"] // 4, case["ctx"])))
    return seqs


# ---------------------------------------------------------------------------
# Inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _cache(g, case, pages):
    """Key and value pages with earlier tokens' entries; an 8-bit cache has one scale per head."""
    Hkv, D = case["Hkv"], case["D"]
    shape = (pages, case["page"], Hkv, D)
    if case["dtype"] == "bf16":
        return _randn(g, *shape).to(torch.bfloat16), _randn(g, *shape).to(torch.bfloat16), None, None
    ks, vs = (torch.rand(Hkv, generator=g, device=DEV) / 64 + 1 / 64 for _ in range(2))
    return tuple((_randn(g, *shape) / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
                 for s in (ks, vs)) + (ks, vs)


def _projection(g, T, case):
    """Rows of the qkv projection: each query head with its gate behind it where gated, then keys, then values."""
    Hq, Hkv, D, w = case["Hq"], case["Hkv"], case["D"], 2 if case["gated"] else 1
    rows = _randn(g, T, (w * Hq + 2 * Hkv) * D).to(torch.bfloat16)
    q, k, v = rows.split((w * Hq * D, Hkv * D, Hkv * D), 1)
    q = q.view(T, Hq, w * D)
    return q[..., :D], q[..., D:] if case["gated"] else None, k.view(T, Hkv, D), v.view(T, Hkv, D)


def prepare(case, seed):
    g, s = _gen(seed), dict(case)
    page, D = case["page"], case["D"]
    if case["op"] == "rotate":
        T, R = case["T"], case["R"]
        s["q"], _, s["k"], s["v"] = _projection(g, T, case)
        s["wq"], s["wk"] = (1.0 + 0.2 * _randn(g, D) for _ in range(2))
        s["inv_freq"] = (1e6 ** (-torch.arange(0, R, 2, device=DEV).double() / R)).float()
        s["axis_of"] = (torch.arange(R // 2, device=DEV) % case["axes"]).int()
        s["positions"] = torch.randint(0, 131072, (case["axes"], T), generator=g, device=DEV).int()
        pages = -(-T // page) + 2
        s["kc"], s["vc"], s["ks"], s["vs"] = _cache(g, case, pages)
        at = torch.randperm(pages, generator=g, device=DEV)[torch.arange(T, device=DEV) // page]
        s["slots"] = (at * page + torch.arange(T, device=DEV) % page).int()
        if case["pad"]:
            s["slots"][T - case["pad"]:] = -1        # padding rows of a fixed-size batch are not kept
        if own:           # what a serving program keeps: the cache's and the rotation's handles
            import fp8_block_scaled_a8w8_amd as lib
            s["cache"] = lib.KvCache(s["kc"], s["vc"], s["ks"], s["vs"])
            s["rope"] = lib.Rope(s["inv_freq"], axes=s["axis_of"], layout=case["layout"])
        return s
    seqs = _lengths(case)
    B, T = len(seqs), sum(n for n, _ in seqs)
    lens = [n + c for n, c in seqs]
    per = [-(-n // page) for n in lens]
    s["kc"], s["vc"], s["ks"], s["vs"] = _cache(g, case, sum(per) + 1)
    order = torch.randperm(sum(per) + 1, generator=g, device=DEV).int()
    table = torch.full((B, max(per)), -1, dtype=torch.int32, device=DEV)
    ends = torch.tensor(per).cumsum(0).tolist()
    for b in range(B):
        table[b, :per[b]] = order[ends[b] - per[b]:ends[b]]
    s["table"] = table
    s["q_start"] = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).to(DEV, torch.int32)
    s["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q, s["gate"], _, _ = _projection(g, T, case)
    s["q"] = 2.0 * q.contiguous()                    # scores of queries and keys with norms spread by more than 1
    if own:               # what a serving program keeps: the cache's handle and a workspace
        import fp8_block_scaled_a8w8_amd as lib
        s["cache"] = lib.KvCache(s["kc"], s["vc"], s["ks"], s["vs"])
        s["workspace"] = lib.Workspace(lib.paged_attention_workspace_bytes(T, B, case["Hq"], s["cache"]))
    return s


# ---------------------------------------------------------------------------
# One pass

def run(s):
    if own:
        import fp8_block_scaled_a8w8_amd as lib
        if s["op"] == "rotate":
            q, _ = lib.qk_norm_rope(s["q"], s["k"], s["rope"], s["positions"], q_weight=s["wq"], k_weight=s["wk"],
                                    eps=1e-6, v=s["v"], cache=s["cache"], slots=s["slots"])
            return q, s["kc"], s["vc"]
        return lib.paged_attention(s["q"], s["cache"], s["table"], s["q_start"], s["kv_lens"], s["workspace"],
                                   window=s["window"], sinks=s["sinks"], gate=s["gate"],
                                   max_new=s["new"] if s["chunks"] else 1)
    return {"rotate": _plain_rotate, "attend": _plain_attend}[s["op"]](s)


def _turn(x, cos, sin, R, layout):
    """Pairs (a, b) of the first R dimensions become (a cos - b sin, b cos + a sin)."""
    if layout == "halves":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., R:]), -1)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., R:]), -1)


def _plain_rotate(s):
    """x weight / sqrt(mean(x^2) + eps) of each head of q and k, rotated by positions[axis_i] * inv_freq_i;
    k and v to their slots of the cache (8 bits: value / scale of the head), rows of slot -1 nowhere."""
    R = s["R"]
    angle = s["positions"][s["axis_of"].long()].t().double() * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q, k = s["q"].float(), s["k"].float()
    q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + 1e-6) * s["wq"]
    k = k * torch.rsqrt((k * k).mean(-1, keepdim=True) + 1e-6) * s["wk"]
    q, k, v = _turn(q, cos, sin, R, s["layout"]), _turn(k, cos, sin, R, s["layout"]), s["v"].float()
    kept = (s["slots"] >= 0)[:, None, None]          # a padding row repeats the first row's entry
    at = torch.where(kept[:, 0, 0], s["slots"], s["slots"][0]).long()
    for x, cache, scale in ((k, s["kc"], s["ks"]), (v, s["vc"], s["vs"])):
        x = torch.where(kept, x, x[:1])
        if scale is None:
            cache.view(-1, *cache.shape[2:])[at] = x.to(torch.bfloat16)
        else:
            x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            cache.view(torch.uint8).view(-1, *cache.shape[2:])[at] = x.view(torch.uint8)
    return q.to(torch.bfloat16), s["kc"], s["vc"]


def _plain_group(s, seqs, rows, n, L):
    """Attention of some sequences' rows [B,n] (-1: none) over their first L cached tokens: fp32 [B,n,Hq,D]."""
    B, Hq, Hkv, D, page, w, sinks = len(seqs), s["Hq"], s["Hkv"], s["D"], s["page"], s["window"], s["sinks"]
    new = (s["q_start"][1:] - s["q_start"][:-1])[seqs]
    p = (s["kv_lens"][seqs] - new)[:, None] + torch.arange(n, device=DEV)      # the rows' positions
    j = torch.arange(L, device=DEV).expand(B, L)
    if w and sinks + w + n < L:                      # only the sinks and what any row's window reaches
        first = (p[:, :1] - w + 1).clamp(min=sinks)
        j = torch.cat((j[:, :sinks], (first + torch.arange(w + n - 1, device=DEV)).clamp(max=L)), 1)
    at, offset = s["table"][seqs].gather(1, (j // page).clamp(max=s["table"].shape[1] - 1)).clamp(min=0).long(), j % page

    def cached(c, scale):                            # [B, Hkv, keys, D]
        x = c[at, offset].float() if scale is None else c.view(torch.uint8)[at, offset].view(c.dtype).float() * scale[:, None]
        return x.permute(0, 2, 1, 3).contiguous()

    G = Hq // Hkv
    q = s["q"][rows.clamp(min=0)].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    score = torch.matmul(q, cached(s["kc"], s["ks"]).transpose(2, 3).contiguous()).mul_(D ** -0.5)
    seen = j[:, None] <= p[:, :, None]
    if w:
        seen &= (j[:, None] > p[:, :, None] - w) | (j[:, None] < sinks)
    score = score.view(B, Hkv, G, n, -1).masked_fill_(~seen[:, None, None], -math.inf)
    e = torch.exp(score.sub_(score.amax(-1, keepdim=True)))
    out = torch.matmul(e.view(B, Hkv, G * n, -1), cached(s["vc"], s["vs"])).view(B, Hkv, G, n, D) / e.sum(-1, keepdim=True)
    return out.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)


def _plain_attend(s):
    """Row i of the n new tokens of a sequence of len tokens is at p = len - n + i and sees the keys j <= p, of
    these with a window only j > p - window and the first sinks: sum_j softmax_j(q . k_j / sqrt(D)) v_j, times
    sigmoid(gate)."""
    T, C, n = s["q"].shape[0], s["chunks"], s["new"]
    out = torch.zeros(T, s["Hq"], s["D"], device=DEV)
    if C:                                            # the chunks, padded to the longest
        seqs = torch.arange(C, device=DEV)
        rows = s["q_start"][:C, None].long() + torch.arange(n, device=DEV)
        there = rows < s["q_start"][1:C + 1, None]
        o = _plain_group(s, seqs, rows.clamp(max=T - 1), n, s["ctx"] + n)
        out.index_add_(0, rows.clamp(max=T - 1).view(-1), torch.where(there[:, :, None, None], o, 0).flatten(0, 1))
    if s["dec"]:                                     # the decoding sequences: one row each
        seqs = torch.arange(C, C + s["dec"], device=DEV)
        rows = s["q_start"][C:-1].long()[:, None]
        out.index_add_(0, rows.view(-1), _plain_group(s, seqs, rows, 1, s["ctx"] + 1)[:, 0])
    if s["gate"] is not None:
        out = out / (1.0 + torch.exp(-s["gate"].float()))
    return out.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# What a pass cannot do without

def _keys(case):
    """(keys that any new row of a sequence sees, keys seen summed over its rows), each summed over the sequences."""
    any_row = all_rows = 0
    w, sinks = case["window"], case["sinks"]
    for n, ctx in _lengths(case):
        if not w:
            any_row += ctx + n
            all_rows += n * ctx + n * (n + 1) // 2
            continue
        any_row += ctx + n - max(0, max(0, ctx - w + 1) - sinks)
        for i in range(n):
            all_rows += ctx + i + 1 - max(0, max(0, ctx + i - w + 1) - sinks)
    return any_row, all_rows


def work(case):
    Hq, Hkv, D, size = case["Hq"], case["Hkv"], case["D"], 2 if case["dtype"] == "bf16" else 1
    if case["op"] == "rotate":
        T = case["T"]
        return {"bytes": T * D * (4 * Hq + 4 * Hkv + 2 * Hkv * size) + 4 * T * (case["axes"] + 1),
                "flops": T * (Hq + Hkv) * (4 * D + 3 * case["R"])}
    any_row, all_rows = _keys(case)
    T = sum(n for n, _ in _lengths(case))
    return {"bytes": 2 * any_row * Hkv * D * size + T * Hq * D * (6 if case["gated"] else 4), "flops": 4 * D * Hq * all_rows}


# ---------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "attend": _exact_attend}[case["op"]](s)


def _exact_rotate(s):
    R, D = s["R"], s["D"]
    half = torch.arange(R // 2, device=DEV)
    first, second = (half, half + R // 2) if s["layout"] == "halves" else (2 * half, 2 * half + 1)
    angle = torch.stack([s["positions"][a].double() * f for a, f in zip(s["axis_of"].tolist(), s["inv_freq"].double())], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def head(x, w):
        x = x.double()
        x = w.double() * x / (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / D + 1e-6).sqrt()
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    out = [head(s["q"], s["wq"])]
    for x, cache, scale in ((head(s["k"], s["wk"]), s["kc"], s["ks"]), (s["v"].double(), s["vc"], s["vs"])):
        if scale is not None:
            x = torch.clamp(x / scale.double()[:, None], -E4M3_MAX, E4M3_MAX)
        c = cache.double()
        keep = torch.nonzero(s["slots"] >= 0)[:, 0]
        slot = s["slots"][keep].long()
        c[slot // s["page"], slot % s["page"]] = x[keep]
        out.append(c)
    return tuple(out)


def _exact_attend(s):
    G, D = s["Hq"] // s["Hkv"], s["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    starts, lens = s["q_start"].tolist(), s["kv_lens"].tolist()
    for b, length in enumerate(lens):
        r0, r1 = starts[b], starts[b + 1]
        t = torch.arange(length, device=DEV)
        place, offset = s["table"][b][t // s["page"]].long(), t % s["page"]
        hidden = t[None] > (torch.arange(r0, r1, device=DEV) + (length - r1))[:, None]
        if s["window"]:
            past = t[None] <= (torch.arange(r0, r1, device=DEV) + (length - r1 - s["window"]))[:, None]
            hidden = hidden | (past & (t[None] >= s["sinks"]))
        for h in range(s["Hkv"]):
            k, v = s["kc"][:, :, h].view(s["kc"].shape[0], -1, D), s["vc"][:, :, h]
            if s["ks"] is not None:
                k, v = (c.view(torch.uint8)[place, offset].view(c.dtype).double() * float(x[h])
                        for c, x in ((k, s["ks"]), (v, s["vs"])))
            else:
                k, v = k[place, offset].double(), v[place, offset].double()
            for i in range(h * G, h * G + G):
                w = (s["q"][r0:r1, i].double() @ k.T) / math.sqrt(D)
                w = torch.softmax(w.masked_fill(hidden, -math.inf), 1)
                out[r0:r1, i] = w @ v
    return out if s["gate"] is None else out * torch.sigmoid(s["gate"].double())
