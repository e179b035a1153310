"""Timed cases of the serving operators beside the a8w8 GEMM, with their plain forms.

Three operators (formulas at each plain form below):

* route  top-k routing of tokens to experts: ``moe_route``;
* moe    a whole mixture-of-experts layer for a few tokens on fp8 block-scaled
         expert weights: ``moe_layer_a16w8_blockscale``;
* lora   low-rank adapters of many requests beside one shared a8w8 projection:
         ``gemm_a8w8_blockscale_lora``.

``own`` chooses what ``run`` calls: the plain forms here (elementary torch
operations in 32 bits, rounded once at the end) or the library's operators.
``exact`` gives the same results from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False
DEV = "cuda"
BLOCK = 128
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# Cases

def listed():
    return [
        # Routing: one decoded token (pure latency), a decode batch with padding rows,
        # and a prompt (the logits of 16381 tokens: bandwidth).
        dict(name="route decode 1x128", op="route", T=1, E=128, k=8, dtype="bf16", score="softmax", renorm=True, pad=0),
        dict(name="route batch 61x60", op="route", T=61, E=60, k=4, dtype="f32", score="sigmoid", renorm=True, pad=3),
        dict(name="route prompt 16381x256", op="route", T=16381, E=256, k=8, dtype="f32", score="softmax", renorm=False,
             pad=0),
        # The layer: one token through many small experts (what a single stream decodes with).
        dict(name="moe 1 token 128x768", op="moe", T=1, E=128, k=8, H=2048, I=768, packed=False, pad=0),
        # A small batch over few wide experts, hidden size of the decode projections.
        dict(name="moe 5 tokens 32x1792", op="moe", T=5, E=32, k=4, H=5120, I=1792, packed=False, pad=0),
        # A full decode tile, weights prepacked offline, two padding rows of a fixed-size batch.
        dict(name="moe 16 tokens packed", op="moe", T=16, E=128, k=8, H=2048, I=768, packed=True, pad=2),
        # A ragged batch that reaches nearly every expert.
        dict(name="moe 61 tokens 256x512", op="moe", T=61, E=256, k=8, H=2048, I=512, packed=False, pad=0),
        # The largest batch of one pass: every expert's weights, several tokens each.
        dict(name="moe 256 tokens 128x768", op="moe", T=256, E=128, k=8, H=2048, I=768, packed=False, pad=0),
        # Adapters: one request decoding beside the out projection.
        dict(name="lora 1 token 5120x6144", op="lora", M=1, N=5120, K=6144, R=16, L=8, ids="tokens", packed=False),
        # A decode batch, each token with its own request's adapter, beside the qkv projection.
        dict(name="lora 16 tokens 14336x5120", op="lora", M=16, N=14336, K=5120, R=16, L=32, ids="tokens", packed=False),
        # A larger ragged decode batch with wide adapters.
        dict(name="lora 133 tokens r64", op="lora", M=133, N=5120, K=6144, R=64, L=24, ids="tokens", packed=False),
        # Prompts of several requests packed one after another, some without an adapter.
        dict(name="lora prompts 2048", op="lora", M=2048, N=14336, K=5120, R=32, L=16, ids="segments", packed=False),
    ]


MOST_EXPERT_BYTES = 3 * 32 * 5120 * 1792     # the largest listed set of expert weights
MOST_GEMM = 2048 * 14336 * 5120              # the largest listed projection


def _log_int(rng, lo, hi, skip=3072):
    while True:
        v = max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
        if v != skip:
            return v


def _of_128(rng, lo, hi, factor=1):
    return 128 * _log_int(rng, lo, hi, skip=24 // factor)


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "lora", "lora"])
    if op == "route":
        E = _log_int(rng, 8, 512)
        return dict(op=op, T=_log_int(rng, 1, 16384 * 256 // max(E, 256)), E=E, k=rng.randint(1, min(16, E)),
                    dtype=rng.choice(["bf16", "f32"]), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, pad=0)
    if op == "moe":
        while True:
            c = dict(op=op, T=_log_int(rng, 1, 256), E=_log_int(rng, 8, 256), k=rng.randint(1, 8),
                     H=_of_128(rng, 4, 40), I=_of_128(rng, 2, 16, factor=2), packed=rng.random() < 0.3)
            c["pad"] = rng.choice([0, c["T"] // 8])
            # at least 4 MB of expert weights, so that a call is more than its launches
            if 4 << 20 <= 3 * c["E"] * c["H"] * c["I"] <= MOST_EXPERT_BYTES // 2:
                return c
    while True:
        c = dict(op=op, M=_log_int(rng, 1, 4096), N=_log_int(rng, 256, 16384), K=_of_128(rng, 8, 48),
                 R=rng.choice([8, 16, 24, 32, 64, 128]), L=_log_int(rng, 1, 48),
                 ids=rng.choice(["tokens", "segments"]), packed=rng.random() < 0.3)
        if c["M"] * c["N"] * c["K"] <= MOST_GEMM:
            return c


# ---------------------------------------------------------------------------
# Inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _block_weights(g, lead, N, K):
    """N(0, 0.02) weights [*lead, N, K] as e4m3 codes with one fp32 scale (amax / 448) per 128 x 128 block."""
    w = torch.randn(*lead, N, K, generator=g, device=DEV, dtype=torch.float32).mul_(0.02)
    full = -(-N // BLOCK) * BLOCK
    wp = torch.nn.functional.pad(w, (0, 0, 0, full - N)) if full != N else w
    blocks = wp.view(*lead, full // BLOCK, BLOCK, K // BLOCK, BLOCK)
    s = blocks.abs().amax(dim=(-3, -1)) / E4M3_MAX
    codes = (blocks / s[..., :, None, :, None]).to(torch.float8_e4m3fn).view(*lead, full, K)[..., :N, :].contiguous()
    return codes, s.contiguous()


def _pack(W):
    """Row-major codes [*lead, N, K] in the library's packed order: per 16-row tile and 128-wide K block
    2 KB, [half][lane][16 bytes], lane l holding row l % 16, columns 64 half + 16 (l // 16) .. + 16."""
    lead, (N, K) = W.shape[:-2], W.shape[-2:]
    n = -(-N // 16) * 16
    b = torch.zeros(*lead, n, K, dtype=torch.uint8, device=W.device)
    b[..., :N, :] = W.view(torch.uint8)
    b = b.view(-1, n // 16, 16, K // 128, 2, 4, 16).permute(0, 1, 3, 4, 5, 2, 6)
    return b.reshape(*lead, n, K).contiguous()


def _unpack(P, N):
    lead, (n, K) = P.shape[:-2], P.shape[-2:]
    b = P.view(-1, n // 16, K // 128, 2, 4, 16, 16).permute(0, 1, 5, 2, 3, 4, 6)
    return b.reshape(*lead, n, K)[..., :N, :].view(torch.float8_e4m3fn)


def _logits(g, T, E, dtype, pad):
    x = torch.randn(T, E, generator=g, device=DEV).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    if pad:
        x[T - pad:] = float("-inf")          # padding rows of a fixed-size batch reach no expert
    return x


def prepare(case, seed):
    g, s = _gen(seed), dict(case)
    if case["op"] == "route":
        s["logits"] = _logits(g, case["T"], case["E"], case["dtype"], case["pad"])
        if own:
            import fp8_block_scaled_a8w8_amd  # noqa: F401  (loaded before the timed call)
        return s
    if case["op"] == "moe":
        T, E, H, I = case["T"], case["E"], case["H"], case["I"]
        s["k"] = min(case["k"], E)
        s["X"] = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
        s["logits"] = _logits(g, T, E, "f32", case["pad"])
        s["W13"], s["s13"] = _block_weights(g, (E,), 2 * I, H)
        s["W2"], s["s2"] = _block_weights(g, (E,), H, I)
        if case["packed"]:
            s["W13"], s["W2"] = _pack(s["W13"]), _pack(s["W2"])
        if own:   # what a serving program keeps: the expert weights' handle and a workspace
            import fp8_block_scaled_a8w8_amd as lib
            s["experts"] = lib.MoeExperts(s["W13"], s["s13"], s["W2"], s["s2"], packed=case["packed"])
            s["workspace"] = lib.Workspace(lib.moe_workspace_bytes(T, s["k"], s["experts"]))
        return s
    M, N, K, R, L = (case[n] for n in ("M", "N", "K", "R", "L"))
    s["X"] = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    s["W"], s["w_scale"] = _block_weights(g, (), N, K)
    s["A"] = (torch.randn(L, R, K, generator=g, device=DEV) / math.sqrt(K)).to(torch.bfloat16)
    s["B"] = (torch.randn(L, N, R, generator=g, device=DEV) * 0.1).to(torch.bfloat16)
    s["scaling"] = torch.rand(L, generator=g, device=DEV) * 1.5 + 0.5
    if case["ids"] == "tokens":              # every token a request of its own, one in L + 1 without an adapter
        ids = torch.randint(-1, L, (M,), generator=g, device=DEV)
    else:                                    # prompts one after another, cut at random places
        cuts = torch.randint(0, M, (max(1, min(L, M // 8)),), generator=g, device=DEV)
        owner = torch.randint(-1, L, (M,), generator=g, device=DEV)
        at = (torch.arange(M, device=DEV)[:, None] >= cuts[None, :]).sum(1)
        ids = owner[at]
    s["ids"] = ids.to(torch.int32)
    if case["packed"]:
        s["W"] = _pack(s["W"])
    if own:       # what a serving program keeps: the adapters' handle and a workspace
        import fp8_block_scaled_a8w8_amd as lib
        s["adapters"] = lib.LoraAdapters(s["A"], s["B"], s["scaling"])
        s["workspace"] = lib.Workspace(lib.lora_workspace_bytes(M, N, K, s["adapters"]))
    return s


# ---------------------------------------------------------------------------
# One pass

def run(s):
    if own:
        import fp8_block_scaled_a8w8_amd as lib
        if s["op"] == "route":
            return lib.moe_route(s["logits"], s["k"], score=s["score"], renormalize=s["renorm"])
        if s["op"] == "moe":
            return lib.moe_layer_a16w8_blockscale(s["X"], s["logits"], s["experts"], s["k"], s["workspace"])
        return lib.gemm_a8w8_blockscale_lora(s["X"], s["W"], s["w_scale"], s["adapters"], s["ids"], s["workspace"],
                                             packed_n=s["N"] if s["packed"] else None)
    return {"route": _plain_route, "moe": _plain_moe, "lora": _plain_lora}[s["op"]](s)


def _route(logits, k, score, renorm):
    """Routing: the k experts of the largest logits, best first, ties to the lowest index.  A logit of
    -inf (or NaN) masks its expert: slots left without one get id -1 and weight 0.  Weights: softmax over
    the row, or sigmoid; renorm divides them by the chosen ones' sum."""
    x = logits.float()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x).clamp(max=torch.finfo(torch.float32).max)
    v, ids = torch.sort(x, dim=1, descending=True, stable=True)
    v, ids = v[:, :k], ids[:, :k]
    there = v > -math.inf
    if score == "softmax":
        top = torch.where(there[:, :1], v[:, :1], torch.zeros_like(v[:, :1]))
        w = torch.exp(v - top)
        total = w.sum(1, keepdim=True) if renorm else torch.exp(x - top).sum(1, keepdim=True)
    else:
        w = 1.0 / (1.0 + torch.exp(-v))
        total = w.sum(1, keepdim=True) if renorm else torch.ones_like(w[:, :1])
    w = torch.where(there & (total > 0), w / total, torch.zeros_like(w))
    return w, torch.where(there, ids, torch.full_like(ids, -1)).to(torch.int32)


def _plain_route(s):
    return _route(s["logits"], s["k"], s["score"], s["renorm"])


def _dequant(codes, s):
    lead, (N, K) = codes.shape[:-2], codes.shape[-2:]
    return codes.float() * s.repeat_interleave(BLOCK, -2)[..., :N, :].repeat_interleave(BLOCK, -1)


def _plain_moe(s):
    """The layer: Y[t] = bf16(sum_j w[t,j] W2[e] (silu(W13[e] gate . x_t) * (W13[e] up . x_t))), e = ids[t,j]."""
    T, E, H, I, k = (s[n] for n in ("T", "E", "H", "I", "k"))
    W13, W2 = s["W13"], s["W2"]
    if s["packed"]:
        W13, W2 = _unpack(W13, 2 * I), _unpack(W2, H)
    w, ids = _route(s["logits"], k, "softmax", True)
    x, at = s["X"].float(), ids.clamp(min=0).long()
    if T * k < E:                            # few slots: each slot's own expert
        e = at.view(-1)
        gu = torch.matmul(_dequant(W13.view(torch.uint8)[e].view(torch.float8_e4m3fn), s["s13"][e]),
                          x.repeat_interleave(k, 0)[:, :, None])[..., 0]
        h = gu[:, :I] / (1.0 + torch.exp(-gu[:, :I])) * gu[:, I:]
        y = torch.matmul(_dequant(W2.view(torch.uint8)[e].view(torch.float8_e4m3fn), s["s2"][e]), h[:, :, None])[..., 0]
        y = (y.view(T, k, H) * w[:, :, None]).sum(1)
    else:                                    # every expert, weighted by zero where it was not chosen
        full = torch.zeros(T, E, device=x.device).scatter_add_(1, at, w)
        gu = torch.matmul(x[None], _dequant(W13, s["s13"]).transpose(1, 2))
        h = gu[..., :I] / (1.0 + torch.exp(-gu[..., :I])) * gu[..., I:]
        y = torch.matmul(h, _dequant(W2, s["s2"]).transpose(1, 2))
        y = (y * full.t()[:, :, None]).sum(0)
    return y.to(torch.bfloat16)


def _plain_lora(s):
    """The projection: Y[m] = bf16(sum of e4m3(x_m) . e4m3(W) times their block scales
    + scaling[a] B[a] (A[a] x_m)), a = ids[m]; nothing added where a is negative."""
    M, N, K, L, R = (s[n] for n in ("M", "N", "K", "L", "R"))
    W = _unpack(s["W"], N) if s["packed"] else s["W"]
    x = s["X"].float()
    xg = x.view(M, K // BLOCK, BLOCK)
    sc = xg.abs().amax(2, keepdim=True) / E4M3_MAX
    q = torch.where(sc > 0, xg / sc, torch.zeros_like(xg)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float()
    y = torch.matmul((q * sc).view(M, K), _dequant(W, s["w_scale"]).t())
    a = s["ids"].long()
    mine = (a[:, None] == torch.arange(L, device=a.device)[None]).float() * s["scaling"][None]
    v = torch.matmul(x, s["A"].float().view(L * R, K).t()).view(M, L, R) * mine[:, :, None]
    y += torch.matmul(v.view(M, L * R), s["B"].float().permute(0, 2, 1).reshape(L * R, N))
    return y.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# What a pass cannot do without

def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * (2 if case["dtype"] == "bf16" else 4) + T * k * 8, "flops": 3 * T * E}
    if case["op"] == "moe":
        T, E, H, I = (case[n] for n in ("T", "E", "H", "I"))
        k, live = min(case["k"], E), T - case["pad"]
        reached = E * (1.0 - (1.0 - k / E) ** live)          # expected distinct experts
        return {"bytes": reached * 3 * H * I * (1 + 4 / BLOCK ** 2) + 4 * T * H + 4 * T * E, "flops": 6 * live * k * H * I}
    M, N, K, R, L = (case[n] for n in ("M", "N", "K", "R", "L"))
    if case["ids"] == "tokens":
        reached = L * (1.0 - (1.0 - 1.0 / (L + 1)) ** M)
    else:
        reached = L * (1.0 - (1.0 - 1.0 / (L + 1)) ** (max(1, min(L, M // 8)) + 1))
    return {"bytes": N * K + 2 * M * K + 2 * M * N + 2 * reached * R * (N + K) + N * K * 4 / BLOCK ** 2,
            "flops": 2 * M * N * K + 2 * M * R * (N + K)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "moe": _exact_moe, "lora": _exact_lora}[case["op"]](s)


def _exact_route(s, score=None, renorm=None, logits=None):
    score, renorm = score or s["score"], s["renorm"] if renorm is None else renorm
    x = (s["logits"] if logits is None else logits).double()
    x = torch.nan_to_num(x, nan=-math.inf, posinf=float(torch.finfo(torch.float32).max), neginf=-math.inf)
    p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    left, rows = x.clone(), torch.arange(len(x), device=x.device)
    w = torch.zeros(len(x), s["k"], dtype=torch.float64, device=x.device)
    ids = torch.full((len(x), s["k"]), -1, dtype=torch.int32, device=x.device)
    for j in range(s["k"]):                  # one expert after another: the lowest index of the largest logit left
        top = left.amax(1, keepdim=True)
        e = torch.where(left == top, torch.arange(x.shape[1], device=x.device)[None], x.shape[1]).amin(1)
        there = top[:, 0] > -math.inf
        ids[:, j] = torch.where(there, e, -1).int()
        w[:, j] = torch.where(there, p[rows, e], 0.0)
        left[rows, e] = -math.inf
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return w, ids


def _weights64(codes, scale):
    N, K = codes.shape
    rows = torch.arange(N, device=codes.device) // BLOCK
    cols = torch.arange(K, device=codes.device) // BLOCK
    return codes.double() * scale.double()[rows][:, cols]


def _exact_moe(s):
    T, E, H, I = (s[n] for n in ("T", "E", "H", "I"))
    W13, W2 = s["W13"], s["W2"]
    if s["packed"]:
        W13, W2 = _unpack(W13, 2 * I), _unpack(W2, H)
    w, ids = _exact_route(s, score="softmax", renorm=True)
    x = s["X"].double()
    y = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    for e in torch.unique(ids[ids >= 0]).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        gu = x[t] @ _weights64(W13[e], s["s13"][e]).T
        g, u = gu[:, :I], gu[:, I:]
        y[t] += w[t, j][:, None] * ((g * torch.sigmoid(g) * u) @ _weights64(W2[e], s["s2"][e]).T)
    return y


def _e4m3_table(device):
    """Every finite magnitude of e4m3 (bias 7, three mantissa bits, code 0x7f is NaN), ascending by code."""
    c = torch.arange(127, device=device)
    e, m = (c >> 3).double(), (c & 7).double()
    return torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)


def _exact_lora(s):
    M, N, K = (s[n] for n in ("M", "N", "K"))
    W = _unpack(s["W"], N) if s["packed"] else s["W"]
    xg = s["X"].float().view(M, K // BLOCK, BLOCK)
    sc = xg.abs().amax(2, keepdim=True) / E4M3_MAX          # the scale and the quotient are 32-bit by definition
    quot = torch.where(sc > 0, xg / sc, torch.zeros_like(xg)).double()
    table = _e4m3_table(quot.device)
    mag = quot.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(table, mag.contiguous()).clamp(1, 126)
    below, above = mag - table[hi - 1], table[hi] - mag
    code = torch.where((below < above) | ((below == above) & ((hi - 1) % 2 == 0)), hi - 1, hi)
    xq = (torch.sign(quot) * table[code] * sc.double()).view(M, K)
    y = xq @ _weights64(W, s["w_scale"]).T
    x, ids = s["X"].double(), s["ids"]
    for a in torch.unique(ids[ids >= 0]).tolist():
        t = torch.nonzero(ids == a)[:, 0]
        y[t] += s["scaling"][a].double() * ((x[t] @ s["A"][a].double().T) @ s["B"][a].double().T)
    return y
