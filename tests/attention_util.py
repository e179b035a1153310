"""Plain 64-bit forms of the attention half's operators, and inputs for them, on the CPU."""
from __future__ import annotations

import math

import torch

EPS32 = 2.0 ** -24      # half a step of fp32, relative
BF16 = 2.0 ** -8        # of bf16
E4M3 = 2.0 ** -4        # of e4m3


def rotate64(x, weight, eps, positions, inv_freq, axes, layout):
    """x [T,H,D] normalised per head (weight None: not) and rotated, float64; also sum |terms| per element, what
    roundings of the products are relative to."""
    x = x.double()
    T, _, D = x.shape
    if weight is not None:
        x = weight.double() * x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    mag = x.abs()
    if inv_freq is not None:
        h = len(inv_freq)
        pos = positions if positions.dim() == 2 else positions[None]
        ax = torch.zeros(h, dtype=torch.long) if axes is None else axes.long().clamp(0, len(pos) - 1)
        # float64 products of a 31-bit and a 24-bit whole or fp32 number: off by 2^-53 of at most 2^31
        angle = pos[ax].t().double() * inv_freq.double()
        c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
        i = torch.arange(h)
        first, second = (i, i + h) if layout == "halves" else (2 * i, 2 * i + 1)
        y, m = x.clone(), mag.clone()
        a, b = x[..., first], x[..., second]
        y[..., first], y[..., second] = a * c - b * s, b * c + a * s
        m[..., first] = m[..., second] = a.abs() + b.abs()
        x, mag = y, m
    return x, mag


def values(cache, scale):
    """The numbers a cache [pages,page,H,D] stands for, float64."""
    x = cache.cpu().double()
    return x if scale is None else x * scale.cpu().double()[:, None]


def attend64(q, k, v, table, page, q_start, lens, scale, window=0, sinks=0, gate=None, out=None):
    """The definition, row by row, from cached values k, v [pages,page,H,D] (float64).  Returns (out, weight) with
    weight = sum_j w_j |v_j| per element, what errors of the softmax weights are relative to, and the largest
    scale * sum_d |q_d k_jd| of any visible key per row and head [T,Hq]."""
    T, Hq, D = q.shape
    pages, _, Hkv, _ = k.shape
    G = Hq // Hkv
    q = q.cpu().double()
    out = torch.zeros(T, Hq, D, dtype=torch.float64) if out is None else out.cpu().double().clone()
    mag, most = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    for b in range(len(lens)):
        r0, r1 = int(q_start[b]), int(q_start[b + 1])
        if r0 < 0 or r1 > T or r1 < r0:
            continue
        for t in range(r0, r1):
            p = int(lens[b]) - (r1 - r0) + t - r0
            j = torch.arange(max(0, min(p + 1, table.shape[1] * page)))      # keys past the table are not seen
            if window:
                j = j[(j > p - window) | (j < sinks)]
            pg = table[b].cpu()[j // page].long()
            ok = (pg >= 0) & (pg < pages)
            j, pg = j[ok], pg[ok]
            if not len(j):
                out[t] = 0
                continue
            kk, vv = k[pg, j % page], v[pg, j % page]                    # [n,Hkv,D]
            for h in range(Hq):
                kh, vh = kk[:, h // G], vv[:, h // G]
                s = scale * (kh @ q[t, h])
                w = torch.softmax(s, 0)
                out[t, h] = (w[:, None] * vh).sum(0)
                mag[t, h] = (w[:, None] * vh.abs()).sum(0)
                most[t, h] = (abs(scale) * (kh.abs() @ q[t, h].abs())).max()
            if gate is not None:
                g = torch.sigmoid(gate[t].cpu().double())
                out[t], mag[t] = out[t] * g, mag[t] * g
    return out, mag, most


def attend_tolerance(out, mag, most, D, rows, keys):
    """Bound on |result - out| element by element.

    A score is a sum of D products in fp32 and a scaling: off by (D + 4) EPS32 most; the exponential doubles
    that at most (numerator and maximum) and adds a few ulps, so a weight is off by d = 2 (D + 8) EPS32 max(1, most)
    relatively, its numerator's rounding to bf16 adds BF16 (2^-16 as two terms, in sequences with up to 16 rows per
    key head), the fp32 sums over the keys keys * EPS32 each; numerator and denominator once each.  The result is
    rounded once."""
    d = 2.0 * (D + 8) * EPS32 * most.clamp(min=1.0)[..., None] + 2 * keys * EPS32
    p = BF16 if rows > 16 else 2.0 ** -16
    return (mag * (p + 2 * d)) * (1 + BF16) + out.abs() * (BF16 + 2.0 ** -20) + 1e-37


class Cache:
    """A paged cache of sequences with the given lengths on the CPU: shuffled pages, everything no sequence owns --
    slots behind the last token, unused pages -- poisoned with NaN and infinities."""

    def __init__(self, lens, Hkv, D, page, dtype, seed, spare=3, std=1.0):
        g = torch.Generator().manual_seed(seed)
        per = [-(-max(0, n) // page) for n in lens]
        self.page, self.lens, pages = page, lens, sum(per) + spare
        order = torch.randperm(pages, generator=g)
        self.table = torch.full((len(lens), max(per + [1]) + 1), -1, dtype=torch.int32)
        shape = (pages, page, Hkv, D)
        k, v = (std * torch.randn(shape, generator=g) for _ in range(2))
        live = torch.zeros(pages, page, dtype=torch.bool)
        at = 0
        for b, n in enumerate(per):
            own = order[at:at + n]
            at += n
            self.table[b, :n] = own.int()
            live[own] = (torch.arange(n * page) < lens[b]).view(n, page)
        self.ks = self.vs = None
        if dtype == "fp8":
            self.ks, self.vs = (torch.rand(Hkv, generator=g) / 64 + 1 / 64 for _ in range(2))
            k, v = ((x / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) for x, s in
                    ((k, self.ks), (v, self.vs)))
            k[~live], v[~live] = 0x7f, 0xff                              # NaN
            self.k, self.v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        else:
            self.k, self.v = k.to(torch.bfloat16), v.to(torch.bfloat16)
            self.k[~live], self.v[~live] = math.nan, math.inf

    def to(self, device):
        import fp8_block_scaled_a8w8_amd as g
        move = [None if x is None else x.to(device) for x in (self.k, self.v, self.ks, self.vs)]
        return g.KvCache(*move)
