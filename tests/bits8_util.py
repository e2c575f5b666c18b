"""The 8-bit operators' definitions in 64 bits on the CPU, for the tests: norm, products, the paged cache with its
growing block scales and attention over it, written from include/ple_8bit.h with plain torch operations."""
from __future__ import annotations

import math

import torch

from fp4_util import e4m3, rotate  # noqa: F401  (a code's value from its fields; the rotation)

F64, U8 = torch.float64, torch.uint8
LEAST, MOST = 2.0 ** -32, 2.0 ** 32


def codes_of(x):
    """The nearest e4m3fn codes of x (64 bits, |x| <= 448 or NaN), ties to the even one: every code's value is searched."""
    grid = e4m3(torch.arange(0x7F, dtype=U8))          # 0 .. 448, rising
    a = x.abs()
    hi = torch.bucketize(a, grid).clamp(max=0x7E)      # the first value not below a
    lo = (hi - 1).clamp(min=0)
    down, up = a - grid[lo], grid[hi] - a
    near = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    near = torch.where(torch.isnan(x), 0x7F, near)
    return (near + 128 * torch.signbit(x)).to(U8)


def block_scale(top):
    """The least power of two s with top <= 448 s, in 2^-32 .. 2^32."""
    s = torch.full_like(top, LEAST, dtype=F64)
    while True:
        more = (top > 448 * s) & (s < MOST)
        if not more.any():
            return s
        s = torch.where(more, 2 * s, s)


def norm8(x, weight, residual, eps):
    """codes (64 bits), scales, h of a norm; rows that are not finite have scale NaN and codes of zero."""
    h = x.to(F64)
    if residual is not None:
        h = (h + residual.to(F64)).to(torch.bfloat16).to(F64)
    t = h * weight.to(F64)
    top = t.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(h).all(-1, keepdim=True) | (h.square().sum(-1, keepdim=True) > 3.4e38) | (127 * top > 3.4e38)
    safe = torch.where((top > 0) & ~bad, top, 1.0)
    codes = torch.where(bad | (top == 0), 0.0, torch.round(127 * t / safe))
    scales = torch.where(bad, math.nan, top / 127 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps))
    return codes, scales[:, 0], h


class Cache:
    """A paged cache on the CPU with random content: values [pages][H][page][D] and scales [pages][H][page/16] in 64 bits
    (`tensors` lays them out), as fp4_util.Cache."""

    def __init__(self, g, lens, *, H, D, page, spare=2, poison=True, magnitude=1.0, spread=0.5):
        self.H, self.D, self.page, self.lens = H, D, page, list(lens)
        need = [-(-max(0, n) // page) for n in lens]
        self.width = max([1] + need) + 1
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g)
        self.table = torch.full((len(lens), self.width), -7, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n].int()
            at += n
        self.codes, self.scales = {}, {}
        live = torch.zeros((self.pages, page), dtype=torch.bool)
        for r, n in enumerate(self.lens):
            for j in range(max(0, n)):
                live[self.table[r, j // page], j % page] = True
        for k in "kv":
            x = torch.randn((self.pages, H, page // 16, 16, D), generator=g).to(F64) * magnitude
            x *= torch.exp(spread * torch.randn((self.pages, H, page // 16, 16, 1), generator=g).to(F64))
            s = block_scale(x.abs().amax((-2, -1)))
            c = codes_of(x / s[..., None, None]).view(self.pages, H, page, D)
            if poison:  # places that hold no token hold NaN, blocks without one NaN scales too
                c = torch.where(live[:, None, :, None], c, torch.tensor(0x7F, dtype=U8))
                s = torch.where(live.view(self.pages, 1, -1, 16).any(-1), s, math.nan)
            self.codes[k], self.scales[k] = c, s

    def tensors(self, dev):
        P, H, page, D = self.codes["k"].shape
        k = self.codes["k"].view(P, H, page // 16, 16, D // 16, 16).transpose(3, 4).contiguous()
        v = self.codes["v"].view(P, H, page // 16, 16, D).transpose(3, 4).contiguous()
        return [t.to(dev) for t in (k, self.scales["k"].float(), v, self.scales["v"].float())]

    def take(self, k_codes, k_scales, v_codes, v_scales):
        """What the tensors of a cache hold, as this cache's content."""
        P, H, page, D = self.codes["k"].shape
        self.codes = {"k": k_codes.cpu().view(U8).transpose(3, 4).reshape(P, H, page, D),
                      "v": v_codes.cpu().view(U8).transpose(3, 4).reshape(P, H, page, D)}
        self.scales = {"k": k_scales.cpu().to(F64), "v": v_scales.cpu().to(F64)}
        return self

    def place(self, r, j):
        p = int(self.table[r, j // self.page]) if 0 <= j < self.table.shape[1] * self.page else -1
        return (p, j % self.page) if 0 <= p < self.pages else None

    def rows(self, k, r, n):
        """[n][H][D] of request r in 64 bits; rows on pages that the table does not name are NaN-free zeros."""
        out = torch.zeros((n, self.H, self.D), dtype=F64)
        p = self.table[r, torch.arange(n) // self.page].long()
        ok = (p >= 0) & (p < self.pages)
        i = torch.arange(n)[ok] % self.page
        out[ok] = e4m3(self.codes[k][p[ok], :, i]) * self.scales[k][p[ok], :, i // 16][..., None]
        return out

    def most(self, k, r, n):
        """448 times the largest scale of request r's blocks, [H]."""
        out = torch.zeros(self.H, dtype=F64)
        for j in range(0, n, 16):
            at = self.place(r, j)
            if at:
                out = torch.maximum(out, 448 * self.scales[k][at[0], :, at[1] // 16])
        return out

    def named(self, r, n):
        p = self.table[r, torch.arange(n) // self.page]
        return (p >= 0) & (p < self.pages)

    def append(self, k, x, qsl, lens):
        """New tokens x [T][H][D] (64 bits): the blocks' scales, the earlier tokens' codes, the new ones' unrounded
        quotients [(page, place, [H][D])], as the header says."""
        got = []
        for r in range(len(lens)):
            a, b = int(qsl[r]), int(qsl[r + 1])
            blocks = {}
            for t in range(a, min(b, x.shape[0])):
                j = int(lens[r]) - (b - t)
                if j >= 0 and self.place(r, j):
                    blocks.setdefault(j // 16, []).append((j, t))
            for block, new in blocks.items():
                (page, place), first = self.place(r, new[0][0]), new[0][0] % 16
                base = place // 16 * 16
                fresh = x[[t for _, t in new]]
                size = torch.where(torch.isfinite(fresh), fresh.abs(), 0.0)
                s = block_scale(size.amax((0, 2)))
                if first:
                    old = self.scales[k][page, :, base // 16]
                    s = torch.maximum(s, old)
                    held = self.codes[k][page, :, base:base + first]
                    self.codes[k][page, :, base:base + first] = codes_of(e4m3(held) * (old / s)[:, None, None])
                self.scales[k][page, :, base // 16] = s
                for j, t in new:
                    q = (x[t] / s[:, None]).clamp(-448, 448)
                    got.append((page, base + j % 16, torch.where(torch.isfinite(x[t]), q, math.nan)))
        return got


def attention(cache, q, qsl, lens, window=0, scale=None):
    """out, lse and an error bound for each, in 64 bits.  The bound counts, with s the scores and w the softmax weights:
    fp32 sums of the scores and the way to their exponents (D + 8 roundings, 2^-23 each, of the sum of magnitudes; the
    values' scale, an exponent of at most 32, and its reciprocal: 2^-18); the weights' fp16 rounding (2^-11) and what fp16
    drops (2^-33 of the heaviest weight times its block's scale, against codes of at most 448); fp32 sums over the tokens;
    the output's bf16 rounding (2^-8)."""
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    G = Hq // cache.H
    out, lse = torch.zeros((T, Hq, D), dtype=F64), torch.full((T, Hq), -math.inf, dtype=F64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(len(lens)):
        a, b = int(qsl[r]), int(qsl[r + 1])
        n = max(0, min(int(lens[r]), cache.table.shape[1] * cache.page))
        if b == a or n == 0:
            continue
        k, v, named = cache.rows("k", r, n), cache.rows("v", r, n), cache.named(r, n)
        x = q[a:b].to(F64).view(b - a, cache.H, G, D).permute(1, 2, 0, 3).reshape(cache.H, G * (b - a), D)
        kt = k.permute(1, 2, 0).contiguous()
        s = (torch.bmm(x, kt) * scale).view(cache.H, G, b - a, n)
        mag = (torch.bmm(x.abs(), kt.abs()) * scale).view(cache.H, G, b - a, n)
        p = torch.arange(int(lens[r]) - (b - a), int(lens[r]))[:, None]
        j = torch.arange(n)[None, :]
        hide = (j > p) | ~named[None, :]
        if window:
            hide = hide | (j <= p - window)
        s = s.masked_fill(hide, -math.inf)
        ds = ((D + 8) * 2.0 ** -23 * mag).masked_fill(hide, 0).amax(-1)
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        w = torch.where(hide, 0.0, torch.exp(s - top))
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
        vv = v.transpose(0, 1).contiguous()
        mix = torch.bmm(w.reshape(cache.H, -1, n), vv).view(cache.H, G, b - a, D)
        size = torch.bmm(w.reshape(cache.H, -1, n), vv.abs()).view(cache.H, G, b - a, D)
        most = cache.most("v", r, n)[:, None, None, None]
        rel = (2.0 ** -11 + 2 * ds + 2.0 ** -18 + (n + 32) * 2.0 ** -23).unsqueeze(-1)
        t = 2.0 ** -8 * mix.abs() + 1.01 * (size * rel + n * 2.0 ** -33 * most)
        put = lambda y: y.permute(2, 0, 1, 3).reshape(b - a, Hq, -1)  # noqa: E731
        out[a:b], tol[a:b] = put(mix), put(t)
        L = (total.log() + top)
        lse[a:b] = put(L)[..., 0]
        tol_lse[a:b] = put((ds + 2.0 ** -18 + (n + 32) * 2.0 ** -23).unsqueeze(-1) + 2.0 ** -21 * L.abs().masked_fill(total == 0, 0))[..., 0]
    return out, lse, tol, tol_lse
