"""The 4-bit operators' definitions in 64 bits on the CPU, for the tests: formats, quantisation, products, rotation and
attention, written from include/ple_fp4.h with plain torch operations."""
from __future__ import annotations

import math

import torch

E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
F64 = torch.float64


def nibbles(codes):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()


def e2m1(codes):
    n = nibbles(codes)
    return torch.where(n >= 8, -1.0, 1.0).to(F64) * E2M1[n & 7]


def e4m3(b):
    n = b.to(F64)
    sign, e, m = torch.where(n >= 128, -1.0, 1.0).to(F64), (n % 128 / 8).floor(), n % 8
    v = sign * torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, e - 7))
    return torch.where(n % 128 == 127, torch.nan, v)


def pack(n):
    n = n.to(torch.uint8).unflatten(-1, (-1, 2))
    return n[..., 0] | n[..., 1] << 4


def quantise(x, g):
    """fp32 x [..., n] by blocks of 16 with fp32 scales g [..., 1]: codes [..., n/2], scales [..., n/16]."""
    b = x.unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = s.float() * g
    step = torch.where(step > 0, step, torch.inf).unsqueeze(-1)
    t = (b / step).flatten(-2)
    a = t.abs()
    near = torch.zeros_like(a)
    for lo, even in ((.25, True), (.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)):
        near += (a > lo) if even else (a >= lo)  # a tie goes to the even code
    return pack(near + 8 * torch.signbit(t)), s.view(torch.uint8)


def scale_layout(scales, page):
    """[P][H][page][D/16] -> the cache's [P][H][page/16][D/16][16]."""
    P, H, _, nb = scales.shape
    return scales.view(P, H, page // 16, 16, nb).transpose(-1, -2).contiguous()


class Cache:
    """A paged cache on the CPU with random content, and its rows in 64 bits."""

    def __init__(self, g, lens, *, H, D, page, spare=2, poison=True, magnitude=1.0):
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
        self.scale = {k: 0.02 + 0.01 * torch.rand(H, generator=g) for k in "kv"}
        self.codes, self.scales = {}, {}
        for k in "kv":
            x = torch.randn((self.pages, H, page, D), generator=g) * magnitude
            c, s = quantise(x, self.scale[k].view(1, H, 1, 1))
            if poison:  # places that hold no token hold NaN scales
                live = torch.zeros((self.pages, page), dtype=torch.bool)
                for r, n in enumerate(self.lens):
                    for j in range(max(0, n)):
                        live[self.table[r, j // page], j % page] = True
                s = torch.where(live[:, None, :, None], s, torch.tensor(0x7F, dtype=torch.uint8))
            self.codes[k], self.scales[k] = c, scale_layout(s, page)

    def tensors(self, dev):
        return [t.to(dev) for t in (self.codes["k"], self.scales["k"], self.codes["v"], self.scales["v"],
                                    self.scale["k"], self.scale["v"])]

    def rows(self, k, r, n):
        """[n][H][D] of request r in 64 bits; rows on pages that the table does not name are NaN-free zeros."""
        out = torch.zeros((n, self.H, self.D), dtype=F64)
        for j in range(n):
            p, i = int(self.table[r, j // self.page]), j % self.page
            if 0 <= p < self.pages:
                s = e4m3(self.scales[k][p, :, i // 16, :, i % 16]).repeat_interleave(16, -1)
                out[j] = e2m1(self.codes[k][p, :, i]) * s * self.scale[k].to(F64)[:, None]
        return out

    def named(self, r, n):
        p = self.table[r, torch.arange(n) // self.page]
        return (p >= 0) & (p < self.pages)


def attention(cache, q, qsl, lens, window=0, scale=None):
    """out, lse and an error bound for each, in 64 bits.  The bound counts: fp32 sums of the scores (D + 8 roundings,
    2^-23 each, of the sum of magnitudes), the weights' fp16 rounding (2^-11) and what fp16 drops (2^-33 of the
    heaviest), fp32 sums over the tokens, and the output's bf16 rounding (2^-8)."""
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    G = Hq // cache.H
    out, lse = torch.zeros((T, Hq, D), dtype=F64), torch.full((T, Hq), -math.inf, dtype=F64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(len(lens)):
        a, b = int(qsl[r]), int(qsl[r + 1])
        n = max(0, int(lens[r]))
        if b == a or n == 0:
            continue
        k, v, named = cache.rows("k", r, n), cache.rows("v", r, n), cache.named(r, n)
        x = q[a:b].to(F64).view(b - a, cache.H, G, D).permute(1, 2, 0, 3).reshape(cache.H, G * (b - a), D)
        kt = k.permute(1, 2, 0).contiguous()
        s = (torch.bmm(x, kt) * scale).view(cache.H, G, b - a, n)
        mag = (torch.bmm(x.abs(), kt.abs()) * scale).view(cache.H, G, b - a, n)
        p = torch.arange(n - (b - a), n)[:, None]
        j = torch.arange(n)[None, :]
        hide = (j > p) | ~named[None, :]
        if window:
            hide = hide | (j <= p - window)
        s = s.masked_fill(hide, -math.inf)
        ds = ((D + 8) * 2.0 ** -23 * mag).masked_fill(hide, 0).amax(-1)
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        w = torch.exp(s - top)
        w = torch.where(hide, 0.0, w)
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
        vv = v.transpose(0, 1).contiguous()
        mix = torch.bmm(w.reshape(cache.H, -1, n), vv).view(cache.H, G, b - a, D)
        size = torch.bmm(w.reshape(cache.H, -1, n), vv.abs()).view(cache.H, G, b - a, D)
        most = vv.abs().amax(1)[:, None, None, :]
        rel = (2.0 ** -11 + 2 * ds + (n + 32) * 2.0 ** -23).unsqueeze(-1)
        t = 2.0 ** -8 * mix.abs() + 1.01 * (size * rel + n * 2.0 ** -33 * most)
        put = lambda y: y.permute(2, 0, 1, 3).reshape(b - a, Hq, -1)  # noqa: E731
        out[a:b], tol[a:b] = put(mix), put(t)
        L = (total.log() + top)
        lse[a:b] = put(L)[..., 0]
        tol_lse[a:b] = put((ds + (n + 32) * 2.0 ** -23).unsqueeze(-1) + 2.0 ** -21 * L.abs().masked_fill(total == 0, 0))[..., 0]
    return out, lse, tol, tol_lse


def rotate(x, pos, inv_freq, interleaved):
    """[T][H][D] bf16 turned by position * inv_freq, in 64 bits."""
    rot = 2 * len(inv_freq)
    x = x.to(F64).clone()
    angle = (pos.to(F64)[:, None] * inv_freq.to(F64)[None, :])[:, None, :]
    c, s = angle.cos(), angle.sin()
    i = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., i[0]].clone(), x[..., i[1]].clone()
    x[..., i[0]], x[..., i[1]] = a * c - b * s, b * c + a * s
    return x
