"""The 8-bit decode operators where values lie at the ends of their types or far apart, against the definitions in 64 bits
(bits8_util)."""
import math

import pytest
import torch

import bits8_util as U
import layer_embedding_lookup_amd as ple
import test_bits8_gpu as G
import test_bits8_kernels as K

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F64, BF, I32 = torch.float64, torch.bfloat16, torch.int32


# ---- norm ----

# powers of two that inputs and weights are of: products from fp32's normal numbers down past its least one
TINY = [(-50, -40), (-50, -52), (-64, -62), (-64, -64), (-66, -64), (-70, -62), (-120, -12), (-20, -112), (-100, -60), (-120, -100),
        (-126, -126), (-131, 0), (0, -131), (-131, 100), (60, -131)]


def check_tiny(x, w, res, eps, got):
    """As G.check_norm, but for the scales, which fp32 rounds by up to half of its least step, 2^-150, where they are below
    its normal numbers."""
    codes, scales, h = got
    want, want_scales, want_h = U.norm8(x, w, res, eps)
    assert torch.equal(codes.cpu().to(F64), want)
    bad = torch.isnan(want_scales)                            # (rows whose squares leave fp32's range)
    assert torch.equal(torch.isnan(scales.cpu()), bad)
    assert ((scales.cpu().to(F64) - want_scales).abs() <= 60 * 2.0 ** -24 * want_scales + 2.0 ** -149)[~bad].all()
    if res is not None:
        assert torch.equal(h.cpu().to(F64), want_h)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("N", [16, 512, 2064, 4096, 8208, 20000])
def test_norm_rows_whose_products_underflow(N, residual):
    """Every row has the codes of its exact quotients, however small its products, beside rows of ordinary size."""
    for a, b in TINY:
        g = G.gen(N + a - b)
        x = torch.randn((6, N), generator=g).double() * 2.0 ** a
        x[1] = torch.randn(N, generator=g)                    # an ordinary row, if the weight is not tiny
        x[4] = 0
        x[5] *= torch.pow(2.0, torch.randint(-4, 5, (N,), generator=g).double())
        x = x.to(BF)
        w = (torch.randn(N, generator=g).double() * 2.0 ** b).to(BF)
        res = (torch.randn((6, N), generator=g).double() * 2.0 ** (a - 1)).to(BF) if residual else None
        if residual:
            res[4] = 0
        got = ple.ple_rms_norm8(x.to(DEV), w.to(DEV), residual=None if res is None else res.to(DEV))
        check_tiny(x, w, res, 1e-6, got)
        assert (got[0][4] == 0).all() and got[1][4] == 0
        assert got[0].abs().amax(1).tolist() == [0 if s != s or s == 0 else 127 for s in U.norm8(x, w, res, 1e-6)[1].tolist()]


def test_norm_tiny_rows_in_place_and_strided():
    for N in (48, 4096, 20000):
        g = G.gen(N)
        wide = torch.full((5, N + 16), math.nan).to(BF)
        wide[:, 8:N + 8] = (torch.randn((5, N), generator=g).double() * 2.0 ** -70).to(BF)
        x, w = wide[:, 8:N + 8], (torch.randn(N, generator=g).double() * 2.0 ** -62).to(BF)
        check_tiny(x, w, None, 1e-6, ple.ple_rms_norm8(wide.to(DEV)[:, 8:N + 8], w.to(DEV)))
        x = x.contiguous()
        res = (torch.randn((5, N), generator=g).double() * 2.0 ** -70).to(BF)
        for into in ("x", "residual"):
            dx, dres = x.to(DEV), res.to(DEV)
            got = ple.ple_rms_norm8(dx, w.to(DEV), residual=dres, residual_out=dx if into == "x" else dres)
            check_tiny(x, w, res, 1e-6, got)


@pytest.mark.parametrize("N", [16, 512, 2064, 4096, 8208, 20000])
def test_norm_weights_of_no_number(N):
    """A NaN or an infinity in the weight is in every row's products, as 0 * infinity too: scales of NaN, codes of zero, the
    residual as ever."""
    g = G.gen(N)
    x, res = torch.randn((5, N), generator=g).to(BF), torch.randn((5, N), generator=g).to(BF)
    x[3] = res[3] = 0
    for at in (0, 7, N // 2, N - 1):
        x[1, at] = res[1, at] = 0
        for value in (math.nan, -math.nan, math.inf, -math.inf):
            w = torch.randn(N, generator=g).to(BF)
            w[at] = value
            for r in (None, res):
                codes, scales, h = ple.ple_rms_norm8(x.to(DEV), w.to(DEV), residual=None if r is None else r.to(DEV))
                assert torch.isnan(scales).all() and (codes == 0).all()
                assert r is None or torch.equal(h.cpu(), (x.float() + r.float()).to(BF))


@pytest.mark.parametrize("N", [48, 4096, 20000])
def test_norm_scales_whose_products_overflow(N):
    """A largest product below fp32's 127th part, times a norm's factor far above 127: the scale itself is in range."""
    g = G.gen(N)
    x = (torch.randn((4, N), generator=g).clamp(-4, 4).double() * 2.0 ** -9).to(BF)
    x[:, 3] = 2.0 ** -7
    w = (torch.rand(N, generator=g).double() * 2.0 ** 126).to(BF)
    w[3] = 2.0 ** 127
    top = (x.double() * w.double()).abs().amax(1)
    factor = 1 / (x.double().square().mean(1) + 1e-6).sqrt()
    assert (127 * top < 3.4e38).all() and (top * factor > 3.5e38).all()
    got = ple.ple_rms_norm8(x.to(DEV), w.to(DEV))
    G.check_norm(x, w, None, 1e-6, got)
    assert torch.isfinite(got[1]).all()


# ---- attention ----

def far_cache(c):
    """A case's cache in which some blocks of each head have values 2^10 .. 2^50 times the others', and zeros in the first half
    of their elements: there only the light blocks count."""
    cache, q, qsl, seq = K.attention_inputs(c)
    g = G.gen(sum(c.lens))
    heavy = torch.rand(cache.scales["v"].shape, generator=g) < 0.2
    for r in range(len(c.lens)):                              # (the first block and the last whole one too)
        for j in (0, (c.lens[r] - 1) // 16 * 16):
            at = cache.place(r, j)
            if c.lens[r] and at:
                heavy[at[0], 0, at[1] // 16] = True
    by = torch.pow(2.0, torch.randint(10, 41, heavy.shape, generator=g).to(F64))
    cache.scales["v"] = torch.where(heavy, cache.scales["v"] * by, cache.scales["v"] * 2.0 ** -10).clamp(U.LEAST, U.MOST)
    codes = cache.codes["v"]
    gone = heavy.repeat_interleave(16, 2)[..., None] & (torch.arange(c.D) < c.D // 2)
    cache.codes["v"] = torch.where(gone & (codes & 0x7F != 0x7F), torch.zeros_like(codes), codes)
    return cache, q, qsl, seq


def far_bound(cache, q, qsl, seq, window):
    """out, lse and bounds as U.attention gives them, but each token's part of an element for itself: a weight is rounded by
    2^-11 of itself, or, where it is less than 2^-14 of what fp16 has at a time, by 2^-25 of the heaviest (of 2^8 at least)
    over the scales' ratio, 2^6 at most: 2^-27 of the token's own value."""
    class Near(U.Cache):
        def most(self, k, r, n):
            return torch.zeros(self.H, dtype=F64)
    near, size = Near.__new__(Near), U.Cache.__new__(U.Cache)
    near.__dict__.update(cache.__dict__)
    size.__dict__.update(cache.__dict__)
    size.codes = {"k": cache.codes["k"], "v": cache.codes["v"] & 0x7F}
    want, lse, tol, tol_lse = U.attention(near, q, qsl, seq, window)
    mean = U.attention(size, torch.zeros_like(q), qsl, seq, window)[0]       # of the sizes of the values that a row sees
    tokens = torch.zeros(q.shape[0], dtype=F64)
    for r in range(len(seq)):
        tokens[int(qsl[r]):int(qsl[r + 1])] = max(0, int(seq[r]))
    return want, lse, tol + 1.01 * 2.0 ** -27 * tokens[:, None, None] * mean, tol_lse


@pytest.mark.parametrize("c", K.ATTENTION, ids=repr)
def test_attention_light_blocks_beside_heavy_ones(c):
    """Blocks whose values are 2^20 times those of others and more, by every kernel: what the light ones add to elements that
    the heavy ones have zeros in comes out as the definition says."""
    print(f"kv8 attention, blocks far apart: {c}", flush=True)
    cache, q, qsl, seq = far_cache(c)
    out, lse = G.run_attention(cache, q, qsl, seq, window=c.window, **K.hints(c))
    want, want_lse, tol, tol_lse = far_bound(cache, q, qsl, seq, c.window)
    assert ((out - want).abs() <= tol).all(), float(((out - want).abs() - tol).max())
    empty = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, empty) and (out[empty] == 0).all()
    assert ((lse - want_lse).abs() <= tol_lse)[~empty].all()


@pytest.mark.parametrize("c", K.ATTENTION, ids=repr)
def test_attention_nan_beside_blocks_far_apart(c):
    """A NaN element of one value there: that element of the rows that see it, nothing else."""
    print(f"kv8 attention, a NaN beside blocks far apart: {c}", flush=True)
    cache, q, qsl, seq = far_cache(c)
    clean, clean_lse = G.run_attention(cache, q, qsl, seq, window=c.window, **K.hints(c))
    r = c.lens.index(max(c.lens))
    before = c.lens[r] - c.news[r]
    first = 0 if c.window == 0 else max(0, c.lens[r] - c.window)
    j = next(j for j in range((first + before) // 2, before + 1) if 0 <= int(cache.table[r, j // c.page]))
    head, d = c.H - 1, 5
    cache.codes["v"][int(cache.table[r, j // c.page]), head, j % c.page, d] = 0x7F
    out, lse = G.run_attention(cache, q, qsl, seq, window=c.window, **K.hints(c))
    mine = torch.zeros(out.shape, dtype=torch.bool)
    p = before + torch.arange(c.news[r])
    sees = (p >= j) & (p - c.window < j if c.window else True)
    mine[int(qsl[r]):int(qsl[r + 1]), head * (c.Hq // c.H):, d] = sees[:, None]
    assert mine.any() and torch.isnan(out[mine]).all()
    assert torch.equal(out[~mine], clean[~mine]) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("D,news", [(64, [1, 1]), (128, [3, 1]), (256, [1, 2]), (64, [90, 3]), (128, [90, 3]), (256, [40, 3])])
def test_attention_scale_beyond_the_products_range(D, news):
    """The largest `scale` of the call over keys of the largest scale, whose product fp32 does not hold: rows of zeros still
    see every token alike."""
    g = G.gen(D + news[0])
    lens = [200, 90]
    cache = U.Cache(g, lens, H=2, D=D, page=16)
    cache.scales["k"] = torch.where(torch.isnan(cache.scales["k"]), math.nan, 2.0 ** 32)
    qsl, seq = G.batch(news, lens)
    q = torch.zeros((int(qsl[-1]), 4, D), dtype=BF)
    G.check_attention(cache, q, qsl, seq, scale=1e30, max_request_tokens=max(news), max_seq_len=max(lens))


# ---- append ----

def fp4_cache():
    codes = [torch.zeros((3, 2, 16, 64), dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros((3, 2, 1, 8, 16), dtype=torch.uint8, device=DEV) for _ in range(2)]
    return ple.KV4Cache(codes[0], scales[0], codes[1], scales[1], *(torch.ones(2, device=DEV) for _ in range(2)))


def bits8_cache():
    codes = [torch.zeros(s, dtype=torch.uint8, device=DEV) for s in ((3, 2, 1, 8, 16, 16), (3, 2, 1, 128, 16))]
    return ple.KV8Cache(codes[0], torch.ones((3, 2, 1), device=DEV), codes[1], torch.ones((3, 2, 1), device=DEV))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("append,make", [(ple.ple_kv8_append, bits8_cache), (ple.ple_kv4_append, fp4_cache)], ids=["kv8", "kv4"])
def test_queries_of_no_request_keep_what_they_hold(append, make, interleaved):
    """A padded batch's rows may hold anything, infinities and NaN too: an element of such a row does not reach the one it
    would be turned with, and zeros keep their sign."""
    g = G.gen(3)
    q, k = (torch.randn((9, h, 128), generator=g).to(BF) for h in (4, 2))
    idle = [0, 1, 5, 6, 7, 8]                                 # requests have tokens 2 .. 4
    q[0, :, 3], q[1, 1, 70], q[5, 2, ::7], q[6], q[7, 0, 1::2], q[8, :, :64] = math.inf, math.nan, -math.inf, math.nan, -0.0, -0.0
    args = [torch.tensor(x, dtype=I32, device=DEV) for x in ([2, 3, 5], [4, 7], [[0], [1]])]
    inv = torch.logspace(0, -4, 64).to(DEV)
    out = append(make(), k.to(DEV), k.to(DEV), *args, inv_freq=inv, interleaved=interleaved, q=q.to(DEV)).cpu()
    nan = torch.isnan(q[idle])
    assert torch.equal(torch.isnan(out[idle]), nan)
    assert torch.equal(out[idle].view(torch.int16)[~nan], q[idle].view(torch.int16)[~nan])
    own = append(make(), k[2:5].to(DEV), k[2:5].to(DEV), args[0] - 2, *args[1:], inv_freq=inv, interleaved=interleaved, q=q[2:5].to(DEV))
    assert torch.equal(out[2:5], own.cpu())


@pytest.mark.parametrize("hint,most", [(False, 24), (True, 24), (True, 18), (True, 2)])
def test_append_and_read_of_more_than_1024_requests(hint, most):
    """Past 1024 requests a unit's request is found by halving: ragged ones, some without new tokens, some over a block's end.
    A hint of fewer tokens than 18 numbers the units by it instead."""
    g = G.gen(8)
    R = 1300
    news = torch.where(torch.rand(R, generator=g) < 0.3, 0, torch.randint(1, most, (R,), generator=g))
    lens = news + torch.randint(0, 40, (R,), generator=g)
    lens[5::200] = news[5::200]
    G.test_append_and_read(64, 2, 1, 16, news.tolist(), lens.tolist(), 32, False, hint)
