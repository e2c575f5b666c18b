"""The 8-bit decode operators on the GPU against their definitions in 64 bits (bits8_util)."""
import math

import pytest
import torch

import bits8_util as U
import layer_embedding_lookup_amd as ple

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F64, BF, I8, I32 = torch.float64, torch.bfloat16, torch.int8, torch.int32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def say(*a):
    print(*a, flush=True)


# ---- norm ----

def check_norm(x, w, res, eps, got):
    codes, scales, h = got
    want, want_scales, want_h = U.norm8(x, w, res, eps)
    # the quotient that is rounded is exact but for half a step that never reaches a border, so codes are equal; scales:
    # a sum of N squares in chains of at most 64 and a tree (half of its relative error), and five roundings
    assert torch.equal(codes.cpu().to(F64), want)
    bad = torch.isnan(want_scales)
    assert torch.equal(torch.isnan(scales.cpu()), bad)
    d = (scales.cpu().to(F64) - want_scales).abs()[~bad]
    assert (d <= 60 * 2.0 ** -24 * want_scales[~bad]).all()
    assert (h is None) == (res is None)
    if h is not None:
        assert torch.equal(h.cpu().to(F64)[~bad], want_h[~bad])


@pytest.mark.parametrize("T,N", [(1, 16), (1, 4096), (3, 256), (5, 512), (9, 528), (4, 2048), (7, 2064), (300, 4096), (2, 4112),
                                 (3, 8192), (2, 8208), (3, 16384), (2, 16400), (2, 131056), (4099, 48)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(T, N, residual):
    say(f"norm T={T} N={N} residual={residual}")
    g = gen(T + N)
    x, w = torch.randn((T, N), generator=g).to(BF), torch.randn(N, generator=g).to(BF)
    res = (torch.randn((T, N), generator=g) * torch.exp(2 * torch.randn((T, 1), generator=g))).to(BF) if residual else None
    got = ple.ple_rms_norm8(x.to(DEV), w.to(DEV), residual=None if res is None else res.to(DEV), eps=1e-5)
    check_norm(x, w, res, 1e-5, got)


@pytest.mark.parametrize("N", [48, 4096, 8192, 20000])
def test_norm_strided_rows_and_in_place(N):
    g = gen(N)
    T = 5
    wide = torch.full((T + 2, N + 88), math.nan, dtype=BF)
    wide[1:-1, 8:N + 8] = torch.randn((T, N), generator=g).to(BF)
    x, w = wide[1:-1, 8:N + 8], torch.randn(N, generator=g).to(BF)
    res = torch.randn((T, N), generator=g).to(BF)
    dx, dres = wide.to(DEV)[1:-1, 8:N + 8], res.to(DEV)
    around = torch.full((T + 2, N), 7, dtype=I8, device=DEV)
    scales = torch.full((T + 2,), 7.0, device=DEV)
    got = ple.ple_rms_norm8(dx, w.to(DEV), residual=dres, residual_out=dres, codes=around[1:-1], scales=scales[1:-1])
    assert got[2].data_ptr() == dres.data_ptr()
    check_norm(x, w, res, 1e-6, got)
    assert (around[0] == 7).all() and (around[-1] == 7).all() and scales[0] == 7 and scales[-1] == 7
    # residual_out may be x
    x, dres = x.contiguous(), res.to(DEV)
    dx = x.to(DEV)
    check_norm(x, w, res, 1e-6, ple.ple_rms_norm8(dx, w.to(DEV), residual=dres, residual_out=dx))
    assert torch.equal(dres.cpu(), res)


def test_norm_ties_and_borders():
    """127 u / a on borders (ties go to the even code) and one step of bf16 beside them."""
    row = torch.zeros(512, dtype=F64)
    for i in range(127):
        row[i] = i + 0.5                                    # of a largest value of 127
    row = row.to(BF)
    up, down = (row.view(torch.int16) + s for s in (1, -1))
    top = torch.tensor([127.0] + [0.0] * 255).to(BF)
    x = torch.cat((row[:256], top)).repeat(3, 1)
    x[1, :127], x[2, :127] = up.view(BF)[:127], down.view(BF)[:127]
    x = torch.cat((x, -x, x * 2.0 ** -40, x * 2.0 ** 30))
    for w in (torch.ones(512), torch.full((512,), -3.0)):
        got = ple.ple_rms_norm8(x.to(DEV), w.to(BF).to(DEV))
        check_norm(x, w.to(BF), None, 1e-6, got)
    assert got[0].abs().max() == 127


def test_norm_rows_of_nothing_and_of_no_number():
    """Zeros give zeros, an infinity, a NaN or a sum beyond fp32 a NaN scale; the other rows are as without them."""
    for N in (256, 4096, 20000):
        g = gen(N)
        x = torch.randn((8, N), generator=g).to(BF)
        x[1] = 0
        x[2, N - 1], x[3, 0], x[4, 5], x[5, 7] = math.inf, math.nan, -math.inf, 3e38
        x[6] *= 1e-30
        w = torch.randn(N, generator=g).to(BF)
        got = ple.ple_rms_norm8(x.to(DEV), w.to(DEV))
        check_norm(x, w, None, 1e-6, got)
        assert (got[0][1] == 0).all() and got[1][1] == 0 and torch.isnan(got[1][2:6]).all()
        # an infinity that the sum makes
        check_norm(x, w, -x, 1e-6, ple.ple_rms_norm8(x.to(DEV), w.to(DEV), residual=(-x).to(DEV)))


def test_norm_no_tokens():
    codes, scales, h = ple.ple_rms_norm8(torch.zeros((0, 64), dtype=BF, device=DEV), torch.ones(64, dtype=BF, device=DEV))
    assert codes.shape == (0, 64) and scales.shape == (0,) and h is None


# ---- products of 8-bit integers ----

def check_linear(x, xs, w, ws, out):
    """Sums are exact; the fp32 of a sum, two products (2^-24 each, 2^-22 in all) and bf16's 2^-8."""
    want = (x.to(F64) @ w.to(F64).t()) * ws.to(F64) * xs.to(F64)[:, None]
    assert ((out.cpu().to(F64) - want).abs() <= (2.0 ** -8 + 2.0 ** -21) * want.abs()).all()


def random_codes(g, shape):
    return torch.randint(-128, 128, shape, generator=g).to(I8)


def scales_of(g, n):
    return torch.exp(3 * torch.randn(n, generator=g))


# every kernel; K in whole steps and slices, ending inside one, of one piece, and of more slices than are on their way at once
LINEAR_T_O = [(1, 1), (1, 300), (5, 17), (16, 48), (17, 333), (32, 100), (33, 70), (37, 5003), (64, 1000), (65, 100), (1, 6500), (100, 4200),
              (130, 8100), (600, 333), (700, 5003), (2051, 4099), (4100, 4104)]
LINEAR_K = [16, 112, 128, 144, 384, 1040]


@pytest.mark.parametrize("K", LINEAR_K)
@pytest.mark.parametrize("T,O", LINEAR_T_O)
def test_linear(T, O, K):
    say(f"w8 linear T={T} O={O} K={K}")
    g = gen(T + O + K)
    x, w = random_codes(g, (T, K)), random_codes(g, (O + 9, K))
    xs, ws = scales_of(g, T), scales_of(g, O + 9)
    wide = random_codes(g, (T + 5, K + 80))               # rows of x out of a wider tensor
    wide[2:T + 2, 32:K + 32] = x
    around = torch.full((T + 16, O), 7, dtype=BF, device=DEV)
    out = around[8:T + 8]                                  # (8 rows: 16-byte aligned for any O)
    ple.ple_w8_linear(wide.to(DEV)[2:T + 2, 32:K + 32], xs.to(DEV), ple.W8Weight(w.to(DEV)[:O], ws.to(DEV)[:O]), out=out)
    check_linear(x, xs, w[:O], ws[:O], out)
    assert (around[:8] == 7).all() and (around[T + 8:] == 7).all()


@pytest.mark.parametrize("T", [1, 40, 100, 300])
def test_linear_long_rows_at_the_ends_of_their_type(T):
    """131056 products of -128 and -128: the largest sum that the call allows."""
    K, O = 131056, 200
    x, w = torch.full((T, K), -128, dtype=I8), torch.full((O, K), -128, dtype=I8)
    w[::3] = 127
    xs, ws = torch.ones(T), torch.ones(O)
    out = ple.ple_w8_linear(x.to(DEV), xs.to(DEV), ple.W8Weight(w.to(DEV), ws.to(DEV)))
    want = torch.tensor([-128.0 * (127 if o % 3 == 0 else -128) * K for o in range(O)]).to(BF)
    assert torch.equal(out.cpu(), want.expand(T, O))


@pytest.mark.parametrize("T", [4, 80, 300])
def test_linear_scales_of_no_number_stay_apart(T):
    g = gen(T)
    x, w, xs, ws = random_codes(g, (T, 272)), random_codes(g, (130, 272)), scales_of(g, T), scales_of(g, 130)
    xs[1], xs[T - 1], ws[5], ws[7] = math.nan, 0.0, math.nan, 0.0
    out = ple.ple_w8_linear(x.to(DEV), xs.to(DEV), ple.W8Weight(w.to(DEV), ws.to(DEV))).cpu()
    assert torch.isnan(out[1]).all() and torch.isnan(out[:, 5]).all()
    keep, cols = [t for t in range(T) if t != 1], [o for o in range(130) if o != 5]
    check_linear(x[keep], xs[keep], w[cols], ws[cols], out[keep][:, cols])


def test_linear_no_tokens():
    w = ple.W8Weight(torch.zeros((70, 64), dtype=I8, device=DEV), torch.ones(70, device=DEV))
    assert ple.ple_w8_linear(torch.zeros((0, 64), dtype=I8, device=DEV), torch.zeros(0, device=DEV), w).shape == (0, 70)


# ---- append and read ----

def batch(news, lens):
    return torch.tensor([0] + list(news)).cumsum(0).int(), torch.tensor(lens, dtype=I32)


def positions(qsl, lens):
    return torch.cat([torch.arange(int(n) - int(b - a), int(n)) for a, b, n in zip(qsl[:-1], qsl[1:], lens)])


def check_append(cache, before, got, tensors):
    """The cache after an append: scales and earlier tokens exactly, each new code the nearest one of its quotient (within
    2^-22 of the quotient, which the rotation's rounding to fp32 can move), everything else as it was."""
    after = U.Cache.__new__(U.Cache)
    after.__dict__.update(cache.__dict__)
    after.take(*tensors)
    for k in "kv":
        new = torch.zeros(before[k].shape[:3], dtype=torch.bool)
        held = U.e4m3(after.codes[k])
        for page, place, q in got[k]:
            new[page, :, place] = True
            x = held[page, :, place]
            assert torch.equal(torch.isnan(x), torch.isnan(q)), (k, page, place)
            _, e = torch.frexp(q)
            step = torch.pow(2.0, (e - 1).clamp(min=-6).to(F64) - 3)
            ok = ((x - q).abs() <= step / 2 + 2.0 ** -22 * q.abs()) | torch.isnan(q)
            assert ok.all(), (k, page, place, float((x - q).abs().max()))
        assert torch.equal(torch.where(new[..., None], 0, after.codes[k]), torch.where(new[..., None], 0, cache.codes[k])), k
        assert torch.equal(torch.nan_to_num(after.scales[k], 7.0), torch.nan_to_num(cache.scales[k], 7.0)), k
    return after


APPEND = [  # D, Hq, H, page, new tokens, lengths, rot, interleaved
    (64, 2, 1, 16, [1], [1], 64, False), (128, 8, 2, 16, [1, 1, 1], [17, 16, 100], 128, False),
    (128, 4, 4, 48, [40, 3, 0, 20], [40, 60, 9, 83], 64, True), (256, 2, 2, 32, [33, 17], [70, 17], 256, False),
    (64, 6, 3, 64, [15, 16, 17, 1], [31, 48, 33, 64], 32, True), (128, 5, 5, 16, [200], [431], 112, False),
    (64, 3, 1, 80, [2, 5, 8], [90, 5, 24], 16, False), (256, 4, 1, 16, [1, 4, 2], [300, 8, 18], 64, True),
    (128, 3, 3, 112, [100], [100], 0, False), (128, 1, 1, 16, [1] * 70, list(range(1, 71)), 128, True),
]


@pytest.mark.parametrize("hint", [False, True])
@pytest.mark.parametrize("D,Hq,H,page,news,lens,rot,interleaved", APPEND)
def test_append_and_read(D, Hq, H, page, news, lens, rot, interleaved, hint):
    say(f"append D={D} H={H} page={page} new={news[:5]} rot={rot} hint={hint}")
    g = gen(D + H + sum(lens))
    cache = U.Cache(g, [n - m for n, m in zip(lens, news)], H=H, D=D, page=page)
    # (pages for the new tokens too)
    need = [-(-n // page) for n in lens]
    whole = U.Cache(g, lens, H=H, D=D, page=page)
    filled = U.Cache.__new__(U.Cache)
    filled.__dict__.update(whole.__dict__)
    filled.codes, filled.scales = {k: whole.codes[k].clone() for k in "kv"}, {k: whole.scales[k].clone() for k in "kv"}
    for r, (n, m) in enumerate(zip(lens, news)):            # what the new tokens' places hold is anything
        for j in range(n - m, n):
            p, i = whole.place(r, j)
            for k in "kv":
                filled.codes[k][p, :, i] = 0x7F
                if j % 16 == 0:
                    filled.scales[k][p, :, i // 16] = math.nan
    del cache, need
    qsl, seq = batch(news, lens)
    T = int(qsl[-1])
    wide = (torch.randn((T, (Hq + 2 * H) * D), generator=g) * torch.exp(torch.randn((T, 1), generator=g))).to(BF)
    parts = lambda t: [v.unflatten(-1, (-1, D)) for v in (t[:, :Hq * D], t[:, Hq * D:(Hq + H) * D], t[:, (Hq + H) * D:])]  # noqa: E731
    q, k, v = parts(wide)
    inv = (1e4 ** (-torch.arange(0, rot, 2, dtype=F64) / max(rot, 1))).float()
    tensors = filled.tensors(DEV)
    c = ple.KV8Cache(*tensors)
    dq, dk, dv = parts(wide.to(DEV))
    where = (qsl.to(DEV), seq.to(DEV), whole.table.to(DEV))
    out = ple.ple_kv8_append(c, dk, dv, *where, inv_freq=inv.to(DEV) if rot else None, interleaved=interleaved, q=dq,
                             max_request_tokens=max(news) if hint else 0)
    pos = positions(qsl, lens)
    turned = U.rotate(k, pos, inv, interleaved)
    before = {n: filled.codes[n].clone() for n in "kv"}
    got = {"k": filled.append("k", turned, qsl, lens), "v": filled.append("v", v.to(F64), qsl, lens)}
    after = check_append(filled, before, got, tensors)
    want = U.rotate(q, pos, inv, interleaved)
    assert ((out.cpu().to(F64) - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -22 * q.abs().max()).all()
    rk, rv = ple.ple_kv8_read(c, *where, T)
    for n, x in (("k", rk), ("v", rv)):
        rows = torch.cat([after.rows(n, r, lens[r])[lens[r] - news[r]:] for r in range(len(lens))])
        assert torch.equal(x.cpu(), rows.float().to(BF))


def test_append_token_by_token():
    """Sixteen calls of one token each, ever larger and smaller: the block's scale only grows, and what it holds is within
    half a step of its type, at the scale of the time or later ones', of what came in."""
    g = gen(5)
    H, D, page, n = 2, 128, 16, 40
    whole = U.Cache(g, [n], H=H, D=D, page=page)
    tensors = whole.tensors(DEV)
    c = ple.KV8Cache(*tensors)
    x = torch.randn((n, H, D), generator=g) * torch.exp(2 * torch.randn((n, 1, 1), generator=g))
    x[20] = 0
    x = x.to(BF)
    table = whole.table.to(DEV)
    one = torch.tensor([0, 1], dtype=I32, device=DEV)
    for t in range(n):
        seq = torch.tensor([t + 1], dtype=I32, device=DEV)
        ple.ple_kv8_append(c, x[t:t + 1].to(DEV), x[t:t + 1].to(DEV), one, seq, table)
        for k in "kv":
            whole.append(k, x[t:t + 1].to(F64), [0, 1], [t + 1])
    ref = {k: (whole.codes[k].clone(), whole.scales[k].clone()) for k in "kv"}
    whole.take(*tensors)
    for k in "kv":
        rows = whole.rows(k, 0, n)
        scale = torch.stack([whole.scales[k][whole.place(0, t)[0], :, 0] for t in range(n)])
        assert torch.equal(whole.scales[k], ref[k][1]) or torch.equal(torch.nan_to_num(whole.scales[k], 1.0), torch.nan_to_num(ref[k][1], 1.0))
        # normal values keep their three bits through powers of two; small ones are within half of the last scale's 2^-9
        # for each of at most 16 growths
        err = (rows - x.to(F64)).abs()
        assert (err <= 2.0 ** -4 * x.to(F64).abs() + 16 * 2.0 ** -10 * scale[..., None]).all()


def test_append_range_and_no_numbers():
    """Largest magnitudes at 448 * 2^k and one bf16 step beside it, at both ends of the scales' range; infinities and NaN."""
    H, D, page = 1, 64, 16
    tops = [448.0, 450.0, 446.0, 448.0 * 2.0 ** 32, 450.0 * 2.0 ** 32, 3e38, 448.0 * 2.0 ** -32, 2.0 ** -40, 2.0 ** -60, 1e-40, 0.0, 7.0]
    news = [3] * len(tops)
    cache = U.Cache(gen(3), news, H=H, D=D, page=page)
    x = torch.randn((3 * len(tops), H, D), generator=gen(4)).clamp(-1, 1).to(F64)
    for r, top in enumerate(tops):
        x[3 * r:3 * r + 3] *= top
        x[3 * r + 1, 0, 5] = -top
    x = x.to(BF)
    x[33, 0, 3], x[34, 0, 4], x[35, 0, 5] = math.inf, -math.inf, math.nan
    qsl, seq = batch(news, news)
    tensors = cache.tensors(DEV)
    c = ple.KV8Cache(*tensors)
    ple.ple_kv8_append(c, x.to(DEV), x.to(DEV), qsl.to(DEV), seq.to(DEV), cache.table.to(DEV))
    before = {n: cache.codes[n].clone() for n in "kv"}
    got = {n: cache.append(n, x.to(F64), qsl, news) for n in "kv"}
    after = check_append(cache, before, got, tensors)
    scales = [float(after.scales["k"][after.place(r, 0)[0], 0, 0]) for r in range(len(tops))]
    assert scales == [1.0, 2.0, 1.0, 2.0 ** 32, 2.0 ** 32, 2.0 ** 32, 2.0 ** -32, 2.0 ** -32, 2.0 ** -32, 2.0 ** -32, 2.0 ** -32, 2.0 ** -6]


def test_append_ties_go_to_the_even_code():
    """Every midpoint between neighbouring codes, and one step of bf16 beside it."""
    grid = U.e4m3(torch.arange(0x7F, dtype=torch.uint8))
    mid = (grid[1:] + grid[:-1]) / 2                        # exact in bf16: at most 5 significant bits
    x = torch.zeros((16, 1, 64), dtype=F64)
    x.view(-1)[:126] = mid
    x = x.to(BF)
    x.view(-1)[126:252] = (mid.to(BF).view(torch.int16) + 1).view(BF)
    x.view(-1)[252:378] = (mid.to(BF).view(torch.int16) - 1).view(BF)
    x.view(-1)[400:526] = -mid.to(BF)
    x.view(-1)[600] = 448.0
    cache = U.Cache(gen(1), [16], H=1, D=64, page=16)
    tensors = cache.tensors(DEV)
    ple.ple_kv8_append(ple.KV8Cache(*tensors), x.to(DEV), x.to(DEV), *(t.to(DEV) for t in batch([16], [16])), cache.table.to(DEV))
    after = cache.take(*tensors)
    want = U.codes_of(x.to(F64).view(16, 1, 64))
    for k in "kv":
        assert torch.equal(after.codes[k][after.place(0, 0)[0], 0], want[:, 0])
        assert after.scales[k][after.place(0, 0)[0], 0, 0] == 1.0


def test_append_bad_pages_and_places_write_nothing():
    g = gen(6)
    cache = U.Cache(g, [50, 20], H=2, D=128, page=16)
    cache.table[0, 1], cache.table[1, 0] = -1, cache.pages
    tensors = cache.tensors(DEV)
    before = [t.clone() for t in tensors]
    k = torch.randn((42, 2, 128), generator=g).to(BF).to(DEV)
    qsl, seq = torch.tensor([0, 40, 42], dtype=I32), torch.tensor([16 * cache.width + 30, 1], dtype=I32)
    c = ple.KV8Cache(*tensors)
    where = (qsl.to(DEV), seq.to(DEV), cache.table.to(DEV))
    ple.ple_kv8_append(c, k, k, *where)                     # request 0: 10 tokens inside the table's unnamed last page
    assert all(torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())) for a, b in zip(tensors, before))
    rk, rv = ple.ple_kv8_read(c, *where, 42)
    assert (rk == 0).all() and (rv == 0).all()


# ---- attention ----

def run_attention(cache, q, qsl, lens, **kw):
    c = ple.KV8Cache(*cache.tensors(DEV))
    out, lse = ple.ple_kv8_attention(q.to(DEV), c, qsl.to(DEV), lens.to(DEV), cache.table.to(DEV), want_lse=True, **kw)
    return out.cpu().to(F64), lse.cpu().to(F64)


def check_attention(cache, q, qsl, lens, window=0, scale=None, **kw):
    out, lse = run_attention(cache, q, qsl, lens, window=window, scale=scale, **kw)
    want, want_lse, tol, tol_lse = U.attention(cache, q, qsl, lens, window, scale)
    err = (out - want).abs()
    assert (err <= tol).all(), (float((err - tol).max()), float(err.max()))
    empty = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    assert (out[empty] == 0).all()
    d = (lse - want_lse).abs()[~empty]
    assert (d <= tol_lse[~empty]).all(), float((d - tol_lse[~empty]).max())


ATTENTION = [  # D, Hq, H, page, news, lens, window
    (64, 1, 1, 16, [1], [1], 0), (64, 4, 2, 32, [1, 1, 0, 1], [1, 64, 9, 65], 0),
    (128, 4, 1, 16, [1], [777], 0), (128, 8, 2, 64, [1, 1, 1], [1, 500, 1300], 0),
    (128, 7, 1, 48, [1, 2, 5], [130, 2, 700], 0), (256, 8, 4, 128, [1, 3], [300, 3], 0),
    (128, 16, 2, 32, [4, 1, 3], [400, 1, 90], 128), (64, 8, 1, 16, [8, 8], [8, 700], 100),
    (256, 4, 2, 16, [5, 8], [600, 8], 33), (128, 4, 4, 16, [100], [100], 0), (128, 8, 2, 64, [70, 33], [300, 33], 0),
    (64, 2, 1, 16, [150], [400], 50), (256, 2, 1, 32, [130], [257], 0), (128, 4, 2, 16, [200], [500], 1),
    (128, 32, 8, 16, [17, 129], [45, 700], 0), (256, 8, 2, 64, [65], [320], 100), (64, 14, 2, 16, [30], [31], 0),
    (128, 64, 1, 16, [1, 2], [99, 200], 0), (128, 3, 1, 80, [300], [1100], 300),
]


@pytest.mark.parametrize("hints", [True, False])
@pytest.mark.parametrize("D,Hq,H,page,news,lens,window", ATTENTION)
def test_attention(D, Hq, H, page, news, lens, window, hints):
    say(f"kv8 attention D={D} Hq={Hq} H={H} page={page} new={news} len={lens} window={window} hints={hints}")
    g = gen(D + Hq + sum(lens))
    cache = U.Cache(g, lens, H=H, D=D, page=page)
    qsl, seq = batch(news, lens)
    q = (1.5 * torch.randn((int(qsl[-1]), Hq, D), generator=g)).to(BF)
    kw = dict(max_request_tokens=max(news), max_seq_len=max(lens)) if hints else {}
    check_attention(cache, q, qsl, seq, window, **kw)


@pytest.mark.parametrize("D,Hq,H,news,lens", [(128, 4, 2, [1, 1], [600, 90]), (64, 8, 1, [4], [300]), (128, 4, 1, [90], [500])])
def test_attention_scales_far_apart(D, Hq, H, news, lens):
    """Blocks whose scales lie between the ends of their range, for keys (small enough to leave scores) and values."""
    g = gen(D + Hq)
    cache = U.Cache(g, lens, H=H, D=D, page=16)
    for k, e in (("k", (-32, 1)), ("v", (-32, 33))):
        s = torch.pow(2.0, torch.randint(*e, cache.scales[k].shape, generator=g).to(F64))
        cache.scales[k] = torch.where(torch.isnan(cache.scales[k]), math.nan, s)
    cache.scales["v"] *= 1.37                               # (any positive scale will do)
    cache.scales["v"].clamp_(max=2.0 ** 32)
    cache.scales["v"] = cache.scales["v"].float().to(F64)
    cache.scales["k"] = cache.scales["k"] * 2.0 ** -7
    qsl, seq = batch(news, lens)
    q = torch.randn((int(qsl[-1]), Hq, D), generator=g).to(BF)
    check_attention(cache, q, qsl, seq, max_request_tokens=max(news), max_seq_len=max(lens))


@pytest.mark.parametrize("news", [[1], [40]])
def test_attention_weight_on_tokens_of_no_value(news):
    """Nearly all weight on tokens whose values are zeros at the least scale: what is left of the others comes out right."""
    g = gen(9)
    n = 300
    cache = U.Cache(g, [n], H=1, D=128, page=16)
    p = int(cache.table[0, 0])
    cache.codes["v"][p], cache.scales["v"][p] = 0, 2.0 ** -32
    q = torch.randn((news[0], 2, 128), generator=g).to(BF)
    direction = q.to(F64).mean((0, 1))
    cache.codes["k"][p] = U.codes_of((direction / direction.abs().max() * 200).expand(1, 16, 128))
    cache.scales["k"][p] = 2.0 ** -4
    qsl, seq = batch(news, [n])
    check_attention(cache, q, qsl, seq, max_request_tokens=news[0], max_seq_len=n)


def test_attention_rows_that_see_nothing():
    g = gen(12)
    for news, lens in (([3, 1], [0, 5]), ([40, 2], [10, 3]), ([1, 1], [-5, 7])):
        cache = U.Cache(g, [max(0, n) for n in lens], H=2, D=128, page=16)
        qsl, seq = batch(news, lens)
        q = torch.randn((int(qsl[-1]), 4, 128), generator=g).to(BF)
        check_attention(cache, q, qsl, seq)


@pytest.mark.parametrize("news", [[1, 1], [40, 3]])
def test_attention_leaves_bad_pages_out(news):
    g = gen(13)
    lens = [300, 90]
    cache = U.Cache(g, lens, H=2, D=128, page=16)
    cache.table[0, 3], cache.table[0, 7], cache.table[1, :] = -1, cache.pages, 2 ** 31 - 1
    qsl, seq = batch(news, lens)
    q = torch.randn((int(qsl[-1]), 8, 128), generator=g).to(BF)
    check_attention(cache, q, qsl, seq)


@pytest.mark.parametrize("D,news,window", [(128, [1], 100), (64, [4], 70), (128, [90], 64), (256, [40], 40), (256, [3], 40)])
def test_attention_nan_where_no_row_looks(D, news, window):
    """NaN codes and scales in front of the window's first token, in the block that it lies in too."""
    g = gen(D)
    n = 333
    cache = U.Cache(g, [n], H=2, D=D, page=16)
    qsl, seq = batch(news, [n])
    q = torch.randn((news[0], 4, D), generator=g).to(BF)
    clean = run_attention(cache, q, qsl, seq, window=window)
    first = n - news[0] - window + 1
    for j in range(first):
        p, i = cache.place(0, j)
        for k in "kv":
            cache.codes[k][p, :, i] = 0xFF
            if j // 16 < first // 16:
                cache.scales[k][p, :, i // 16] = math.nan
    got = run_attention(cache, q, qsl, seq, window=window)
    assert all(torch.equal(a, b) for a, b in zip(clean, got))


@pytest.mark.parametrize("k", ["k", "v"])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("D,n,Hq", [(128, 4, 2), (64, 8, 8), (128, 50, 2), (256, 40, 1), (256, 6, 2), (64, 90, 2), (128, 1, 4)])
def test_attention_nan_code_reaches_only_rows_that_see_it(k, window, D, n, Hq):
    """A NaN element of one head's key or value, at several places: a key's makes NaN the rows that see it, a value's that
    element of them; every other output keeps its bits."""
    g = gen(D + n)
    length = 200
    cache = U.Cache(g, [length], H=2, D=D, page=16)
    qsl, seq = batch([n], [length])
    q = torch.randn((n, 2 * Hq, D), generator=g).to(BF)
    kw = dict(window=window, max_request_tokens=n, max_seq_len=length)
    clean, clean_lse = run_attention(cache, q, qsl, seq, **kw)
    before = length - n
    for j in (before + n // 2, before, length - 1, max(0, before - 70), max(0, before - 59)):
        p, i = cache.place(0, j)
        d = (7 * j) % D
        held = cache.codes[k][p, 1, i, d].item()
        cache.codes[k][p, 1, i, d] = 0xFF if j % 2 else 0x7F
        out, lse = run_attention(cache, q, qsl, seq, **kw)
        cache.codes[k][p, 1, i, d] = held
        pos = before + torch.arange(n)
        sees = (pos >= j) & ((pos - window < j) if window else True)
        mine = torch.zeros((n, 2 * Hq), dtype=torch.bool)
        mine[:, Hq:] = sees[:, None]
        assert torch.equal(out[~mine], clean[~mine]) and torch.equal(lse[~mine], clean_lse[~mine])
        if k == "k":
            assert torch.isnan(out[mine]).all() and torch.isnan(lse[mine]).all()
        else:
            rest = [e for e in range(D) if e != d]
            assert torch.isnan(out[mine][:, d]).all() and torch.equal(out[mine][:, rest], clean[mine][:, rest])
            assert torch.equal(lse[mine], clean_lse[mine])


@pytest.mark.parametrize("n", [1, 40])
def test_attention_nonfinite_and_wide_queries(n):
    """Rows with an infinity or NaN are their own affair; rows of 2^100 and 2^-100 come out as the definition says."""
    g = gen(n)
    cache = U.Cache(g, [120], H=1, D=128, page=16)
    qsl, seq = batch([n], [120])
    q = torch.randn((n, 6, 128), generator=g).to(BF)
    clean, clean_lse = run_attention(cache, q, qsl, seq)
    bad = q.clone()
    bad[0, 0, 3], bad[n - 1, 1, 9], bad[0, 2] = math.nan, math.inf, -math.inf
    bad[0, 3], bad[0, 4] = (q[0, 3].float() * 2.0 ** 100).to(BF), (q[0, 4].float() * 2.0 ** -100).to(BF)
    out, lse = run_attention(cache, bad, qsl, seq)
    assert torch.isnan(out[0, 0]).all() and torch.isnan(out[n - 1, 1]).all() and torch.isnan(out[0, 2]).all()
    keep = torch.ones((n, 6), dtype=torch.bool)
    keep[0, :5] = keep[n - 1, 1] = False
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
    want, want_lse, tol, tol_lse = U.attention(cache, bad[:1, 3:5], [0, 1], [120 - n + 1])
    assert ((out[:1, 3:5] - want).abs() <= tol).all() and ((lse[:1, 3:5] - want_lse).abs() <= tol_lse).all()


def test_attention_is_the_same_every_time():
    g = gen(21)
    cache = U.Cache(g, [3000, 100, 2000], H=2, D=128, page=16)
    for news in ([1, 1, 1], [50, 60, 70]):
        qsl, seq = batch(news, cache.lens)
        q = torch.randn((int(qsl[-1]), 8, 128), generator=g).to(BF)
        first = run_attention(cache, q, qsl, seq)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, run_attention(cache, q, qsl, seq)))


def test_attention_no_tokens():
    cache = U.Cache(gen(1), [5], H=1, D=64, page=16)
    out, lse = run_attention(cache, torch.zeros((0, 2, 64), dtype=BF), torch.zeros(2, dtype=I32), torch.tensor([5], dtype=I32))
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
