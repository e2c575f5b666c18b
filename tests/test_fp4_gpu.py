"""The 4-bit decode operators on the GPU against their definitions in 64 bits (fp4_util)."""
import math

import pytest
import torch

import fp4_util as U
import layer_embedding_lookup_amd as ple

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F64, BF = torch.float64, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---- products with 4-bit weights ----

def make_weight(g, fmt, O, K, G, zeros):
    """(W4Weight, W in 64 bits)"""
    codes = torch.randint(0, 256, (O, K // 2), generator=g).to(torch.uint8)
    if fmt == "nvfp4":
        scales = torch.randint(0, 0x7F, (O, K // 16), generator=g).to(torch.uint8)  # every finite scale, 0 and subnormals too
        ts = torch.tensor([0.37])
        w = U.e2m1(codes) * U.e4m3(scales).repeat_interleave(16, -1) * ts.to(F64)
        return ple.W4Weight.nvfp4(codes.to(DEV), scales.to(DEV), ts.to(DEV)), w
    scales = (torch.randn((O, K // G), generator=g) * torch.exp(4 * torch.randn((O, K // G), generator=g))).to(BF)
    zero = torch.randint(0, 16, (O, K // G), generator=g).to(torch.uint8) if zeros else None
    z = zero.to(F64) if zeros else torch.full((O, K // G), 8.0, dtype=F64)
    w = (U.nibbles(codes).to(F64) - z.repeat_interleave(G, -1)) * scales.to(F64).repeat_interleave(G, -1)
    return ple.W4Weight.int4(codes.to(DEV), scales.to(DEV), None if zero is None else zero.to(DEV)), w


def check_linear(x, w, W, out):
    """fp32 sums: (K + 8) roundings of at most 2^-23 of the sum of magnitudes; then bf16's 2^-8."""
    want = x.to(F64) @ W.t()
    acc = (x.shape[1] + 8) * 2.0 ** -23 * (x.to(F64).abs() @ W.abs().t())
    err = (out.cpu().to(F64) - want).abs()
    assert (err <= 2.0 ** -8 * (want.abs() + acc) + acc).all(), float((err - acc).max())


FORMATS = [("nvfp4", 16, False), ("int4", 32, False), ("int4", 64, True), ("int4", 128, True), ("int4", 128, False)]


@pytest.mark.parametrize("fmt,G,zeros", FORMATS)
@pytest.mark.parametrize("T,O,K", [(1, 1, 128), (1, 300, 512), (2, 17, 384), (5, 515, 1152), (16, 48, 256),
                                   (17, 100, 640), (33, 333, 1280), (64, 130, 512), (65, 257, 896), (129, 65, 384),
                                   (200, 270, 1024), (257, 520, 2048), (600, 1031, 640), (1024, 2048, 512), (2051, 2053, 384),
                                   (900, 4096, 1152)])
def test_linear(fmt, G, zeros, T, O, K):
    print(f"linear {fmt} G={G} T={T} O={O} K={K}", flush=True)
    g = gen(T * 7 + O + K)
    w, W = make_weight(g, fmt, O, K, G, zeros)
    x = torch.randn((T, K), generator=g).to(BF)
    out = ple.ple_w4_linear(x.to(DEV), w)
    check_linear(x, w, W, out)


@pytest.mark.parametrize("fmt,G,K", [("nvfp4", 16, 32), ("nvfp4", 16, 32 * 33), ("int4", 32, 32 * 5), ("int4", 64, 64 * 3)])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_linear_short_last_step(fmt, G, K, T):
    g = gen(K + T)
    w, W = make_weight(g, fmt, 77, K, G, fmt == "int4")
    x = torch.randn((T, K), generator=g).to(BF)
    check_linear(x, w, W, ple.ple_w4_linear(x.to(DEV), w))


@pytest.mark.parametrize("T", [3, 70, 300])
def test_linear_strided_rows_and_wide_range(T):
    """Rows sliced out of a wider tensor, values from 1e-30 to 1e30 (one magnitude a token)."""
    g = gen(T)
    w, W = make_weight(g, "nvfp4", 90, 512, 16, False)
    wide = torch.randn((T, 1024), generator=g) * torch.pow(10.0, torch.randint(-30, 31, (T, 1), generator=g).float())
    wide = wide.to(BF)
    out = ple.ple_w4_linear(wide.to(DEV)[:, 256:768], w)
    check_linear(wide[:, 256:768], w, W, out)


@pytest.mark.parametrize("fmt,G", [("nvfp4", 16), ("int4", 64)])
@pytest.mark.parametrize("T", [4, 80, 300])
def test_linear_nonfinite_rows_stay_apart(fmt, G, T):
    g = gen(T + G)
    w, W = make_weight(g, fmt, 50, 256, G, False)
    x = torch.randn((T, 256), generator=g).to(BF)
    bad = x.clone()
    bad[1, 7], bad[2, 100] = math.inf, math.nan
    out = ple.ple_w4_linear(bad.to(DEV), w).cpu()
    assert not torch.isfinite(out[1]).any() or (W[:, 7] == 0).any()
    assert torch.isnan(out[2]).all()
    keep = [i for i in range(T) if i not in (1, 2)]
    assert torch.equal(out[keep], ple.ple_w4_linear(x.to(DEV), w).cpu()[keep])


def test_linear_no_tokens():
    w, _ = make_weight(gen(1), "nvfp4", 32, 64, 16, False)
    assert ple.ple_w4_linear(torch.empty((0, 64), dtype=BF, device=DEV), w).shape == (0, 32)


# ---- the cache ----

def batch(news, lens, cache):
    qsl = torch.tensor([0] + news).cumsum(0).int()
    return qsl, torch.tensor(lens, dtype=torch.int32), cache.table


def positions(qsl, lens):
    r = torch.repeat_interleave(torch.arange(len(lens)), (qsl[1:] - qsl[:-1]).long())
    t = torch.arange(int(qsl[-1]))
    return r, lens[r].long() - (qsl[r + 1].long() - t)


APPEND = [(64, 1, 1, 16, [1], [1], 64, False), (64, 8, 2, 32, [1, 0, 3], [17, 5, 33], 32, True),
          (128, 8, 8, 16, [2, 5, 1], [2, 100, 1], 128, False), (128, 7, 1, 64, [40], [200], 64, True),
          (256, 4, 4, 128, [3, 9], [130, 9], 64, False), (256, 6, 2, 48, [1] * 5, [100001, 1, 2, 3, 77], 256, True),
          (128, 2, 2, 16, [20], [20], 0, False)]


@pytest.mark.parametrize("D,Hq,H,page,news,lens,rot,interleaved", APPEND)
def test_append_and_read(D, Hq, H, page, news, lens, rot, interleaved):
    print(f"append D={D} Hq={Hq} H={H} page={page} rot={rot}", flush=True)
    g = gen(D + Hq + page)
    # the table of a long sequence names the pages of its new tokens only
    short = [min(n, 512) for n in lens]
    cache = U.Cache(g, short, H=H, D=D, page=page, poison=False)
    width = max(-(-n // page) for n in lens)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for r, n in enumerate(lens):
        need = -(-n // page)
        have = -(-short[r] // page)
        table[r, need - have:need] = cache.table[r, :have]
    qsl, seq = torch.tensor([0] + news).cumsum(0).int(), torch.tensor(lens, dtype=torch.int32)
    T = int(qsl[-1])
    qkv = torch.randn((T, (Hq + 2 * H) * D), generator=g).to(BF)
    qkv[0, :16] = 0
    qkv[0, Hq * D:Hq * D + 16] = 0       # a key block of zeros
    qkv[-1, -16:] *= 1e4                 # a value block beyond the largest scale
    inv = (1e4 ** (-torch.arange(0, rot, 2, dtype=F64) / max(rot, 1))).float()
    q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([Hq * D, H * D, H * D], -1))
    dev = [t.to(DEV) for t in cache.tensors("cpu")]
    c = ple.KV4Cache(*dev)
    dq = qkv.to(DEV)
    gq, gk, gv = (t.unflatten(-1, (-1, D)) for t in dq.split([Hq * D, H * D, H * D], -1))
    args = (qsl.to(DEV), seq.to(DEV), table.to(DEV))
    out = ple.ple_kv4_append(c, gk, gv, *args, inv_freq=inv.to(DEV) if rot else None, interleaved=interleaved, q=gq)
    back = ple.ple_kv4_read(c, *args, T)
    r, pos = positions(qsl, seq)
    want_q, want_k = (U.rotate(x, pos, inv, interleaved) if rot else x.to(F64) for x in (q, k))
    # 64-bit angles and products: what is left is the rounding to fp32 (2^-24) and to bf16 (2^-8)
    assert ((out.cpu().to(F64) - want_q).abs() <= (2.0 ** -8 + 2.0 ** -20) * want_q.abs() + 2.0 ** -40).all()
    for i, (name, x) in enumerate((("k", want_k.float()), ("v", v.float()))):
        codes, scales = U.quantise(x, cache.scale[name][:, None])
        page_of, at = table[r, pos // page].long(), pos % page
        assert torch.equal(dev[2 * i].cpu()[page_of, :, at], codes), name
        assert torch.equal(dev[2 * i + 1].cpu()[page_of, :, at // 16, :, at % 16], scales), name
        # nothing else has changed
        cc, ss = cache.codes[name].clone(), cache.scales[name].clone()
        cc[page_of, :, at], ss[page_of, :, at // 16, :, at % 16] = codes, scales
        assert torch.equal(dev[2 * i].cpu(), cc) and torch.equal(dev[2 * i + 1].cpu(), ss)
        held = U.e2m1(codes) * U.e4m3(scales).repeat_interleave(16, -1) * cache.scale[name].to(F64)[:, None]
        assert torch.equal(back[i].cpu(), held.float().to(BF)), name


def test_append_ties_go_to_the_even_code():
    """Quotients on every border, next to it and beyond the largest code, of both signs: scales that are powers of two
    make them exact."""
    border = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0]).to(BF)
    above, below = ((border.view(torch.int16) + i).view(BF) for i in (1, -1))
    t = torch.cat((border, above, below, torch.tensor([0., .5, 1., 1.5, 2., 3., 4., 6., 5.75]).to(BF))).float()
    t = torch.cat((t, -t, torch.tensor([0., -0., 6., -6.])))           # 64 quotients
    blocks = torch.cat((t.view(-1, 8), torch.full((len(t) // 8, 1), 6.0), torch.zeros(len(t) // 8, 7)), 1)
    k = blocks.reshape(1, 1, 128).to(BF)                                # each block's largest is 6, so its step is 1
    assert torch.equal(k.float().view(-1), blocks.view(-1))
    cache = U.Cache(gen(22), [1], H=1, D=128, page=16, poison=False)
    cache.scale = {n: torch.tensor([2.0 ** -4]) for n in "kv"}
    dev = [x.to(DEV) for x in cache.tensors("cpu")]
    args = (torch.tensor([0, 1], dtype=torch.int32, device=DEV), torch.tensor([1], dtype=torch.int32, device=DEV),
            cache.table.to(DEV))
    ple.ple_kv4_append(ple.KV4Cache(*dev), k.to(DEV), k.to(DEV), *args)
    codes, scales = U.quantise(k.float(), cache.scale["k"][:, None])
    assert (scales == torch.tensor(16.0).to(torch.float8_e4m3fn).view(torch.uint8)).all()
    page = int(cache.table[0, 0])
    for i in (0, 2):
        assert torch.equal(U.nibbles(dev[i].cpu()[page, 0, 0]), U.nibbles(codes[0, 0]))


def test_append_bad_pages_and_places_write_nothing():
    """Table entries outside the cache, and tokens before position 0: dropped, read back as zeros."""
    g = gen(5)
    cache = U.Cache(g, [64, 64, 2], H=2, D=128, page=16, poison=False)
    table = cache.table.clone()
    table[0, 3], table[1, 3] = -1, cache.pages
    qsl, seq = torch.tensor([0, 2, 3, 8], dtype=torch.int32), torch.tensor([64, 64, 2], dtype=torch.int32)
    dev = [t.to(DEV) for t in cache.tensors("cpu")]
    c = ple.KV4Cache(*dev)
    k = torch.randn((8, 2, 128), generator=g).to(BF).to(DEV)
    args = (qsl.to(DEV), seq.to(DEV), table.to(DEV))
    ple.ple_kv4_append(c, k, k, *args)
    got, _ = ple.ple_kv4_read(c, *args, 8)
    assert (got[:6] == 0).all() and (got[6:] != 0).any()  # request 2 has 5 new tokens but 2 in all: places -3, -2, -1, 0, 1
    changed = (dev[0].cpu() != cache.codes["k"]).flatten(1).any(1)
    assert changed.sum() == 1 and changed[int(table[2, 0])]


def test_append_nonfinite_blocks():
    """A NaN makes its block's scale NaN, an infinity the largest; other blocks are untouched by them."""
    g = gen(6)
    cache = U.Cache(g, [1], H=1, D=64, page=16, poison=False)
    dev = [t.to(DEV) for t in cache.tensors("cpu")]
    c = ple.KV4Cache(*dev)
    k = torch.randn((1, 1, 64), generator=g).to(BF)
    k[0, 0, 3], k[0, 0, 20] = math.nan, math.inf
    args = (torch.tensor([0, 1], dtype=torch.int32, device=DEV), torch.tensor([1], dtype=torch.int32, device=DEV),
            cache.table.to(DEV))
    ple.ple_kv4_append(c, k.to(DEV), k.to(DEV), *args)
    s = dev[1].cpu()[int(cache.table[0, 0]), 0, 0, :, 0]
    assert int(s[0]) & 0x7F == 0x7F and int(s[1]) == 0x7E
    codes, scales = U.quantise(k.float(), cache.scale["k"][:, None])
    assert torch.equal(s[2:], scales[0, 0, 2:])
    assert torch.equal(dev[0].cpu()[int(cache.table[0, 0]), 0, 0, 16:], codes[0, 0, 16:])


# ---- attention ----

def run_attention(cache, q, qsl, lens, **kw):
    c = ple.KV4Cache(*cache.tensors(DEV))
    out, lse = ple.ple_kv4_attention(q.to(DEV), c, qsl.to(DEV), lens.to(DEV), cache.table.to(DEV), want_lse=True, **kw)
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
    print(f"attention D={D} Hq={Hq} H={H} page={page} news={news} lens={lens} window={window}", flush=True)
    g = gen(D + Hq * 3 + page + sum(lens))
    cache = U.Cache(g, lens, H=H, D=D, page=page)
    qsl, seq, _ = batch(news, lens, cache)
    q = (1.5 * torch.randn((int(qsl[-1]), Hq, D), generator=g)).to(BF)
    kw = dict(max_request_tokens=max(news), max_seq_len=max(lens)) if hints else {}
    check_attention(cache, q, qsl, seq, window, **kw)


@pytest.mark.parametrize("D,Hq,H,page,news,lens,window", [
    (128, 8, 2, 64, [150, 0, 40, 129], [2500, 3, 1700, 129], 0), (64, 4, 1, 16, [300, 70], [1900, 2600], 0),
    (256, 4, 2, 32, [33, 200], [2049, 260], 0), (128, 16, 2, 48, [90, 41], [1500, 2200], 700),
    (128, 8, 1, 16, [20] * 65, [20 + 9 * i for i in range(65)], 0), (64, 4, 2, 16, [3, 40] * 20, [64, 200] * 20, 0),
    (128, 2, 1, 16, [100], [4500], 0)])
def test_attention_chunks_of_ragged_lengths(D, Hq, H, page, news, lens, window):
    """Query tiles cut into pieces at any place, whole ones between them, requests without tokens; more requests than
    lanes of a wave."""
    print(f"chunks D={D} Hq={Hq} H={H} page={page} news={news[:4]} lens={lens[:4]} window={window}", flush=True)
    g = gen(D + Hq + sum(lens))
    cache = U.Cache(g, lens, H=H, D=D, page=page)
    qsl, seq, _ = batch(news, lens, cache)
    q = (1.5 * torch.randn((int(qsl[-1]), Hq, D), generator=g)).to(BF)
    check_attention(cache, q, qsl, seq, window, max_request_tokens=max(news), max_seq_len=max(lens))


def test_attention_chunk_rows_that_see_nothing():
    """As below, with enough new tokens for the many-row kernel."""
    g = gen(20)
    lens = [30, 0, 700, -5]
    cache = U.Cache(g, lens, H=1, D=128, page=16)
    cache.table[2, :] = -1
    qsl, seq = torch.tensor([0, 60, 80, 150, 190], dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
    q = torch.randn((190, 4, 128), generator=g).to(BF)
    out, lse = run_attention(cache, q, qsl, seq)
    assert (lse[:30] == -math.inf).all() and (lse[60:] == -math.inf).all() and (out[:30] == 0).all() and (out[60:] == 0).all()
    want, want_lse, tol, tol_lse = U.attention(cache, q[30:60], torch.tensor([0, 30]), seq[:1])
    assert ((out[30:60] - want).abs() <= tol).all() and ((lse[30:60] - want_lse).abs() <= tol_lse).all()


def test_attention_rows_that_see_nothing():
    """More new tokens than the sequence holds (rows before position 0), an empty sequence, a sequence of bad pages."""
    g = gen(11)
    lens = [3, 0, 40, -5]
    cache = U.Cache(g, lens, H=2, D=128, page=16)
    cache.table[2, :] = -1
    qsl, seq = torch.tensor([0, 6, 8, 10, 11], dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)
    q = torch.randn((11, 4, 128), generator=g).to(BF)
    out, lse = run_attention(cache, q, qsl, seq)
    assert (lse[:3] == -math.inf).all() and (lse[6:] == -math.inf).all() and (out[:3] == 0).all() and (out[6:] == 0).all()
    want, want_lse, tol, tol_lse = U.attention(cache, q[3:6], torch.tensor([0, 3]), seq[:1])
    assert ((out[3:6] - want).abs() <= tol).all() and ((lse[3:6] - want_lse).abs() <= tol_lse).all()


@pytest.mark.parametrize("news", [[1, 1], [40, 3]])
def test_attention_leaves_bad_pages_out(news):
    g = gen(12)
    lens = [200, 330]
    cache = U.Cache(g, lens, H=2, D=128, page=16)
    cache.table[0, 4], cache.table[1, 0], cache.table[1, 9] = -1, cache.pages, 2 ** 31 - 1
    qsl, seq, _ = batch(news, lens, cache)
    q = torch.randn((int(qsl[-1]), 8, 128), generator=g).to(BF)
    check_attention(cache, q, qsl, seq)


@pytest.mark.parametrize("D,news,window", [(128, [1], 100), (64, [4], 70), (128, [90], 64), (256, [40], 40)])
def test_attention_nan_where_no_row_looks(D, news, window):
    """Tokens before every row's window hold NaN scales."""
    g = gen(13)
    lens = [450]
    cache = U.Cache(g, lens, H=1, D=D, page=16)
    for j in range(0, lens[0] - news[0] - window + 1):
        for k in "kv":
            cache.scales[k][int(cache.table[0, j // 16]), :, 0, :, j % 16] = 0xFF
    clean = U.Cache(gen(13), lens, H=1, D=D, page=16)
    qsl, seq, _ = batch(news, lens, cache)
    q = torch.randn((news[0], 4, D), generator=g).to(BF)
    out, lse = run_attention(cache, q, qsl, seq, window=window)
    want, want_lse, tol, tol_lse = U.attention(clean, q, qsl, seq, window)
    assert ((out - want).abs() <= tol).all() and ((lse - want_lse).abs() <= tol_lse).all()


@pytest.mark.parametrize("k", ["k", "v"])
@pytest.mark.parametrize("D,n,Hq", [(128, 4, 2), (64, 8, 8), (128, 50, 2), (256, 40, 1)])
def test_attention_nan_token_reaches_only_rows_that_see_it(k, D, n, Hq):
    """A draft whose key or value is NaN must not reach the rows before it."""
    g = gen(14)
    cache = U.Cache(g, [300], H=1, D=D, page=32)
    qsl, seq, _ = batch([n], [300], cache)
    q = torch.randn((n, Hq, D), generator=g).to(BF)
    clean, _ = run_attention(cache, q, qsl, seq)
    j = 300 - n + n // 2
    cache.scales[k][int(cache.table[0, j // 32]), 0, (j % 32) // 16, 1, j % 16] = 0x7F
    out, lse = run_attention(cache, q, qsl, seq)
    assert torch.equal(out[:n // 2], clean[:n // 2])
    assert torch.isnan(out[n // 2:, :, 16:32]).all()


@pytest.mark.parametrize("n", [1, 40])
def test_attention_nonfinite_and_wide_queries(n):
    """A query row with NaN or an infinity spoils only itself; rows of 1e-30 and 1e30 keep their precision."""
    g = gen(15)
    cache = U.Cache(g, [150], H=1, D=128, page=16)
    qsl, seq, _ = batch([n], [150], cache)
    q = torch.randn((n, 6, 128), generator=g).to(BF)
    clean, _ = run_attention(cache, q, qsl, seq)
    bad = q.clone()
    bad[0, 1, 5], bad[0, 2, 9] = math.nan, math.inf
    out, lse = run_attention(cache, bad, qsl, seq)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1]) and torch.isnan(out[0, 2]).all()
    out[0, 1:3], clean[0, 1:3] = 0, 0
    assert torch.equal(out, clean)
    tiny = q.clone()
    tiny[0, 0] *= 1e-30
    check_attention(cache, tiny, qsl, seq)
    big = q.clone()
    big[0, 0] *= 1e30
    check_attention(cache, big, qsl, seq, scale=1e-30)


def test_attention_one_token_dominates_many():
    """One key with almost all of the weight in front of thousands of light ones."""
    g = gen(16)
    cache = U.Cache(g, [3000], H=1, D=64, page=16, magnitude=0.05)
    qsl, seq, _ = batch([1], [3000], cache)
    p = int(cache.table[0, 0])
    cache.codes["k"][p, 0, 0], cache.scales["k"][p, 0, 0, :, 0] = 0x77, 0x70
    q = torch.full((1, 2, 64), 0.02).to(BF)
    check_attention(cache, q, qsl, seq)


def test_attention_strided_queries_streams_and_graph():
    """Queries sliced out of a fused row, another stream, a caller's workspace, and replays of a captured call with
    eager work between them."""
    g = gen(17)
    lens = [900, 300, 1]
    cache = U.Cache(g, lens, H=2, D=128, page=64)
    qsl, seq, _ = batch([1, 1, 1], lens, cache)
    wide = torch.randn((3, 12 * 128), generator=g).to(BF).to(DEV)
    q = wide[:, :1024].unflatten(-1, (8, 128))
    c = ple.KV4Cache(*cache.tensors(DEV))
    args = (c, qsl.to(DEV), seq.to(DEV), cache.table.to(DEV))
    kw = dict(max_request_tokens=1, max_seq_len=900, want_lse=True)
    want, want_lse = ple.ple_kv4_attention(q.contiguous(), *args, **kw)
    need = ple.ple_kv4_attention_workspace_bytes(c, 8, 3, 3, cache.width, max_request_tokens=1, max_seq_len=900)
    ws = torch.empty((max(need, 16),), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = ple.ple_kv4_attention(q, *args, workspace=ws, **kw)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    w, _ = make_weight(gen(3), "nvfp4", 256, 1024, 16, False)
    y = torch.empty((3, 256), dtype=BF, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ple.ple_kv4_attention(q, *args, workspace=ws, out=out, lse=lse, **kw)
        ple.ple_w4_linear(out.view(3, 1024), w, out=y)
    for i in range(4):
        wide.normal_(generator=torch.Generator(device=DEV).manual_seed(i))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        eager, eager_lse = ple.ple_kv4_attention(q, *args, **kw)
        assert torch.equal(out, eager) and torch.equal(lse, eager_lse)
        assert torch.equal(y, ple.ple_w4_linear(eager.view(3, 1024), w))


@pytest.mark.parametrize("handle", [False, True])
def test_attention_keeps_its_workspace_for_another_stream(handle):
    """A call on a stream of the caller's that is still busy: its own workspace must not go to the next allocation."""
    g = gen(21)
    cache = U.Cache(g, [2500], H=1, D=128, page=16)
    qsl, seq, _ = batch([1], [2500], cache)
    q = torch.randn((1, 8, 128), generator=g).to(BF)
    c = ple.KV4Cache(*cache.tensors(DEV))
    args = (q.to(DEV), c, qsl.to(DEV), seq.to(DEV), cache.table.to(DEV))
    kw = dict(max_request_tokens=1, max_seq_len=2500, want_lse=True)
    need = ple.ple_kv4_attention_workspace_bytes(c, 8, 1, 1, cache.width, max_request_tokens=1, max_seq_len=2500)
    assert need > 0
    want, want_lse = ple.ple_kv4_attention(*args, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms
    out, lse = ple.ple_kv4_attention(*args, stream=side.cuda_stream if handle else side, **kw)
    taken = [torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(8)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and len(taken) == 8


def test_attention_is_the_same_every_time():
    g = gen(18)
    lens = [2000, 700]
    cache = U.Cache(g, lens, H=1, D=128, page=16)
    qsl, seq, _ = batch([1, 1], lens, cache)
    q = torch.randn((2, 8, 128), generator=g).to(BF)
    first = run_attention(cache, q, qsl, seq, max_request_tokens=1, max_seq_len=2000)
    for _ in range(3):
        again = run_attention(cache, q, qsl, seq, max_request_tokens=1, max_seq_len=2000)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attention_no_tokens():
    cache = U.Cache(gen(19), [5], H=1, D=64, page=16)
    out, lse = run_attention(cache, torch.empty((0, 2, 64), dtype=BF), torch.tensor([0, 0], dtype=torch.int32),
                             torch.tensor([5], dtype=torch.int32))
    assert out.shape == (0, 2, 64)
