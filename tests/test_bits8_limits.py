"""Calls of the 8-bit decode operators at the limits that the header states and at those of a launch (below 2^32 threads
along x, grids that go on along y)."""
import ctypes

import pytest
import torch

import bits8_util as U
import layer_embedding_lookup_amd as ple
from layer_embedding_lookup_amd import capi

FAKE = 1 << 40
DEV = "cuda:0"
BF, I8, I32, U8 = torch.bfloat16, torch.int8, torch.int32, torch.uint8


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="made-up addresses stay off hosts with a GPU")
@pytest.mark.parametrize("T,R,H,Hq,width,new,refused", [
    (8192, 8192, 8, 32, 5, 0, True), (8192, 8192, 8, 32, 5, 1, False), (8191, 8191, 8, 32, 5, 0, False),
    (1 << 16, 1 << 16, 256, 256, 5, 1, True), (1 << 24, 1, 1, 64, 5000, 1, True)])
def test_attention_launches(T, R, H, Hq, width, new, refused):
    lib = capi.load()
    cache = ctypes.byref(capi.ple_kv8_cache(FAKE, FAKE, FAKE, FAKE, 10, H, 16, 128, 0))
    batch = ctypes.byref(capi.ple_kv4_batch(FAKE, FAKE, FAKE, T, R, width, new, 0))
    rc = lib.ple_kv8_attention(FAKE, Hq * 128, Hq, cache, batch, 0, 0.1, FAKE, None, FAKE, 1 << 62, None)
    assert (rc == capi.PLE_ERR_UNSUPPORTED and "max_request_tokens" in ple.ple_error_message()) == refused
    assert rc != capi.PLE_ERR_INVALID_ARGUMENT


def random_codes(shape, g, low=-128):
    return torch.randint(low, 128, shape, dtype=I8, device=DEV, generator=g)


@pytest.mark.gpu
@pytest.mark.parametrize("T,N", [(1 << 24, 16), ((1 << 22) + 5, 528), ((1 << 20) + 3, 4112), (40000, 65552)])
def test_norm_of_many_tokens(T, N):
    """Grids past 2^20 blocks and rows past 4 GiB: the last tokens are those of a call of their own, and every scale is
    there."""
    g = torch.Generator(device=DEV).manual_seed(40)
    x = torch.empty((T, N), dtype=BF, device=DEV).normal_(generator=g)
    w = torch.randn(N, generator=g, device=DEV).to(BF)
    scales = torch.full((T,), -1.0, device=DEV)
    codes, scales, h = ple.ple_rms_norm8(x, w, residual=x, scales=scales, residual_out=x.clone())
    assert (scales > 0).all()
    own = ple.ple_rms_norm8(x[-5:], w, residual=x[-5:])
    assert all(torch.equal(a[-5:], b) for a, b in zip((codes, scales, h), own))


@pytest.mark.gpu
def test_append_and_read_of_the_most_tokens():
    """PLE_MAX_TOKENS tokens of one request, the same 65536 in every page."""
    T, page, D = 1 << 24, 1 << 16, 64
    g = torch.Generator().manual_seed(41)
    base = torch.randn((page, 1, D), generator=g).to(BF)
    k = base.to(DEV).repeat(T // page, 1, 1)
    pages = T // page
    codes = [torch.zeros(s, dtype=U8, device=DEV) for s in ((pages, 1, page // 16, D // 16, 16, 16), (pages, 1, page // 16, D, 16))]
    scales = [torch.zeros((pages, 1, page // 16), device=DEV) for _ in range(2)]
    c = ple.KV8Cache(codes[0], scales[0], codes[1], scales[1])
    args = (torch.tensor([0, T], dtype=I32, device=DEV), torch.tensor([T], dtype=I32, device=DEV),
            torch.arange(pages, dtype=I32, device=DEV)[None])
    ple.ple_kv8_append(c, k, k, *args)
    x = base.double().view(page // 16, 16, D)
    s = U.block_scale(x.abs().amax((1, 2)))
    want = U.codes_of(x / s[:, None, None])                   # [blocks][16][D]
    assert (codes[0] == want.view(-1, 16, D // 16, 16).transpose(1, 2).to(DEV)).all()
    assert (codes[1] == want.transpose(1, 2).to(DEV)).all()
    assert all((y == s.float().to(DEV)).all() for y in scales)
    held = (U.e4m3(want) * s[:, None, None]).float().to(BF).view(1, page, D).to(DEV)
    for y in ple.ple_kv8_read(c, *args, T):
        assert (y.view(pages, page, D) == held).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n,Hq", [(1, 4), (5, 4), (5, 8), (100, 2)])
def test_a_cache_of_more_than_4_gib(n, Hq):
    """The same three pages at the far ends of such a cache and in one of their own: append, read and attention agree to
    the bit."""
    pages, page, D, at = 550, 65536, 128, [549, 3, 530]
    g = torch.Generator(device=DEV).manual_seed(42)

    def tensors(p):
        codes = [torch.empty(s, dtype=U8, device=DEV) for s in ((p, 1, page // 16, D // 16, 16, 16), (p, 1, page // 16, D, 16))]
        return [codes[0], torch.empty((p, 1, page // 16), device=DEV), codes[1], torch.empty((p, 1, page // 16), device=DEV)]

    big, small = tensors(pages), tensors(3)
    for i, (x, y) in enumerate(zip(big, small)):
        # (codes of up to 1.875, scales of powers of two)
        y.copy_(random_codes(y.shape, g).view(U8) & 0xBF if i % 2 == 0 else
                torch.pow(2.0, torch.randint(-2, 1, y.shape, device=DEV, generator=g)))
        x[at] = y
    length = 2 * page + 777
    args = [torch.tensor([0, n], dtype=I32, device=DEV), torch.tensor([length], dtype=I32, device=DEV)]
    q, k = (torch.randn((n, h, D), generator=g, device=DEV).to(BF) for h in (Hq, 1))
    got = []
    for t, table in ((big, at), (small, [0, 1, 2])):
        c = ple.KV8Cache(*t)
        where = (*args, torch.tensor([table], dtype=I32, device=DEV))
        ple.ple_kv8_append(c, k, k, *where)
        got.append((*ple.ple_kv8_read(c, *where, n),
                    *ple.ple_kv8_attention(q, c, *where, max_request_tokens=n, max_seq_len=length, want_lse=True)))
    assert all(torch.equal(x, y) for x, y in zip(*got)) and torch.isfinite(got[0][2]).all()
    assert all(torch.equal(x[at], y) for x, y in zip(big, small))


@pytest.mark.gpu
@pytest.mark.parametrize("T,O,K", [(3, (1 << 20) + 40, 4112), (20, (1 << 20) + 40, 4112), (100, (1 << 20) + 40, 4112),
                                   (2100, (1 << 20) + 40, 64), ((1 << 20) + 40, 130, 4112), ((1 << 20) + 40, 4100, 16)])
def test_weights_inputs_and_outputs_of_more_than_4_gib(T, O, K):
    """The last features of the first and the last tokens, of weights, inputs or outputs of 4.3 GB and more."""
    g = torch.Generator(device=DEV).manual_seed(43)
    w, x = random_codes((O, K), g), random_codes((T, K), g)
    ws, xs = torch.rand(O, generator=g, device=DEV), torch.rand(T, generator=g, device=DEV)
    out = ple.ple_w8_linear(x, xs, ple.W8Weight(w, ws))
    n, m = min(T, 100), min(O, 100)
    for rows in (slice(0, n), slice(T - n, T)):
        want = (x[rows].cpu().double() @ w[-m:].cpu().double().t()) * ws[-m:].cpu().double() * xs[rows].cpu().double()[:, None]
        # (as in test_bits8_gpu.check_linear)
        assert ((out[rows, -m:].cpu().double() - want).abs() <= (2.0 ** -8 + 2.0 ** -21) * want.abs()).all()


@pytest.mark.gpu
def test_queries_and_outputs_of_more_than_4_gib():
    """A decode step of 2^19 + 5 requests of 1 .. 40 tokens, 32 heads of 128: its last rows are those of a call of their
    own, in append too."""
    T, Hq, D, page, last = (1 << 19) + 5, 32, 128, 64, 300
    g = torch.Generator(device=DEV).manual_seed(44)
    c = ple.KV8Cache(random_codes((64, 1, page // 16, D // 16, 16, 16), g).view(U8) & 0xBF, torch.ones((64, 1, page // 16), device=DEV),
                     random_codes((64, 1, page // 16, D, 16), g).view(U8) & 0xBF, torch.ones((64, 1, page // 16), device=DEV))
    q = torch.empty((T, Hq, D), dtype=BF, device=DEV).normal_(generator=g)
    seq = torch.randint(1, 41, (T,), dtype=I32, device=DEV, generator=g)
    table = torch.randint(0, 64, (T, 1), dtype=I32, device=DEV, generator=g)
    qsl = torch.arange(T + 1, dtype=I32, device=DEV)
    kw = dict(max_request_tokens=1, max_seq_len=40, want_lse=True)
    out, lse = ple.ple_kv8_attention(q, c, qsl, seq, table, **kw)
    mine = (qsl[:last + 1], seq[-last:].clone(), table[-last:].clone())
    own, own_lse = ple.ple_kv8_attention(q[-last:], c, *mine, **kw)
    assert torch.equal(out[-last:], own) and torch.equal(lse[-last:], own_lse) and torch.isfinite(own).all()
    none = torch.full_like(table, -1)                         # (no page: only the queries are turned)
    inv = torch.logspace(0, -4, 64).to(DEV)
    k = q[:, :1].contiguous()
    turned = ple.ple_kv8_append(c, k, k, qsl, seq, none, inv_freq=inv, q=q, max_request_tokens=1)
    own = ple.ple_kv8_append(c, k[-last:], k[-last:], mine[0], mine[1], none[-last:].clone(), inv_freq=inv, q=q[-last:])
    assert torch.equal(turned[-last:], own)
