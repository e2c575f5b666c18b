"""Calls at the limits that the header states and at those of a launch (below 2^32 threads along x)."""
import ctypes

import pytest
import torch

import fp4_util as U
import layer_embedding_lookup_amd as ple
from layer_embedding_lookup_amd import capi

FAKE = 1 << 40
DEV = "cuda:0"


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="made-up addresses stay off hosts with a GPU")
@pytest.mark.parametrize("T,R,H,Hq,width,new,refused", [
    (8192, 8192, 8, 32, 5, 0, True), (8192, 8192, 8, 32, 5, 1, False),   # 2^24 blocks of 256 threads, 2^16
    (8191, 8191, 8, 32, 5, 0, False),                                    # 2^24 less 2048
    (1 << 16, 1 << 16, 256, 256, 5, 1, True),                            # 2^24 blocks of four waves, a row each
    (1 << 24, 1, 1, 64, 5000, 1, True)])                                # (a wrong hint: splits of one token, joined for 2^30 rows)
def test_attention_launches(T, R, H, Hq, width, new, refused):
    lib = capi.load()
    cache = ctypes.byref(capi.ple_kv4_cache(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 10, H, 16, 128, 0))
    batch = ctypes.byref(capi.ple_kv4_batch(FAKE, FAKE, FAKE, T, R, width, new, 0))
    rc = lib.ple_kv4_attention(FAKE, Hq * 128, Hq, cache, batch, 0, 0.1, FAKE, None, FAKE, 1 << 62, None)
    assert (rc == capi.PLE_ERR_UNSUPPORTED and "max_request_tokens" in ple.ple_error_message()) == refused
    assert rc != capi.PLE_ERR_INVALID_ARGUMENT


@pytest.mark.gpu
def test_append_and_read_of_the_most_tokens():
    """PLE_MAX_TOKENS tokens of one request, the same 65536 in every page."""
    T, page, D = 1 << 24, 1 << 16, 64
    g = torch.Generator().manual_seed(41)
    base = torch.randn((page, 1, D), generator=g).bfloat16()
    k = base.to(DEV).repeat(T // page, 1, 1)
    codes = [torch.zeros((T // page, 1, page, D // 2), dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros((T // page, 1, page // 16, D // 16, 16), dtype=torch.uint8, device=DEV) for _ in range(2)]
    one = torch.full((1,), 0.03, device=DEV)
    c = ple.KV4Cache(codes[0], scales[0], codes[1], scales[1], one, one)
    args = (torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.tensor([T], dtype=torch.int32, device=DEV),
            torch.arange(T // page, dtype=torch.int32, device=DEV)[None])
    ple.ple_kv4_append(c, k, k, *args)
    want, want_scales = U.quantise(base.float(), one.cpu()[:, None])
    for x, y in zip(codes, scales):
        assert (x == want.to(DEV).view(1, 1, page, D // 2)).all()
        assert (y == U.scale_layout(want_scales.view(1, 1, page, D // 16), page).to(DEV)).all()
    held = U.e2m1(want) * U.e4m3(want_scales).repeat_interleave(16, -1) * one.cpu().double()
    held = held.float().bfloat16().to(DEV)
    for x in ple.ple_kv4_read(c, *args, T):
        assert (x.view(T // page, page, D) == held.view(1, page, D)).all()


# ---- byte offsets past 2^32 ----

def random_bytes(shape, g, top=256):
    return torch.randint(0, top, shape, dtype=torch.uint8, device=DEV, generator=g)


@pytest.mark.gpu
@pytest.mark.parametrize("n,Hq", [(1, 4), (5, 4), (5, 8), (100, 2)])
def test_a_cache_of_more_than_4_gib(n, Hq):
    """The same three pages at the far ends of such a cache and in one of their own: append, read and attention agree to
    the bit."""
    pages, page, D, at = 1100, 65536, 128, [1099, 3, 1060]
    g = torch.Generator(device=DEV).manual_seed(42)
    one = torch.full((1,), 0.02, device=DEV)

    def tensors(p):
        codes = [torch.empty((p, 1, page, D // 2), dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.empty((p, 1, page // 16, D // 16, 16), dtype=torch.uint8, device=DEV) for _ in range(2)]
        return [codes[0], scales[0], codes[1], scales[1]]

    big, small = tensors(pages), tensors(3)
    for x, y in zip(big, small):
        y.copy_(random_bytes(y.shape, g, 256 if y.dim() == 4 else 0x60))
        x[at] = y
    length = 2 * page + 777
    args = [torch.tensor([0, n], dtype=torch.int32, device=DEV), torch.tensor([length], dtype=torch.int32, device=DEV)]
    q, k = (torch.randn((n, h, D), generator=g, device=DEV).bfloat16() for h in (Hq, 1))
    got = []
    for t, table in ((big, at), (small, [0, 1, 2])):
        c = ple.KV4Cache(*t, one, one)
        where = (*args, torch.tensor([table], dtype=torch.int32, device=DEV))
        ple.ple_kv4_append(c, k, k, *where)
        got.append((*ple.ple_kv4_read(c, *where, n),
                    *ple.ple_kv4_attention(q, c, *where, max_request_tokens=n, max_seq_len=length, want_lse=True)))
    assert all(torch.equal(x, y) for x, y in zip(*got)) and torch.isfinite(got[0][2]).all()
    assert all(torch.equal(x[at], y) for x, y in zip(big, small))


@pytest.mark.gpu
@pytest.mark.parametrize("T,O,K,group", [(3, (1 << 20) + 40, 8320, 16), (100, (1 << 20) + 40, 8320, 128), (2100, (1 << 20) + 40, 64, 16),
                                         (2100, (1 << 20) + 40, 64, 32)])
def test_weights_and_outputs_of_more_than_4_gib(T, O, K, group):
    """The last features (and tokens) of a weight of 4.4 GB, and of an output of 4.4 GB."""
    g = torch.Generator(device=DEV).manual_seed(43)
    codes = random_bytes((O, K // 2), g)
    x = torch.randn((T, K), generator=g, device=DEV).bfloat16()
    if group == 16:
        scales = random_bytes((O, K // 16), g, 0x60)
        w = ple.W4Weight.nvfp4(codes, scales, torch.ones(1, device=DEV))
    else:
        scales = torch.randn((O, K // group), generator=g, device=DEV).bfloat16()
        w = ple.W4Weight.int4(codes, scales)
    out = ple.ple_w4_linear(x, w)
    tail = slice(O - 100, O)
    if group == 16:
        W = U.e2m1(codes[tail].cpu()) * U.e4m3(scales[tail].cpu()).repeat_interleave(16, -1)
    else:
        W = (U.nibbles(codes[tail].cpu()).double() - 8) * scales[tail].cpu().double().repeat_interleave(group, -1)
    x = x[-100:].cpu().double()
    want, most = x @ W.t(), x.abs() @ W.abs().t()
    # fp32 sums: (K + 8) roundings of at most 2^-23 of the sum of magnitudes; then bf16's 2^-8
    acc = (K + 8) * 2.0 ** -23 * most
    assert ((out[-100:, tail].cpu().double() - want).abs() <= 2.0 ** -8 * (want.abs() + acc) + acc).all()


@pytest.mark.gpu
def test_queries_and_outputs_of_more_than_4_gib():
    """A decode step of 2^19 + 5 requests of 1 .. 40 tokens, 32 heads of 128: its last rows are those of a call of their
    own."""
    T, Hq, D, page, last = (1 << 19) + 5, 32, 128, 64, 300
    g = torch.Generator(device=DEV).manual_seed(44)
    one = torch.full((1,), 0.02, device=DEV)
    codes = [random_bytes((64, 1, page, D // 2), g) for _ in range(2)]
    scales = [random_bytes((64, 1, page // 16, D // 16, 16), g, 0x60) for _ in range(2)]
    c = ple.KV4Cache(codes[0], scales[0], codes[1], scales[1], one, one)
    q = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    seq = torch.randint(1, 41, (T,), dtype=torch.int32, device=DEV, generator=g)
    table = torch.randint(0, 64, (T, 1), dtype=torch.int32, device=DEV, generator=g)
    qsl = torch.arange(T + 1, dtype=torch.int32, device=DEV)
    kw = dict(max_request_tokens=1, max_seq_len=40, want_lse=True)
    out, lse = ple.ple_kv4_attention(q, c, qsl, seq, table, **kw)
    own, own_lse = ple.ple_kv4_attention(q[-last:], c, qsl[:last + 1], seq[-last:].clone(), table[-last:].clone(), **kw)
    assert torch.equal(out[-last:], own) and torch.equal(lse[-last:], own_lse) and torch.isfinite(own).all()
