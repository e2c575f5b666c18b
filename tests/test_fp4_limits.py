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
