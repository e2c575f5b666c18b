"""Where new tokens stand: tokens of no request (a batch padded to a graph's size), sequences longer than the page table
covers and requests longer than the call, the same for append, read and attention."""
import math

import pytest
import torch

import fp4_util as U
import layer_embedding_lookup_amd as ple

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F64, BF, I32 = torch.float64, torch.bfloat16, torch.int32


def tensors(cache, qsl, seq, table):
    dev = cache.tensors(DEV)
    return dev, ple.KV4Cache(*dev), tuple(torch.as_tensor(t, dtype=I32).to(DEV) for t in (qsl, seq, table))


def same_cache(dev, before):
    return all(torch.equal(a.cpu(), b) for a, b in zip(dev, before))


@pytest.mark.parametrize("qsl,T", [([0, 2, 3], 7), ([4, 5, 5, 6], 6), ([3, 4, 6], 40), ([0, 0, 0], 5)])
def test_tokens_of_no_request(qsl, T):
    """Append stores nothing for them (the table's unused entries name a page of another request), read gives zeros,
    attention zeros and -inf; the requests' own tokens are as in a call without them."""
    g = torch.Generator().manual_seed(T)
    R, a, b = len(qsl) - 1, qsl[0], qsl[-1]
    lens = [16 * (r + 1) for r in range(R)]                    # the next place lies on the next page
    cache = U.Cache(g, lens, H=2, D=128, page=16)
    table = torch.where(cache.table < 0, cache.table[0, 0], cache.table)
    before = cache.tensors("cpu")
    q, k = (torch.randn((T, h, 128), generator=g).to(BF).to(DEV) for h in (4, 2))
    inv = torch.logspace(0, -4, 64).to(DEV)
    dev, c, args = tensors(cache, qsl, lens, table)
    out_q = ple.ple_kv4_append(c, k, k, *args, inv_freq=inv, q=q)
    only, oc, own = tensors(cache, [x - a for x in qsl], lens, table)
    own_q = ple.ple_kv4_append(oc, k[a:b], k[a:b], *own, inv_freq=inv, q=q[a:b])
    assert all(torch.equal(x, y) for x, y in zip(dev, only))
    if a == b:
        assert same_cache(dev, before)
    idle = [t for t in range(T) if t < a or t >= b]
    assert torch.equal(out_q[a:b], own_q) and torch.equal(out_q[idle], q[idle])
    for x, y in zip(ple.ple_kv4_read(c, *args, T), ple.ple_kv4_read(oc, *own, b - a)):
        assert (x[idle] == 0).all() and torch.equal(x[a:b], y)


@pytest.mark.parametrize("D,Hq,H,qsl,lens,T,hint", [
    (128, 4, 2, [0, 1, 2], [300, 40], 9, 1), (64, 4, 1, [2, 3], [5000], 70, 1), (256, 2, 1, [1, 3, 3, 5], [90, 8, 33], 600, 2),
    (128, 8, 2, [5, 60, 200], [500, 140], 333, 140), (64, 2, 2, [7, 80], [73], 100, 73), (256, 4, 1, [0, 90], [300], 91, 90),
    (128, 2, 1, [3] + [3 + 20 * (i + 1) for i in range(65)], [20] * 65, 1310, 128), (128, 4, 4, [0, 0], [9], 33, 0)])
def test_attention_of_tokens_of_no_request(D, Hq, H, qsl, lens, T, hint):
    print(f"idle tokens D={D} Hq={Hq} H={H} T={T}", flush=True)
    g = torch.Generator().manual_seed(T + D)
    cache = U.Cache(g, lens, H=H, D=D, page=16)
    q = torch.randn((T, Hq, D), generator=g).to(BF).to(DEV)
    _, c, args = tensors(cache, qsl, lens, cache.table)
    out = torch.full((T, Hq, D), math.nan, dtype=BF, device=DEV)
    lse = torch.full((T, Hq), math.nan, device=DEV)
    ple.ple_kv4_attention(q, c, *args, max_request_tokens=hint, max_seq_len=max(lens), out=out, lse=lse)
    idle = [t for t in range(T) if t < qsl[0] or t >= qsl[-1]]
    assert (out[idle] == 0).all() and (lse[idle] == -math.inf).all()
    want, want_lse, tol, tol_lse = U.attention(cache, q.cpu(), qsl, torch.tensor(lens))
    a, b = qsl[0], qsl[-1]
    assert ((out.cpu().to(F64) - want).abs() <= tol)[a:b].all()
    assert ((lse.cpu().to(F64) - want_lse).abs() <= tol_lse)[a:b].all()
    out.fill_(math.nan)
    ple.ple_kv4_attention(q, c, *args, max_request_tokens=hint, max_seq_len=max(lens), out=out)
    assert (out[idle] == 0).all()
