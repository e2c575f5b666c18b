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
