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


@pytest.mark.parametrize("D,Hq,n,extra,window", [(128, 4, 10, 6, 0), (64, 2, 3, 2, 0), (128, 2, 10, 6, 8), (128, 8, 40, 30, 0),
                                                 (256, 4, 40, 30, 16), (128, 4, 10, 40, 8), (64, 8, 60, 70, 32)])
def test_sequences_longer_than_the_table(D, Hq, n, extra, window):
    """A sequence of `extra` tokens more than the 64 that its table row covers: the tokens past it stand on no page, the
    others keep their positions."""
    g = torch.Generator().manual_seed(n + extra)
    lens = [64 + extra, 64]
    cache = U.Cache(g, lens, H=1, D=D, page=16, poison=False)
    cache.table[:, 4:] = -7                                    # (the definition's table: these pages do not exist)
    qsl, seq = torch.tensor([0, n, n + 1], dtype=I32), torch.tensor(lens, dtype=I32)
    q, k = (torch.randn((n + 1, h, D), generator=g).to(BF) for h in (Hq, 1))
    dev, c, args = tensors(cache, qsl, seq, cache.table[:, :4].contiguous())
    out, lse = ple.ple_kv4_attention(q.to(DEV), c, *args, window=window, want_lse=True)
    want, want_lse, tol, tol_lse = U.attention(cache, q, qsl, seq, window)
    empty = want_lse == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, empty) and (out.cpu()[empty] == 0).all()
    assert ((out.cpu().to(F64) - want).abs() <= tol).all()
    assert ((lse.cpu().to(F64) - want_lse).abs() <= tol_lse)[~empty].all()
    ple.ple_kv4_append(c, k.to(DEV), k.to(DEV), *args)
    got, _ = ple.ple_kv4_read(c, *args, n + 1)
    stored = torch.cat((lens[0] - n + torch.arange(n) < 64, torch.tensor([True])))
    assert (got.cpu()[~stored] == 0).all() and (got.cpu()[stored].flatten(1) != 0).any(1).all()
    codes, _ = U.quantise(k.float(), cache.scale["k"][:, None])
    for t in range(n):
        p = lens[0] - n + t
        if p < 64:
            assert torch.equal(dev[0].cpu()[int(cache.table[0, p // 16]), :, p % 16], codes[t])


@pytest.mark.parametrize("n,T", [(10, 6), (100, 70), (64, 1)])
def test_requests_longer_than_the_call(n, T):
    """query_start_loc that runs past T: the tokens that are there stand where they would in the whole request."""
    g = torch.Generator().manual_seed(n)
    cache = U.Cache(g, [200], H=2, D=128, page=16)
    qsl, seq = torch.tensor([0, n], dtype=I32), torch.tensor([200], dtype=I32)
    q = torch.randn((n, 4, 128), generator=g).to(BF)
    _, c, args = tensors(cache, qsl, seq, cache.table)
    out, lse = ple.ple_kv4_attention(q[:T].to(DEV), c, *args, want_lse=True)
    want, want_lse, tol, tol_lse = U.attention(cache, q, qsl, seq)
    assert ((out.cpu().to(F64) - want[:T]).abs() <= tol[:T]).all()
    assert ((lse.cpu().to(F64) - want_lse[:T]).abs() <= tol_lse[:T]).all()


def test_lengths_at_the_ends_of_their_type():
    g = torch.Generator().manual_seed(3)
    lens = [40, -2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1]
    cache = U.Cache(g, [40, 0, 0, 48], H=1, D=64, page=16)
    qsl = [0, 1, 3, 4, 44]
    q = torch.randn((44, 2, 64), generator=g).to(BF).to(DEV)
    _, c, args = tensors(cache, qsl, lens, cache.table)
    for window in (0, 7, 2 ** 30 - 1):
        out, lse = ple.ple_kv4_attention(q, c, *args, window=window, want_lse=True)
        assert (out[1:4] == 0).all() and (lse[1:4] == -math.inf).all()
        # request 3 stands far past its 48 tokens: its rows see all of them without a window, none with one
        assert torch.isfinite(out).all() and ((lse[4:] == -math.inf) == (window > 0)).all()
        want, want_lse, tol, tol_lse = U.attention(cache, q[:1].cpu(), [0, 1], [40], window)
        assert ((out[:1].cpu().to(F64) - want).abs() <= tol).all()


@pytest.mark.parametrize("qsl", [[-2 ** 31, 3, 5], [0, -2 ** 31, 5], [5, 2, 2 ** 31 - 1], [2 ** 31 - 1, 0, -2 ** 31]])
def test_broken_offsets_stay_in_bounds(qsl):
    """Offsets at the ends of their type and falling ones: results are unspecified, what surrounds the outputs and the
    cache's other tensors stays."""
    g = torch.Generator().manual_seed(8)
    cache = U.Cache(g, [90, 30], H=1, D=64, page=16)
    q = torch.randn((5, 2, 64), generator=g).to(BF).to(DEV)
    for hint in (0, 1):
        _, c, args = tensors(cache, qsl, [90, 30], cache.table)
        out, lse = torch.full((15, 2, 64), 7, dtype=BF, device=DEV), torch.full((16, 2), 7.0, device=DEV)
        ple.ple_kv4_attention(q, c, *args, max_request_tokens=hint, out=out[5:10], lse=lse[4:9])
        assert (out[:5] == 7).all() and (out[10:] == 7).all() and (lse[:4] == 7).all() and (lse[9:] == 7).all()
        ple.ple_kv4_read(c, *args, 5, k_out=(k := torch.full((15, 1, 64), 7, dtype=BF, device=DEV))[5:10], v_out=k.clone()[5:10])
        assert (k[:5] == 7).all() and (k[10:] == 7).all()
