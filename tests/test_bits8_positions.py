"""Where new tokens stand in the 8-bit cache: tokens of no request (a batch padded to a graph's size), sequences longer
than the page table covers and requests longer than the call, the same for append, read and attention."""
import math

import pytest
import torch

import bits8_util as U
import layer_embedding_lookup_amd as ple

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F64, BF, I32 = torch.float64, torch.bfloat16, torch.int32


def tensors(cache, qsl, seq, table):
    dev = cache.tensors(DEV)
    return dev, ple.KV8Cache(*dev), tuple(torch.as_tensor(t, dtype=I32).to(DEV) for t in (qsl, seq, table))


def same(a, b):
    """The same bytes (scales of blocks without tokens may be NaN)."""
    return all(torch.equal(x.cpu().contiguous().view(torch.uint8), y.cpu().contiguous().view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("hint", [False, True])
@pytest.mark.parametrize("qsl,T", [([0, 2, 3], 7), ([4, 5, 5, 6], 6), ([3, 4, 6], 40), ([0, 0, 0], 5), ([30, 67], 200)])
def test_tokens_of_no_request(qsl, T, hint):
    """Append stores nothing for them (the table's unused entries name a page of another request) and leaves queries as they
    are, read gives zeros; the requests' own tokens are as in a call without them."""
    g = torch.Generator().manual_seed(T)
    R, a, b = len(qsl) - 1, qsl[0], qsl[-1]
    lens = [16 * (r + 1) + (b - a) // 16 * 16 for r in range(R)]  # the next place lies on the next page
    cache = U.Cache(g, lens, H=2, D=128, page=16)
    table = torch.where(cache.table < 0, cache.table[0, 0], cache.table)
    before = cache.tensors("cpu")
    q, k = (torch.randn((T, h, 128), generator=g).to(BF).to(DEV) for h in (4, 2))
    inv = torch.logspace(0, -4, 64).to(DEV)
    most = max(y - x for x, y in zip(qsl, qsl[1:])) if hint else 0
    dev, c, args = tensors(cache, qsl, lens, table)
    out_q = ple.ple_kv8_append(c, k, k, *args, inv_freq=inv, q=q, max_request_tokens=most)
    only, oc, own = tensors(cache, [x - a for x in qsl], lens, table)
    own_q = ple.ple_kv8_append(oc, k[a:b], k[a:b], *own, inv_freq=inv, q=q[a:b])
    assert same(dev, only)
    if a == b:
        assert same(dev, before)
    idle = [t for t in range(T) if t < a or t >= b]
    assert torch.equal(out_q[a:b], own_q) and torch.equal(out_q[idle], q[idle])
    for x, y in zip(ple.ple_kv8_read(c, *args, T), ple.ple_kv8_read(oc, *own, b - a)):
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
    ple.ple_kv8_attention(q, c, *args, max_request_tokens=hint, max_seq_len=max(lens), out=out, lse=lse)
    idle = [t for t in range(T) if t < qsl[0] or t >= qsl[-1]]
    assert (out[idle] == 0).all() and (lse[idle] == -math.inf).all()
    want, want_lse, tol, tol_lse = U.attention(cache, q.cpu(), qsl, torch.tensor(lens))
    a, b = qsl[0], qsl[-1]
    assert ((out.cpu().to(F64) - want).abs() <= tol)[a:b].all()
    assert ((lse.cpu().to(F64) - want_lse).abs() <= tol_lse)[a:b].all()
    out.fill_(math.nan)
    ple.ple_kv8_attention(q, c, *args, max_request_tokens=hint, max_seq_len=max(lens), out=out)
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
    out, lse = ple.ple_kv8_attention(q.to(DEV), c, *args, window=window, want_lse=True)
    want, want_lse, tol, tol_lse = U.attention(cache, q, qsl, seq, window)
    empty = want_lse == -math.inf
    assert torch.equal(lse.cpu() == -math.inf, empty) and (out.cpu()[empty] == 0).all()
    assert ((out.cpu().to(F64) - want).abs() <= tol).all()
    assert ((lse.cpu().to(F64) - want_lse).abs() <= tol_lse)[~empty].all()
    ple.ple_kv8_append(c, k.to(DEV), k.to(DEV), *args)
    got, _ = ple.ple_kv8_read(c, *args, n + 1)
    stored = torch.cat((lens[0] - n + torch.arange(n) < 64, torch.tensor([True])))
    assert (got.cpu()[~stored] == 0).all() and (got.cpu()[stored].flatten(1) != 0).any(1).all()
    before = {"k": cache.codes["k"].clone()}
    places = [(r, j) for r, m in ((0, n), (1, 1)) for j in range(lens[r] - m, lens[r]) if j < 64]
    new = cache.append("k", k.to(F64), qsl, seq)
    assert len(new) == len(places) == int(stored.sum())
    after = U.Cache.__new__(U.Cache)
    after.__dict__.update(cache.__dict__)
    after.take(*dev)
    live = torch.zeros(before["k"].shape[:3], dtype=torch.bool)
    for page, place, x in new:  # (no rotation: the quotients are exact)
        live[page, :, place] = True
        assert torch.equal(after.codes["k"][page, :, place], U.codes_of(x))
    assert torch.equal(after.codes["k"][~live], cache.codes["k"][~live])
    assert torch.equal(after.scales["k"], cache.scales["k"])


@pytest.mark.parametrize("n,T", [(10, 6), (100, 70), (64, 1)])
def test_requests_longer_than_the_call(n, T):
    """query_start_loc that runs past T: the tokens that are there stand where they would in the whole request."""
    g = torch.Generator().manual_seed(n)
    cache = U.Cache(g, [200], H=2, D=128, page=16)
    qsl, seq = torch.tensor([0, n], dtype=I32), torch.tensor([200], dtype=I32)
    q, k = (torch.randn((n, h, 128), generator=g).to(BF) for h in (4, 2))
    dev, c, args = tensors(cache, qsl, seq, cache.table)
    out, lse = ple.ple_kv8_attention(q[:T].to(DEV), c, *args, want_lse=True)
    want, want_lse, tol, tol_lse = U.attention(cache, q, qsl, seq)
    assert ((out.cpu().to(F64) - want[:T]).abs() <= tol[:T]).all()
    assert ((lse.cpu().to(F64) - want_lse[:T]).abs() <= tol_lse[:T]).all()
    ple.ple_kv8_append(c, k[:T].to(DEV), k[:T].to(DEV), *args)
    short, _, own = tensors(cache, [0, T], [200 - n + T], cache.table)
    ple.ple_kv8_append(ple.KV8Cache(*short), k[:T].to(DEV), k[:T].to(DEV), *own)
    assert same(dev, short)


def test_lengths_at_the_ends_of_their_type():
    g = torch.Generator().manual_seed(3)
    lens = [40, -2 ** 31, 2 ** 31 - 1, 2 ** 31 - 1]
    cache = U.Cache(g, [40, 0, 0, 48], H=1, D=64, page=16)
    qsl = [0, 1, 3, 4, 44]
    q = torch.randn((44, 2, 64), generator=g).to(BF).to(DEV)
    dev, c, args = tensors(cache, qsl, lens, cache.table)
    for window in (0, 7, 2 ** 30 - 1):
        out, lse = ple.ple_kv8_attention(q, c, *args, window=window, want_lse=True)
        assert (out[1:4] == 0).all() and (lse[1:4] == -math.inf).all()
        # request 3 stands far past its 48 tokens: its rows see all of them without a window, none with one
        assert torch.isfinite(out).all() and ((lse[4:] == -math.inf) == (window > 0)).all()
        want, want_lse, tol, tol_lse = U.attention(cache, q[:1].cpu(), [0, 1], [40], window)
        assert ((out[:1].cpu().to(F64) - want).abs() <= tol).all()
    before = cache.tensors("cpu")
    k = torch.randn((43, 1, 64), generator=g).to(BF).to(DEV)
    where = (args[0][1:] - 1, args[1][1:].contiguous(), args[2][1:].contiguous())
    ple.ple_kv8_append(c, k, k, *where)                        # none of these stands on a place
    assert same(dev, before)
    assert all((x == 0).all() for x in ple.ple_kv8_read(c, *where, 43))


@pytest.mark.parametrize("qsl", [[-2 ** 31, 3, 5], [0, -2 ** 31, 5], [5, 2, 2 ** 31 - 1], [2 ** 31 - 1, 0, -2 ** 31]])
def test_broken_offsets_stay_in_bounds(qsl):
    """Offsets at the ends of their type and falling ones: results are unspecified, what surrounds the outputs and the
    cache's tensors stays."""
    g = torch.Generator().manual_seed(8)
    cache = U.Cache(g, [90, 30], H=1, D=64, page=16)
    q, k = (torch.randn((5, h, 64), generator=g).to(BF).to(DEV) for h in (2, 1))
    for hint in (0, 1):
        _, _, args = tensors(cache, qsl, [90, 30], cache.table)
        around = [torch.full((t.shape[0] + 2, *t.shape[1:]), 7, dtype=t.dtype, device=DEV) for t in cache.tensors("cpu")]
        for x, y in zip(around, cache.tensors(DEV)):
            x[1:-1] = y
        c = ple.KV8Cache(*(x[1:-1] for x in around))
        out, lse = torch.full((15, 2, 64), 7, dtype=BF, device=DEV), torch.full((16, 2), 7.0, device=DEV)
        ple.ple_kv8_attention(q, c, *args, max_request_tokens=hint, out=out[5:10], lse=lse[4:9])
        assert (out[:5] == 7).all() and (out[10:] == 7).all() and (lse[:4] == 7).all() and (lse[9:] == 7).all()
        ko, vo = (torch.full((15, 1, 64), 7, dtype=BF, device=DEV) for _ in range(2))
        ple.ple_kv8_read(c, *args, 5, k_out=ko[5:10], v_out=vo[5:10])
        assert all((x[:5] == 7).all() and (x[10:] == 7).all() for x in (ko, vo))
        ple.ple_kv8_append(c, k, k, *args, max_request_tokens=hint)
        assert all((x[0] == 7).all() and (x[-1] == 7).all() for x in around)
