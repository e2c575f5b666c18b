"""What the 8-bit operators refuse, without a GPU: the C entry points with addresses that are never touched, and the
Python binding with a library that must not be called."""
import ctypes

import pytest
import torch

import layer_embedding_lookup_amd as ple
from layer_embedding_lookup_amd import capi

lib = capi.load()
E_ARG, E_UNSUP, E_WS, OK = capi.PLE_ERR_INVALID_ARGUMENT, capi.PLE_ERR_UNSUPPORTED, capi.PLE_ERR_WORKSPACE, capi.PLE_OK
FAKE = 1 << 40
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="made-up addresses stay off hosts with a GPU")
BF, I8, I32, U8 = torch.bfloat16, torch.int8, torch.int32, torch.uint8


def weight(codes=FAKE, scales=FAKE, O=64, K=128):
    return ctypes.byref(capi.ple_w8_weight(codes, scales, O, K))


def cache(kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, pages=10, H=2, page=16, D=128):
    return ctypes.byref(capi.ple_kv8_cache(kc, ks, vc, vs, pages, H, page, D, 0))


def batch(qsl=FAKE, seq=FAKE, table=FAKE, T=4, R=2, width=5, new=0, most=0):
    return ctypes.byref(capi.ple_kv4_batch(qsl, seq, table, T, R, width, new, most))


def test_exports_every_header_function():
    names = capi.header_functions(capi.BITS8_HEADER)
    assert set(names) == set(capi._BITS8_PROTOS)
    for n in names:
        assert hasattr(lib, n)


@no_gpu
def test_norm_rejects():
    def call(x=FAKE, stride=128, res=None, w=FAKE, T=4, n=128, eps=1e-6, codes=FAKE, scales=FAKE, out=None):
        return lib.ple_rms_norm8(x, stride, res, w, T, n, eps, codes, scales, out, None)
    for n in (0, 8, 24, 131072, -16):
        assert call(n=n) == E_UNSUP
    for kw in (dict(x=None), dict(x=FAKE + 2), dict(stride=120), dict(stride=132), dict(stride=-128), dict(T=-1), dict(T=1 << 25),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(w=None), dict(w=FAKE + 8),
               dict(codes=None), dict(codes=FAKE + 4), dict(scales=None), dict(scales=FAKE + 2), dict(res=FAKE), dict(out=FAKE),
               dict(res=FAKE + 2, out=FAKE), dict(res=FAKE, out=FAKE + 8), dict(res=FAKE + 4096, out=FAKE, stride=136)):
        assert call(**kw) == E_ARG, kw
    assert call(T=0, x=None, w=None, codes=None, scales=None) == OK


@no_gpu
def test_linear_rejects():
    def call(w, x=FAKE, stride=128, xs=FAKE, T=4, out=FAKE):
        return lib.ple_w8_linear(x, stride, xs, w, T, out, None)
    assert call(None) == E_ARG
    for K in (0, 8, 40, 131072, -16):
        assert call(weight(K=K)) == E_UNSUP
    for w in (weight(O=0), weight(O=(1 << 24) + 1), weight(codes=None), weight(codes=FAKE + 8), weight(scales=None),
              weight(scales=FAKE + 2)):
        assert call(w) == E_ARG
    for kw in (dict(x=None), dict(x=FAKE + 8), dict(stride=112), dict(stride=136), dict(stride=(1 << 22) + 16), dict(xs=None),
               dict(xs=FAKE + 1), dict(T=-1), dict(T=1 << 25), dict(out=None), dict(out=FAKE + 8)):
        assert call(weight(), **kw) == E_ARG, kw
    assert call(weight(O=1 << 24), T=1 << 24) == E_UNSUP
    assert call(weight(), T=0, x=None, xs=None, out=None) == OK


@no_gpu
def test_cache_calls_reject():
    def append(c=cache(), b=batch(), k=FAKE, ks=256, v=FAKE, vs=256, q=None, qs=0, hq=0, qo=None, f=None, rot=0):
        return lib.ple_kv8_append(c, b, k, ks, v, vs, q, qs, hq, qo, f, rot, 0, None)
    for c in (cache(D=96), cache(D=512), cache(page=8), cache(page=24), cache(page=1 << 17), cache(pages=0), cache(pages=1 << 30),
              cache(pages=1 << 40)):
        assert append(c) == E_UNSUP
    for c in (None, cache(H=0), cache(H=1025), cache(kc=None), cache(vc=FAKE + 4), cache(ks=None), cache(vs=FAKE + 1)):
        assert append(c) == E_ARG
    for b in (None, batch(T=-1), batch(T=1 << 25), batch(R=-1), batch(R=0), batch(new=-1), batch(most=-1), batch(qsl=None), batch(seq=FAKE + 2),
              batch(table=None)):
        assert append(b=b) == E_ARG
    assert append(b=batch(width=0)) == E_UNSUP and append(b=batch(width=1 << 27)) == E_UNSUP
    for kw in (dict(k=None), dict(k=FAKE + 2), dict(ks=248), dict(ks=260), dict(v=None), dict(vs=0), dict(q=FAKE), dict(qo=FAKE),
               dict(q=FAKE, qo=FAKE + 256, hq=3, qs=512), dict(q=FAKE, qo=FAKE, hq=4, qs=512), dict(q=FAKE, qo=FAKE + 256, hq=4, qs=256),
               dict(rot=32), dict(rot=32, f=FAKE + 2)):
        assert append(**kw) == E_ARG, kw
    assert append(rot=24, f=FAKE) == E_UNSUP and append(rot=256, f=FAKE) == E_UNSUP and append(rot=-16, f=FAKE) == E_UNSUP
    # 2 * 2^31 blocks of 16 tokens, 512 parts each, are more than a launch holds
    most = cache(H=1024)
    assert append(most, batch(R=(1 << 31) - 1), ks=1 << 17, vs=1 << 17) == E_UNSUP
    assert lib.ple_kv8_read(most, batch(R=(1 << 31) - 1), FAKE, FAKE, None) == E_UNSUP
    assert append(b=batch(T=0, R=0), k=None, v=None) == OK
    assert lib.ple_kv8_read(cache(), batch(), None, FAKE, None) == E_ARG
    assert lib.ple_kv8_read(cache(), batch(), FAKE, FAKE + 8, None) == E_ARG
    assert lib.ple_kv8_read(cache(), batch(T=0), None, None, None) == OK


@no_gpu
def test_attention_rejects():
    def call(q=FAKE, qs=512, hq=4, c=cache(), b=batch(), window=0, scale=0.1, out=FAKE, lse=None, ws=None, nws=0):
        return lib.ple_kv8_attention(q, qs, hq, c, b, window, scale, out, lse, ws, nws, None)
    for kw in (dict(q=None), dict(q=FAKE + 4), dict(qs=504), dict(qs=516), dict(hq=3), dict(hq=0), dict(hq=2048), dict(window=-1), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None), dict(lse=FAKE + 2), dict(c=None), dict(b=None)):
        assert call(**kw) == E_ARG, kw
    long = batch(T=1, R=1, width=10000, new=1)
    need = lib.ple_kv8_attention_workspace_bytes(4, cache(), long, 0)
    assert need > 0
    assert call(b=long) == E_ARG
    assert call(b=long, ws=FAKE, nws=need - 1) == E_WS
    assert call(b=long, ws=FAKE + 4, nws=need) == E_ARG
    assert call(b=batch(T=0), q=None, out=None) == OK
    assert call(b=batch(T=1 << 24, R=1 << 20), c=cache(H=2)) == E_UNSUP  # no hint: too many query tiles


def test_workspace_sizes():
    f = lib.ple_kv8_attention_workspace_bytes
    assert f(4, cache(D=96), batch(), 0) == 0 and f(4, cache(), batch(T=0), 0) == 0
    assert f(4, cache(), batch(T=1, R=1, new=1, most=64), 0) == 0  # one split
    a = f(8, cache(), batch(T=1, R=1, width=10000, new=1), 0)
    # a window bounds what there is to split
    assert 0 <= f(8, cache(), batch(T=1, R=1, width=10000, new=1), 128) < a


@pytest.fixture
def no_library(monkeypatch):
    class Stub:
        def __getattr__(self, name):
            raise AssertionError(f"the binding called {name} before rejecting the arguments")
    stub = Stub()
    monkeypatch.setattr(capi, "load", lambda: stub)


class _W:
    k_dim, out_dim, codes, desc, device = 128, 64, None, None, -1


def test_binding_rejects(no_library):
    x, w = torch.zeros((4, 128), dtype=BF), torch.zeros(128, dtype=BF)
    for bad in (torch.zeros((4, 128)), torch.zeros((4, 128, 1), dtype=BF), torch.zeros((128, 4), dtype=BF).t()):
        with pytest.raises(ValueError, match="x must be bf16"):
            ple.ple_rms_norm8(bad, w)
    for kw, what in ((dict(weight=w[:64]), "weight has shape"), (dict(residual=x[:2]), "residual has shape"),
                     (dict(residual_out=x), "residual_out given without"), (dict(codes=torch.zeros((4, 128), dtype=U8)), "codes has dtype"),
                     (dict(scales=torch.zeros(5)), "scales has shape"), (dict(residual=x, residual_out=x.float()), "residual_out has dtype"),
                     (dict(), "GPU tensors"), (dict(residual=x), "GPU tensors")):
        with pytest.raises(ValueError, match=what):
            ple.ple_rms_norm8(x, **{"weight": w, **kw})
    codes = torch.zeros((8, 64), dtype=I8)
    with pytest.raises(ValueError, match="codes has dtype"):
        ple.W8Weight(codes.view(U8), torch.zeros(8))
    with pytest.raises(ValueError, match="scales has shape"):
        ple.W8Weight(codes, torch.zeros(9))
    with pytest.raises(ValueError, match="GPU tensors"):
        ple.W8Weight(codes, torch.zeros(8))
    i8 = torch.zeros((4, 128), dtype=I8)
    for bad in (i8[:, :64], i8.view(U8), torch.zeros((128, 4), dtype=I8).t()):
        with pytest.raises(ValueError, match="x must be int8"):
            ple.ple_w8_linear(bad, torch.zeros(4), _W)
    with pytest.raises(ValueError, match="x_scales has shape"):
        ple.ple_w8_linear(i8, torch.zeros(3), _W)
    with pytest.raises(ValueError, match="out has shape"):
        ple.ple_w8_linear(i8, torch.zeros(4), _W, out=torch.zeros((4, 65), dtype=BF))
    kc, vc, s = torch.zeros((4, 2, 3, 8, 16, 16), dtype=U8), torch.zeros((4, 2, 3, 128, 16), dtype=U8), torch.zeros((4, 2, 3))
    for args, what in (((kc[:, :, :, :, :8], s, vc, s), "k_codes has shape"), ((kc, s, vc[:, :, :, :64], s), "v_codes has shape"),
                       ((kc, s[:, :, :2], vc, s), "k_scales has shape"), ((kc, s, vc, s.to(BF)), "v_scales has dtype"),
                       ((kc, s, vc, s), "GPU tensors"), ((kc.float(), s, vc, s), "k_codes has dtype")):
        with pytest.raises(ValueError, match=what):
            ple.KV8Cache(*args)
    c = object.__new__(ple.KV8Cache)
    c.tensors, c.device = (kc,), 0
    c.num_pages, c.num_kv_heads, c.page_size, c.head_dim = 4, 2, 48, 128
    k = torch.zeros((3, 2, 128), dtype=BF)
    qsl, seq, table = torch.zeros(2, dtype=I32), torch.zeros(1, dtype=I32), torch.zeros((1, 3), dtype=I32)
    for bad in (torch.zeros((3, 1, 128), dtype=BF), torch.zeros((2, 2, 128), dtype=BF), torch.zeros((3, 2, 64), dtype=BF),
                torch.zeros((3, 128, 2), dtype=BF).transpose(1, 2), torch.zeros((3, 2, 128))):
        with pytest.raises(ValueError, match="^v "):
            ple.ple_kv8_append(c, k, bad, qsl, seq, table)
    with pytest.raises(ValueError, match="q_out given without q"):
        ple.ple_kv8_append(c, k, k, qsl, seq, table, q_out=k)
    with pytest.raises(ValueError, match="seq_lens has shape"):
        ple.ple_kv8_append(c, k, k, qsl, torch.zeros(2, dtype=I32), table)
    with pytest.raises(ValueError, match="GPU tensors"):
        ple.ple_kv8_append(c, k, k, qsl, seq, table)
    with pytest.raises(ValueError, match="k_out has shape"):
        ple.ple_kv8_read(c, qsl, seq, table, 3, k_out=k[:2], v_out=k)
    with pytest.raises(ValueError, match="lse has dtype"):
        ple.ple_kv8_attention(k, c, qsl, seq, table, lse=torch.zeros((3, 2), dtype=BF))
