"""What the 4-bit operators refuse, without a GPU: the C entry points with addresses that are never touched, the Python
binding with a library that must not be called, and the page lookup compiled for the host."""
import ctypes
import os
import subprocess

import pytest
import torch

import layer_embedding_lookup_amd as ple
from layer_embedding_lookup_amd import build as B
from layer_embedding_lookup_amd import capi

lib = capi.load()
E_ARG, E_UNSUP, E_WS, OK = capi.PLE_ERR_INVALID_ARGUMENT, capi.PLE_ERR_UNSUPPORTED, capi.PLE_ERR_WORKSPACE, capi.PLE_OK
FAKE = 1 << 40
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="made-up addresses stay off hosts with a GPU")


def weight(fmt=capi.PLE_W4_NVFP4, O=64, K=128, G=16, codes=FAKE, scales=FAKE, zeros=None, ts=FAKE):
    return ctypes.byref(capi.ple_w4_weight(codes, scales, zeros, ts, fmt, O, K, G))


def cache(kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, kg=FAKE, vg=FAKE, pages=10, H=2, page=16, D=128):
    return ctypes.byref(capi.ple_kv4_cache(kc, ks, vc, vs, kg, vg, pages, H, page, D, 0))


def batch(qsl=FAKE, seq=FAKE, table=FAKE, T=4, R=2, width=5, new=0, most=0):
    return ctypes.byref(capi.ple_kv4_batch(qsl, seq, table, T, R, width, new, most))


def test_exports_every_header_function():
    names = capi.header_functions(capi.FP4_HEADER)
    assert set(names) == set(capi._FP4_PROTOS)
    for n in names:
        assert hasattr(lib, n)


@no_gpu
def test_linear_rejects():
    def call(w, x=FAKE, stride=128, T=4, out=FAKE):
        return lib.ple_w4_linear(x, stride, w, T, out, None)
    INT4 = capi.PLE_W4_INT4
    assert call(None) == E_ARG
    for w in (weight(fmt=2), weight(G=32), weight(K=48), weight(fmt=INT4, G=16, ts=None), weight(fmt=INT4, G=128, K=192, ts=None)):
        assert call(w) == E_UNSUP
    for w in (weight(O=0), weight(K=0), weight(K=(1 << 20) + 32), weight(codes=None), weight(codes=FAKE + 8),
              weight(scales=None), weight(scales=FAKE + 1), weight(ts=None), weight(ts=FAKE + 2), weight(zeros=FAKE),
              weight(fmt=INT4, G=32)):
        assert call(w) == E_ARG
    for kw in (dict(x=None), dict(x=FAKE + 2), dict(stride=120), dict(stride=132), dict(T=-1), dict(T=1 << 25), dict(out=None),
               dict(out=FAKE + 8)):
        assert call(weight(), **kw) == E_ARG
    assert call(weight(O=1 << 24), T=1 << 24) == E_UNSUP
    assert call(weight(), T=0, x=None, out=None) == OK


@no_gpu
def test_cache_calls_reject():
    def append(c=cache(), b=batch(), k=FAKE, ks=256, v=FAKE, vs=256, q=None, qs=0, hq=0, qo=None, f=None, rot=0):
        return lib.ple_kv4_append(c, b, k, ks, v, vs, q, qs, hq, qo, f, rot, 0, None)
    for c in (cache(D=96), cache(D=512), cache(page=8), cache(page=24), cache(page=1 << 17), cache(pages=0), cache(pages=1 << 30),
              cache(pages=1 << 40)):
        assert append(c) == E_UNSUP
    for c in (None, cache(H=0), cache(H=1025), cache(kc=None), cache(vs=FAKE + 4), cache(kg=None), cache(vg=FAKE + 1)):
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
    assert append(b=batch(T=0, R=0), k=None, v=None) == OK
    assert lib.ple_kv4_read(cache(), batch(), None, FAKE, None) == E_ARG
    assert lib.ple_kv4_read(cache(), batch(), FAKE, FAKE + 8, None) == E_ARG
    assert lib.ple_kv4_read(cache(), batch(T=0), None, None, None) == OK


@no_gpu
def test_attention_rejects():
    def call(q=FAKE, qs=512, hq=4, c=cache(), b=batch(), window=0, scale=0.1, out=FAKE, lse=None, ws=None, nws=0):
        return lib.ple_kv4_attention(q, qs, hq, c, b, window, scale, out, lse, ws, nws, None)
    for kw in (dict(q=None), dict(q=FAKE + 4), dict(qs=504), dict(qs=516), dict(hq=3), dict(hq=0), dict(hq=2048), dict(window=-1), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None), dict(lse=FAKE + 2), dict(c=None), dict(b=None)):
        assert call(**kw) == E_ARG, kw
    long = batch(T=1, R=1, width=10000, new=1)
    need = lib.ple_kv4_attention_workspace_bytes(4, cache(), long, 0)
    assert need > 0
    assert call(b=long) == E_ARG
    assert call(b=long, ws=FAKE, nws=need - 1) == E_WS
    assert call(b=long, ws=FAKE + 4, nws=need) == E_ARG
    assert call(b=batch(T=0), q=None, out=None) == OK
    assert call(b=batch(T=1 << 24, R=1 << 20), c=cache(H=2)) == E_UNSUP  # no hint: too many query tiles


def test_workspace_sizes():
    f = lib.ple_kv4_attention_workspace_bytes
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


def _view(pages=4, H=2, page=16, D=128):
    """A cache object over host tensors (built without its device check)."""
    c = object.__new__(ple.KV4Cache)
    c.tensors = (torch.zeros((pages, H, page, D // 2), dtype=torch.uint8),)
    c.device, c._workspaces = 0, {}
    c.num_pages, c.num_kv_heads, c.page_size, c.head_dim = pages, H, page, D
    return c


def test_binding_rejects(no_library):
    u8, bf, f32, i32 = torch.uint8, torch.bfloat16, torch.float32, torch.int32
    with pytest.raises(ValueError, match="block_scales has shape"):
        ple.W4Weight.nvfp4(torch.zeros((8, 64), dtype=u8), torch.zeros((8, 4), dtype=u8), torch.zeros(1))
    with pytest.raises(ValueError, match="codes has dtype"):
        ple.W4Weight.nvfp4(torch.zeros((8, 64)), torch.zeros((8, 8), dtype=u8), torch.zeros(1))
    with pytest.raises(ValueError, match="do not divide"):
        ple.W4Weight.int4(torch.zeros((8, 64), dtype=u8), torch.zeros((8, 3), dtype=bf))
    with pytest.raises(ValueError, match="zeros has shape"):
        ple.W4Weight.int4(torch.zeros((8, 64), dtype=u8), torch.zeros((8, 4), dtype=bf), torch.zeros((8, 2), dtype=u8))
    with pytest.raises(ValueError, match="GPU tensors"):
        ple.W4Weight.int4(torch.zeros((8, 64), dtype=u8), torch.zeros((8, 4), dtype=bf))
    for x in (torch.zeros((4, 64), dtype=bf), torch.zeros((4, 128)), torch.zeros((128, 4), dtype=bf).t()):
        with pytest.raises(ValueError, match="x must be bf16"):
            ple.ple_w4_linear(x, _W)
    with pytest.raises(ValueError, match="out has shape"):
        ple.ple_w4_linear(torch.zeros((4, 128), dtype=bf), _W, out=torch.zeros((4, 65), dtype=bf))
    codes, scales = torch.zeros((4, 2, 32, 64), dtype=u8), torch.zeros((4, 2, 2, 8, 16), dtype=u8)
    with pytest.raises(ValueError, match="v_scales has shape"):
        ple.KV4Cache(codes, scales, codes, scales[:, :, :1], torch.zeros(2), torch.zeros(2))
    with pytest.raises(ValueError, match="k_scale has dtype"):
        ple.KV4Cache(codes, scales, codes, scales, torch.zeros(2, dtype=bf), torch.zeros(2))
    with pytest.raises(ValueError, match="GPU tensors"):
        ple.KV4Cache(codes, scales, codes, scales, torch.zeros(2), torch.zeros(2))
    c = _view()
    k = torch.zeros((3, 2, 128), dtype=bf)
    qsl, seq, table = torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros((1, 3), dtype=i32)
    for bad in (torch.zeros((3, 1, 128), dtype=bf), torch.zeros((2, 2, 128), dtype=bf), torch.zeros((3, 2, 64), dtype=bf),
                torch.zeros((3, 128, 2), dtype=bf).transpose(1, 2), torch.zeros((3, 2, 128))):
        with pytest.raises(ValueError, match="^v "):
            ple.ple_kv4_append(c, k, bad, qsl, seq, table)
    with pytest.raises(ValueError, match="q_out given without q"):
        ple.ple_kv4_append(c, k, k, qsl, seq, table, q_out=k)
    with pytest.raises(ValueError, match="seq_lens has shape"):
        ple.ple_kv4_append(c, k, k, qsl, torch.zeros(2, dtype=i32), table)
    with pytest.raises(ValueError, match="page_table has dtype"):
        ple.ple_kv4_append(c, k, k, qsl, seq, table.long())
    with pytest.raises(ValueError, match="GPU tensors"):
        ple.ple_kv4_append(c, k, k, qsl, seq, table)
    with pytest.raises(ValueError, match="k_out has shape"):
        ple.ple_kv4_read(c, qsl, seq, table, 3, k_out=k[:2], v_out=k)
    with pytest.raises(ValueError, match="lse has dtype"):
        ple.ple_kv4_attention(k, c, qsl, seq, table, lse=torch.zeros((3, 2), dtype=bf))


def test_page_lookup_on_the_host(tmp_path):
    """kv4_group names the group of a valid entry and refuses every other, at page sizes that are no power of two too."""
    src = tmp_path / "lookup.cpp"
    src.write_text(r"""
#include "ple_fp4_launch.h"
#include <stdio.h>
int main() {
    int bad = 0;
    const int32_t table[6] = {3, -1, 7, 8, 2147483647, -2147483647 - 1};
    for (int page : {16, 48, 128}) {
        ple_kv4_cache c = {};
        c.num_pages = 8; c.num_kv_heads = 3; c.page_size = page; c.head_dim = 128;
        for (int t = 0; t < 6 * page; t += 16)
            for (int h = 0; h < 3; ++h) {
                const int e = table[t / page];
                const int want = e < 0 || e >= 8 ? -1 : (e * 3 + h) * (page / 16) + (t % page) / 16;
                bad += ple::kv4_group(c, table, h, t / 16) != want;
            }
    }
    printf("%d\n", bad);
    return bad != 0;
}
""")
    exe = tmp_path / "lookup"
    cmd = [B.hipcc(), "-x", "hip", f"--offload-arch={B.ARCH}", "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, str(src), "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0 and os.path.exists(exe), res.stderr
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip() == "0"
