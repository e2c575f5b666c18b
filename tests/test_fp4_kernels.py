"""Every kernel of the 4-bit products and of the attention, by shapes that reach it: the dispatch of a built library is
asked on the host which kernels the shapes below launch, and the GPU tests run just these shapes."""
import math
import os
import re
import subprocess

import pytest
import torch

import fp4_util as U
import layer_embedding_lookup_amd as ple
import test_fp4_gpu as G
from layer_embedding_lookup_amd import build as B
from layer_embedding_lookup_amd import capi

DEV = "cuda:0"
F64, BF = torch.float64, torch.bfloat16

# T, O, K by group: one for each shape of a block, K in whole steps of 128 and with a short last one
SHAPES = [(7, 100, 1152), (24, 70, 1152), (50, 333, 1152), (37, 5003, 1152), (100, 4200, 1152), (600, 4999, 384),
          (2051, 4099, 384)]
SHORT = {16: (32, 160, 1056), 32: (32, 160, 1056), 64: (64, 192, 1088), 128: (128, 384)}
LINEAR = [(T, O, k, g) for T, O, K in SHAPES for g in SHORT for k in dict.fromkeys((K, *SHORT[g]))]
# (more than one round of every wave's steps)
LINEAR += [(3, 200, 8192, g) for g in SHORT] + [(37, 5003, 4224, g) for g in SHORT] + [(600, 4999, 4224, 128), (2051, 4099, 4224, 16)]


def ragged(R, most, some=()):
    """R lengths up to `most`, the last ones `some`."""
    return [1 + (37 * i * i + 11 * i) % most for i in range(R - len(some))] + list(some)


class Case:
    def __init__(self, D, Hq, H, news, lens, window=0, page=16, bad=()):
        self.D, self.Hq, self.H, self.news, self.lens, self.window, self.page, self.bad = D, Hq, H, news, lens, window, page, bad

    def __repr__(self):
        return (f"D{self.D}-{self.Hq}x{self.H}-R{len(self.lens)}-new{max(self.news)}-len{max(self.lens)}-w{self.window}"
                f"{'-bad' if self.bad else ''}")


# bad: (request, first entry, past the last entry) of the page table that names no page
ATTENTION = []
for D in (64, 128, 256):
    ATTENTION += [
        # a full decode batch (blocks of four waves), short; with a window; of two splits, one of them of bad pages only
        Case(D, 16, 8, [1] * 40, ragged(40, 200), bad=((3, 1, 2), (39, 0, 40))),
        Case(D, 24, 8, [1] * 40, ragged(40, 200), window=50),
        Case(D, 16, 8, [1] * 33, ragged(33, 100, [1500, 2300]), bad=((32, 0, 90),)),
        # verify windows in more blocks than CUs, one and two row tiles
        Case(D, 16, 8, [1 + i % 9 for i in range(40)], [9 + n for n in ragged(40, 150)]),
        Case(D, 32, 8, [1 + i % 12 for i in range(33)], [12 + n for n in ragged(33, 150)], window=40),
        # few blocks, of eight waves: splits joined by a wave a row and by four
        Case(D, 4, 1, [1], [2500], bad=((0, 70, 80),)), Case(D, 24, 1, [1, 1], [5, 3100]),
        Case(D, 4, 1, [1], [9300]), Case(D, 6, 1, [2, 1], [9500, 40], bad=((0, 64, 200), (0, 400, 401)), page=32),
        Case(D, 3, 1, [4], [9900], window=9200),
        # many rows, in shares and a block a query tile
        Case(D, 8, 2, [90, 33], [1500, 700], bad=((0, 20, 40),)), Case(D, 4, 1, [20] * 65, [20 + 3 * i for i in range(65)])]


def hints(c):
    return dict(max_request_tokens=max(c.news), max_seq_len=max(c.lens))


def width(c):
    return max(-(-n // c.page) for n in c.lens) + 1


def kernels_of(tmp_path, lines):
    src = tmp_path / "dispatch.cpp"
    src.write_text(r"""
#include "ple_fp4_launch.h"
#include <stdio.h>
#include <string.h>
using namespace ple;
int main() {
    char what[16];
    long T, R, H, Hq, D, page, width, most_new, most, window, O, K, g;
    while (scanf("%15s", what) == 1) {
        if (what[0] == 'l') {
            if (scanf("%ld %ld %ld", &T, &O, &g) != 3) return 1;
            const W4Shape s = w4_linear_shape(T, (int)O, (int)g);
            printf("w4_%s_%dx%d_%ld_kernel\n", s.many ? "gemm" : "rows", s.mt, s.nt, g);
            continue;
        }
        if (scanf("%ld %ld %ld %ld %ld %ld %ld %ld %ld %ld", &T, &R, &H, &Hq, &D, &page, &width, &most_new, &most, &window) != 10)
            return 1;
        Kv4AttentionArgs a;
        memset(&a, 0, sizeof(a));
        a.cache.num_kv_heads = (int)H, a.cache.head_dim = (int)D, a.cache.page_size = (int)page;
        a.batch.num_tokens = T, a.batch.num_reqs = (int)R, a.batch.table_width = (int)width;
        a.batch.max_request_tokens = (int)most_new, a.batch.max_seq_len = (int)most;
        a.num_q_heads = (int)Hq, a.group = (int)(Hq / H), a.window = (int)window;
        plan_kv4_attention(a);
        if (a.rows == 128)
            printf("kv4_attention_chunk_%ld_kernel\n", D);
        else
            printf("kv4_attention_%ld_%dx%d_kernel\n", D, a.rows / 16, a.waves);
        if (a.flat > 0)
            printf("kv4_attention_flat_join_%ld_kernel\n", D);
        else if (a.splits > 1)
            printf("kv4_attention_join_%ld_%d_kernel\n", D, a.splits <= 8 ? 1 : 4);
    }
}
""")
    exe = tmp_path / "dispatch"
    cmd = [B.hipcc(), "-x", "hip", f"--offload-arch={B.ARCH}", "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, str(src), "-x", "none",
           capi.LIB_PATH, f"-Wl,-rpath,{os.path.dirname(capi.LIB_PATH)}", "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([str(exe)], input="\n".join(lines), capture_output=True, text=True)
    assert res.returncode == 0
    return set(res.stdout.split())


def test_shapes_reach_every_kernel(tmp_path):
    lines = [f"linear {T} {O} {g}" for T, O, _, g in LINEAR]
    lines += [f"attention {sum(c.news)} {len(c.lens)} {c.H} {c.Hq} {c.D} {c.page} {width(c)} {max(c.news)} {max(c.lens)} {c.window}"
              for c in ATTENTION]
    names = subprocess.run(["nm", "-D", capi.LIB_PATH], capture_output=True, text=True, check=True).stdout
    built = set(re.findall(r"\d((?:w4|kv4_attention)_[a-z0-9_]+_kernel)E", names))
    assert len(built) == 48
    assert kernels_of(tmp_path, lines) == built


def weight(g, O, K, group):
    """As G.make_weight, in front of rows that must not be read: NaN scales."""
    fmt, zeros = ("nvfp4", False) if group == 16 else ("int4", group >= 64)
    w, W = G.make_weight(g, fmt, O + 9, K, group, zeros)
    w.scales.view(torch.uint8)[O:] = 0x7F if group == 16 else 0xFF
    if group == 16:
        return ple.W4Weight.nvfp4(w.codes[:O], w.scales[:O], w.tensor_scale), W[:O]
    return ple.W4Weight.int4(w.codes[:O], w.scales[:O], None if w.zeros is None else w.zeros[:O]), W[:O]


def rows(g, T, K):
    """x [T][K] out of a wider tensor that is NaN around it."""
    wide = torch.full((T + 5, K + 136), math.nan, dtype=BF)
    wide[2:T + 2, 64:K + 64] = torch.randn((T, K), generator=g).to(BF)
    return wide[2:T + 2, 64:K + 64], wide.to(DEV)[2:T + 2, 64:K + 64]


@pytest.mark.gpu
@pytest.mark.parametrize("T,O,K,group", LINEAR)
def test_linear_kernels(T, O, K, group):
    print(f"linear T={T} O={O} K={K} group={group}", flush=True)
    g = G.gen(T + O + K + group)
    w, W = weight(g, O, K, group)
    x, dx = rows(g, T, K)
    around = torch.full((T + 16, O), 7, dtype=BF, device=DEV)
    out = around[8:T + 8]                       # (8 rows: 16-byte aligned for any O)
    ple.ple_w4_linear(dx, w, out=out)
    G.check_linear(x, w, W, out)
    assert (around[:8] == 7).all() and (around[T + 8:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,O,K,group", [(T, O, SHORT[g][-1], g) for T, O, _ in SHAPES for g in SHORT])
def test_linear_kernels_nonfinite_rows_stay_apart(T, O, K, group):
    """An infinity in the first and a NaN in the last place of two rows, the ends of the first and the last step."""
    g = G.gen(T + O + group)
    w, W = weight(g, O, K, group)
    _, x = rows(g, T, K)
    want = ple.ple_w4_linear(x, w)
    x[1, 0], x[T - 1, K - 1] = math.inf, math.nan
    out = ple.ple_w4_linear(x, w)
    live = (W[:, 0] != 0).to(DEV)
    assert not torch.isfinite(out[1, live]).any() and torch.isnan(out[T - 1]).all()
    keep = [t for t in range(T) if t not in (1, T - 1)]
    assert torch.equal(out[keep], want[keep])


def attention_inputs(c):
    g = G.gen(c.D + c.Hq + sum(c.lens))
    cache = U.Cache(g, c.lens, H=c.H, D=c.D, page=c.page)
    for r, a, b in c.bad:
        cache.table[r, a:b] = -1
    qsl, seq, _ = G.batch(c.news, c.lens, cache)
    return cache, (1.5 * torch.randn((int(qsl[-1]), c.Hq, c.D), generator=g)).to(BF), qsl, seq


@pytest.mark.gpu
@pytest.mark.parametrize("c", ATTENTION, ids=repr)
def test_attention_kernels(c):
    print(f"attention {c}", flush=True)
    cache, q, qsl, seq = attention_inputs(c)
    assert cache.width == width(c)
    G.check_attention(cache, q, qsl, seq, c.window, **hints(c))


@pytest.mark.gpu
@pytest.mark.parametrize("k", ["k", "v"])
@pytest.mark.parametrize("c", ATTENTION, ids=repr)
def test_attention_kernels_nan_in_one_request(c, k):
    """A key or value block of one head in the middle of the longest request (of one split, wave and tile): NaN for the
    rows and heads that see it, nothing else changes."""
    cache, q, qsl, seq = attention_inputs(c)
    clean, clean_lse = G.run_attention(cache, q, qsl, seq, window=c.window, **hints(c))
    r = c.lens.index(max(c.lens))
    before = c.lens[r] - c.news[r]
    first = 0 if c.window == 0 else max(0, c.lens[r] - c.window)
    j = next(j for j in range((first + before) // 2, before + 1) if 0 <= int(cache.table[r, j // c.page]))
    head, block = c.H - 1, c.D // 16 - 2
    cache.scales[k][int(cache.table[r, j // c.page]), head, (j % c.page) // 16, block, j % 16] = 0xFF
    out, lse = G.run_attention(cache, q, qsl, seq, window=c.window, **hints(c))
    mine = torch.zeros((q.shape[0], c.Hq), dtype=torch.bool)
    mine[int(qsl[r]):int(qsl[r + 1]), head * (c.Hq // c.H):] = True
    # of the request's rows, those that see token j (row i stands at before + i)
    p = before + torch.arange(c.news[r])
    sees = (p >= j) & (p - c.window < j if c.window else True)
    mine[int(qsl[r]):int(qsl[r + 1])] &= sees[:, None]
    assert mine.any() and torch.equal(out[~mine], clean[~mine]) and torch.equal(lse[~mine], clean_lse[~mine])
    if k == "k":
        assert torch.isnan(out[mine]).all() and torch.isnan(lse[mine]).all()
    else:
        part = torch.zeros(c.D, dtype=torch.bool)
        part[block * 16:block * 16 + 16] = True
        assert torch.isnan(out[mine][:, part]).all() and torch.equal(out[mine][:, ~part], clean[mine][:, ~part])
        assert torch.equal(lse[mine], clean_lse[mine])
