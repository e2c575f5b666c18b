"""Every kernel of the 8-bit decode operators, by shapes that reach it: the dispatch of a built library is asked on the
host which kernels the shapes below (and those of test_bits8_gpu) launch, and the GPU tests run just these shapes."""
import os
import re
import subprocess

import pytest
import torch

import bits8_util as U
import test_bits8_gpu as G
from layer_embedding_lookup_amd import build as B
from layer_embedding_lookup_amd import capi
from test_fp4_kernels import ATTENTION as OF_4_BITS
from test_fp4_kernels import Case, hints, width

BF = torch.bfloat16
# (many rows far into the cache, in shares: with two and with three pieces of a query tile)
ATTENTION = OF_4_BITS + [c for D in (64, 128, 256) for c in (
    Case(D, 8, 2, [90, 33], [1900, 700], bad=((0, 20, 40),)), Case(D, 8, 1, [60, 33], [9000, 1100]),
    Case(D, 4, 1, [200], [4000], window=1700, bad=((0, 200, 210),)))]
NORM = [16, 512, 528, 2048, 2064, 4096, 4112, 8192, 8208, 16384, 16400]


def kernels_of(tmp_path, lines):
    src = tmp_path / "dispatch.cpp"
    src.write_text(r"""
#include "ple_8bit_launch.h"
#include <stdio.h>
#include <string.h>
using namespace ple;
int main() {
    char what[16];
    long T, R, H, Hq, D, page, width, most_new, most, window, O, n;
    while (scanf("%15s", what) == 1) {
        if (what[0] == 'n') {
            if (scanf("%ld", &n) != 1) return 1;
            const RmsNorm8Shape f = rms_norm8_shape((int)n);
            if (f.waves == 0)
                printf("rms_norm8_long_kernel\n");
            else
                printf("rms_norm8_%dx%d_kernel\n", f.waves, f.chunks);
            continue;
        }
        if (what[0] == 'l') {
            if (scanf("%ld %ld", &T, &O) != 2) return 1;
            const W8Shape f = w8_linear_shape(T, (int)O);
            if (f.block == 256)
                printf("w8_gemm_256_kernel\n");
            else if (f.block == 64)
                printf("w8_tile_%dx%d_kernel\n", f.rows, f.nt);
            else
                printf("w8_rows_%dx%d_%d_kernel\n", f.rows, f.nt, f.step);
            continue;
        }
        if (scanf("%ld %ld %ld %ld %ld %ld %ld %ld %ld %ld", &T, &R, &H, &Hq, &D, &page, &width, &most_new, &most, &window) != 10)
            return 1;
        Kv8AttentionArgs a;
        memset(&a, 0, sizeof(a));
        a.cache.num_kv_heads = (int)H, a.cache.head_dim = (int)D, a.cache.page_size = (int)page;
        a.batch.num_tokens = T, a.batch.num_reqs = (int)R, a.batch.table_width = (int)width;
        a.batch.max_request_tokens = (int)most_new, a.batch.max_seq_len = (int)most;
        a.num_q_heads = (int)Hq, a.group = (int)(Hq / H), a.window = (int)window;
        plan_kv8_attention(a);
        if (a.rows == 128)
            printf("kv8_attention_chunk_%ld_kernel\n", D);
        else
            printf("kv8_attention_%ld_%dx%d_kernel\n", D, a.rows / 16, a.waves);
        if (a.flat > 0)
            printf("kv8_attention_flat_join_%ld_kernel\n", D);
        else if (a.splits > 1)
            printf("kv8_attention_join_%ld_%d_kernel\n", D, a.splits <= 8 ? 1 : 4);
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
    lines = [f"norm {n}" for n in NORM] + [f"linear {T} {O}" for T, O in G.LINEAR_T_O]
    lines += [f"attention {sum(c.news)} {len(c.lens)} {c.H} {c.Hq} {c.D} {c.page} {width(c)} {max(c.news)} {max(c.lens)} {c.window}"
              for c in ATTENTION]
    names = subprocess.run(["nm", "-D", capi.LIB_PATH], capture_output=True, text=True, check=True).stdout
    built = set(re.findall(r"\d((?:w8|rms_norm8|kv8)_[a-z0-9_]+_kernel)E", names))
    assert len(built) == 41
    got = kernels_of(tmp_path, lines)
    # (append and read have one kernel for each head size, and test_bits8_gpu calls them with each)
    got |= {f"kv8_{what}_{D}_kernel" for what in ("append", "read") for D in {c[0] for c in G.APPEND}}
    assert got == built


def attention_inputs(c):
    g = G.gen(c.D + c.Hq + sum(c.lens))
    cache = U.Cache(g, c.lens, H=c.H, D=c.D, page=c.page)
    for r, a, b in c.bad:
        cache.table[r, a:b] = -1
    qsl, seq = G.batch(c.news, c.lens)
    return cache, (1.5 * torch.randn((int(qsl[-1]), c.Hq, c.D), generator=g)).to(BF), qsl, seq


@pytest.mark.gpu
@pytest.mark.parametrize("c", ATTENTION, ids=repr)
def test_attention_kernels(c):
    print(f"kv8 attention {c}", flush=True)
    cache, q, qsl, seq = attention_inputs(c)
    assert cache.width == width(c)
    G.check_attention(cache, q, qsl, seq, c.window, **hints(c))


@pytest.mark.gpu
@pytest.mark.parametrize("k", ["k", "v"])
@pytest.mark.parametrize("c", ATTENTION, ids=repr)
def test_attention_kernels_nan_in_one_request(c, k):
    """A NaN code of one head in the middle of the longest request (of one split, wave and tile): NaN for the rows and heads
    that see it (of a value, that element of them), nothing else changes."""
    cache, q, qsl, seq = attention_inputs(c)
    clean, clean_lse = G.run_attention(cache, q, qsl, seq, window=c.window, **hints(c))
    r = c.lens.index(max(c.lens))
    before = c.lens[r] - c.news[r]
    first = 0 if c.window == 0 else max(0, c.lens[r] - c.window)
    j = next(j for j in range((first + before) // 2, before + 1) if 0 <= int(cache.table[r, j // c.page]))
    head, d = c.H - 1, c.D - 19
    cache.codes[k][int(cache.table[r, j // c.page]), head, j % c.page, d] = 0xFF
    out, lse = G.run_attention(cache, q, qsl, seq, window=c.window, **hints(c))
    mine = torch.zeros((q.shape[0], c.Hq), dtype=torch.bool)
    mine[int(qsl[r]):int(qsl[r + 1]), head * (c.Hq // c.H):] = True
    p = before + torch.arange(c.news[r])                     # of the request's rows, those that see token j
    sees = (p >= j) & (p - c.window < j if c.window else True)
    mine[int(qsl[r]):int(qsl[r + 1])] &= sees[:, None]
    assert mine.any() and torch.equal(out[~mine], clean[~mine]) and torch.equal(lse[~mine], clean_lse[~mine])
    if k == "k":
        assert torch.isnan(out[mine]).all() and torch.isnan(lse[mine]).all()
    else:
        rest = [e for e in range(c.D) if e != d]
        assert torch.isnan(out[mine][:, d]).all() and torch.equal(out[mine][:, rest], clean[mine][:, rest])
        assert torch.equal(lse[mine], clean_lse[mine])
