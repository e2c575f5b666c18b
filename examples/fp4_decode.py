#!/usr/bin/env python3
"""An attention layer that decodes in 4 bits: NVFP4 projections (ple_w4_linear), a paged 4-bit key/value cache
(ple_kv4_append) and attention over it (ple_kv4_attention).

Ragged prompts go in as one prefill; the decode steps of one token per request are captured into a HIP graph, which
moves the requests' lengths on by itself, and replayed.  At the end the last step is checked against a plain attention
in 32 bits over what the cache holds (ple_kv4_read).

    python examples/fp4_decode.py [--requests 64] [--prompt 700] [--steps 32]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import layer_embedding_lookup_amd as ple  # noqa: E402

DEV = "cuda"
E2M1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6])


def nvfp4(w):
    """A weight matrix [O][K] in NVFP4: codes, block scales and tensor scale."""
    ts = (w.abs().amax() / (6 * 448)).reshape(1)
    b = w.unflatten(-1, (-1, 16))
    s = (b.abs().amax(-1) / (6 * ts)).to(torch.float8_e4m3fn)
    t = (b / (s.float() * ts).clamp_min(1e-30).unsqueeze(-1)).flatten(-2)
    grid = E2M1.to(w.device)
    code = torch.bucketize(t.abs(), (grid[1:] + grid[:-1]) / 2) | torch.signbit(t).long() << 3
    code = code.unflatten(-1, (-1, 2))
    return (code[..., 0] | code[..., 1] << 4).to(torch.uint8), s.view(torch.uint8), ts.float()


class AttentionLayer:
    """hidden -> q, k, v -> attention over the cache -> hidden, for up to `requests` requests of `most` tokens."""

    def __init__(self, hidden, q_heads, kv_heads, dim, requests, most, page=64, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.q_heads, self.kv_heads, self.dim, self.most = q_heads, kv_heads, dim, most
        rnd = lambda o, k: torch.randn((o, k), generator=g, device=DEV) * k ** -0.5  # noqa: E731
        self.qkv = ple.W4Weight.nvfp4(*nvfp4(rnd((q_heads + 2 * kv_heads) * dim, hidden)))
        self.out = ple.W4Weight.nvfp4(*nvfp4(rnd(hidden, q_heads * dim)))
        width = -(-most // page)
        pages = requests * width
        codes = lambda: torch.zeros((pages, kv_heads, page, dim // 2), dtype=torch.uint8, device=DEV)  # noqa: E731
        scales = lambda: torch.zeros((pages, kv_heads, page // 16, dim // 16, 16), dtype=torch.uint8, device=DEV)  # noqa: E731
        one = torch.full((kv_heads,), 0.01, device=DEV)  # a block's scale covers 0.01 * 6 * 448 and 13 octaves below
        self.cache = ple.KV4Cache(codes(), scales(), codes(), scales(), one, one.clone())
        self.table = torch.randperm(pages, generator=g, device=DEV).int().view(requests, width)
        self.inv_freq = (1e4 ** (-torch.arange(0, dim, 2, device=DEV, dtype=torch.float64) / dim)).float()

    def __call__(self, x, query_start_loc, seq_lens, max_new, max_len):
        """x bf16 [T][hidden], the requests' new tokens; seq_lens counts them.  Returns the layer's output, and the
        rotated queries and their attention for the check."""
        d, a, b = self.dim, self.q_heads, self.q_heads + self.kv_heads
        heads = ple.ple_w4_linear(x, self.qkv).view(-1, b + self.kv_heads, d)
        where = (query_start_loc, seq_lens, self.table)
        q = ple.ple_kv4_append(self.cache, heads[:, a:b], heads[:, b:], *where, inv_freq=self.inv_freq, q=heads[:, :a])
        att, _ = ple.ple_kv4_attention(q, self.cache, *where, max_request_tokens=max_new, max_seq_len=max_len)
        return ple.ple_w4_linear(att.view(-1, a * d), self.out), q, att


def plain_attention(layer, q, r, length):
    """Request r's last token against the cache's keys and values, in 32 bits."""
    all_of = torch.tensor([0, length], dtype=torch.int32, device=DEV)
    k, v = ple.ple_kv4_read(layer.cache, all_of, all_of[1:], layer.table[r:r + 1], length)
    k, v = (t.float().permute(1, 0, 2).contiguous() for t in (k, v))
    q = q.float().view(layer.kv_heads, -1, layer.dim)
    p = torch.softmax(torch.bmm(q, k.transpose(1, 2).contiguous()) * layer.dim ** -0.5, -1)
    return torch.bmm(p, v).view(-1, layer.dim)


def main(requests=64, prompt=700, steps=32, hidden=4096, q_heads=32, kv_heads=8, dim=128, seed=0):
    """Returns the largest difference to the plain attention, over the largest value there, and the time of a step."""
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    lens = torch.randint(1, prompt + 1, (requests,), generator=torch.Generator().manual_seed(seed))
    most = prompt + steps
    layer = AttentionLayer(hidden, q_heads, kv_heads, dim, requests, most, seed=seed)
    start = torch.zeros(requests + 1, dtype=torch.int32)
    start[1:] = lens.cumsum(0)
    seq = lens.int().to(DEV)
    x = torch.randn((int(start[-1]), hidden), generator=g, device=DEV).bfloat16()
    layer(x, start.to(DEV), seq, prompt, prompt)

    ones = torch.arange(requests + 1, dtype=torch.int32, device=DEV)
    token = torch.randn((requests, hidden), generator=g, device=DEV).bfloat16()

    def step():
        seq.add_(1)
        return layer(token, ones, seq, 1, most)

    out, q, att = step()  # (an eager step first: it loads the kernels)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, q, att = step()
        token.copy_(torch.nn.functional.rms_norm(y, (hidden,)))  # the next step's input
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(steps - 1):
        graph.replay()
    end.record()
    end.synchronize()
    assert int(seq.max()) == int(lens.max()) + steps
    worst = 0.0
    for r in range(0, requests, max(1, requests // 8)):
        want = plain_attention(layer, q[r], r, int(seq[r]))
        worst = max(worst, float((att[r].float() - want).abs().max() / want.abs().max()))
    return worst, begin.elapsed_time(end) / max(1, steps - 1)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    error, ms = main(a.requests, a.prompt, a.steps)
    print(f"{a.requests} requests of up to {a.prompt} + {a.steps} tokens: {ms * 1e3:.1f} us a step, "
          f"largest difference to plain attention {error:.4f} of the largest value")
