#!/usr/bin/env python3
"""Attention layers that decode in 8 bits: the residual's addition and norm straight to 8-bit activations
(ple_rms_norm8), 8-bit projections (ple_w8_linear), a paged 8-bit key/value cache whose block scales grow as tokens come
in (ple_kv8_append) and attention over it (ple_kv8_attention).

Ragged prompts go in as one prefill; the decode steps of one token per request are captured into a HIP graph, which
moves the requests' lengths on by itself, and replayed.  At the end the last step of the last layer is checked against a
plain attention in 32 bits over what its cache holds (ple_kv8_read).

    python examples/bits8_decode.py [--requests 64] [--prompt 700] [--steps 32] [--layers 2]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import layer_embedding_lookup_amd as ple  # noqa: E402

DEV = "cuda"


def w8(w):
    """A weight matrix [O][K] in 8 bits with a scale per row."""
    s = w.abs().amax(1) / 127
    return ple.W8Weight((w / s[:, None]).round().to(torch.int8), s.float())


class AttentionLayer:
    """norm -> q, k, v -> attention over the cache -> norm -> projection, for up to `requests` requests of `most` tokens;
    the residual is added by the next layer's norm."""

    def __init__(self, hidden, q_heads, kv_heads, dim, requests, most, page=64, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.q_heads, self.kv_heads, self.dim = q_heads, kv_heads, dim
        rnd = lambda o, k: torch.randn((o, k), generator=g, device=DEV) * k ** -0.5  # noqa: E731
        self.qkv, self.out = w8(rnd((q_heads + 2 * kv_heads) * dim, hidden)), w8(rnd(hidden, q_heads * dim))
        self.norms = [torch.ones(n, dtype=torch.bfloat16, device=DEV) for n in (hidden, q_heads * dim)]
        width = -(-most // page)
        pages, blocks = requests * width, page // 16
        u8 = lambda *s: torch.zeros((pages, kv_heads, blocks, *s), dtype=torch.uint8, device=DEV)  # noqa: E731
        f32 = lambda: torch.zeros((pages, kv_heads, blocks), device=DEV)  # noqa: E731
        self.cache = ple.KV8Cache(u8(dim // 16, 16, 16), f32(), u8(dim, 16), f32())  # (a block's first tokens set its scale)
        self.table = torch.randperm(pages, generator=g, device=DEV).int().view(requests, width)
        self.inv_freq = (1e4 ** (-torch.arange(0, dim, 2, device=DEV, dtype=torch.float64) / dim)).float()

    def __call__(self, x, residual, query_start_loc, seq_lens, max_new, max_len):
        """x, residual bf16 [T][hidden], the requests' new tokens (residual None: x is it); seq_lens counts them.  Returns the
        layer's output without the residual, the residual, and the rotated queries and their attention for the check."""
        d, a, b = self.dim, self.q_heads, self.q_heads + self.kv_heads
        codes, scales, hidden = ple.ple_rms_norm8(x, self.norms[0], residual=residual)
        heads = ple.ple_w8_linear(codes, scales, self.qkv).view(-1, b + self.kv_heads, d)
        where = (query_start_loc, seq_lens, self.table)
        q = ple.ple_kv8_append(self.cache, heads[:, a:b], heads[:, b:], *where, inv_freq=self.inv_freq, q=heads[:, :a],
                               max_request_tokens=max_new)
        att, _ = ple.ple_kv8_attention(q, self.cache, *where, max_request_tokens=max_new, max_seq_len=max_len)
        codes, scales, _ = ple.ple_rms_norm8(att.view(-1, a * d), self.norms[1])
        return ple.ple_w8_linear(codes, scales, self.out), x if hidden is None else hidden, q, att


def plain_attention(layer, q, r, length):
    """Request r's last token against the cache's keys and values, in 32 bits."""
    all_of = torch.tensor([0, length], dtype=torch.int32, device=DEV)
    k, v = ple.ple_kv8_read(layer.cache, all_of, all_of[1:], layer.table[r:r + 1], length)
    k, v = (t.float().permute(1, 0, 2).contiguous() for t in (k, v))
    q = q.float().view(layer.kv_heads, -1, layer.dim)
    p = torch.softmax(torch.bmm(q, k.transpose(1, 2).contiguous()) * layer.dim ** -0.5, -1)
    return torch.bmm(p, v).view(-1, layer.dim)


def main(requests=64, prompt=700, steps=32, layers=2, hidden=4096, q_heads=32, kv_heads=8, dim=128, seed=0):
    """Returns the largest difference to the plain attention, over the largest value there, and the time of a step."""
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    lens = torch.randint(1, prompt + 1, (requests,), generator=torch.Generator().manual_seed(seed))
    most = prompt + steps
    stack = [AttentionLayer(hidden, q_heads, kv_heads, dim, requests, most, seed=seed + i) for i in range(layers)]
    start = torch.zeros(requests + 1, dtype=torch.int32)
    start[1:] = lens.cumsum(0)
    seq = lens.int().to(DEV)

    def run(x, *where):
        h = None
        for layer in stack:
            x, h, q, att = layer(x, h, *where)
        return x, q, att

    run(torch.randn((int(start[-1]), hidden), generator=g, device=DEV).bfloat16(), start.to(DEV), seq, prompt, prompt)
    ones = torch.arange(requests + 1, dtype=torch.int32, device=DEV)
    token = torch.randn((requests, hidden), generator=g, device=DEV).bfloat16()

    def step():
        seq.add_(1)
        return run(token, ones, seq, 1, most)

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
        want = plain_attention(stack[-1], q[r], r, int(seq[r]))
        worst = max(worst, float((att[r].float() - want).abs().max() / want.abs().max()))
    return worst, begin.elapsed_time(end) / max(1, steps - 1)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--layers", type=int, default=2)
    a = ap.parse_args()
    error, ms = main(a.requests, a.prompt, a.steps, a.layers)
    print(f"{a.layers} layers, {a.requests} requests of up to {a.prompt} + {a.steps} tokens: {ms * 1e3:.1f} us a step, "
          f"largest difference to plain attention {error:.4f} of the largest value")
