"""The 8-bit decode operators (include/ple_8bit.h): the residual's addition and RMS norm with an 8-bit output, products
of 8-bit integers, a paged 8-bit key/value cache and attention over it.

    codes, scales, hidden = ple_rms_norm8(x, norm_weight, residual=hidden)
    w = W8Weight(weight_codes, channel_scales)
    y = ple_w8_linear(codes, scales, w)
    cache = KV8Cache(k_codes, k_scales, v_codes, v_scales)
    q = ple_kv8_append(cache, k, v, query_start_loc, seq_lens, page_table, inv_freq=inv_freq, q=q)
    out, lse = ple_kv8_attention(q, cache, query_start_loc, seq_lens, page_table, want_lse=True)

Like the rest of the binding these only marshal tensors; the header states
formats, layouts and limits.  Outputs and workspaces that a call makes itself
belong to the stream it runs on (`stream`, or the current one).  Tensors are on
the current device, or on that of a `stream` that is not a default one.
"""
from __future__ import annotations

import ctypes

import torch

from . import capi
from . import _BF16, _F32, _ptr, _req, _same_device
from .fp4 import (_BF, _FP8, _MOST, _attention, _attention_workspace_bytes, _fits, _append, _given, _new, _raw_stream, _read)

_I8, _FLOAT = torch.int8, torch.float32


def ple_rms_norm8(x, weight, *, residual=None, eps: float = 1e-6, codes=None, scales=None, residual_out=None, stream=None):
    """x bf16 [T][N] (rows may be strided), residual bf16 [T][N] or None, weight bf16 [N] -> (codes int8 [T][N], scales fp32
    [T], residual_out bf16 [T][N]: x + residual, or None without one).  residual_out may be residual."""
    shape = x.shape
    if len(shape) != 2 or x.dtype not in _BF16 or (shape[0] and x.stride(1) != 1):
        raise ValueError(f"x must be bf16 [T][N] with contiguous rows, got {tuple(shape)} {x.dtype}")
    T, N = shape
    dev, device = x.get_device(), x.device
    if residual is None and residual_out is not None:
        raise ValueError("residual_out given without residual")
    # (what most calls pass goes through the checks that name the fault only where one is off)
    if (dev < 0 or not _fits(weight, _BF, (N,), dev) or not (residual is None or _fits(residual, _BF, shape, dev))
            or codes is not None or scales is not None or residual_out is not None):
        _req("weight", weight, (N,), _BF16)
        _req("residual", residual, (T, N), _BF16, optional=True)
        _req("residual_out", residual_out, (T, N), _BF16, optional=True)
        _req("codes", codes, (T, N), (_I8,), optional=True)
        _req("scales", scales, (T,), _F32, optional=True)
        _same_device(x, weight, residual, codes, scales, residual_out)
    if residual is not None and residual_out is None:
        residual_out = _new((T, N), _BF, device, stream)
    if codes is None:
        codes = _new((T, N), _I8, device, stream)
    if scales is None:
        scales = _new((T,), _FLOAT, device, stream)
    rc = capi.load().ple_rms_norm8(x.data_ptr(), x.stride(0) if T > 1 else N, _ptr(residual), _ptr(weight), T, N, eps,
                                   _ptr(codes), _ptr(scales), _ptr(residual_out),
                                   _raw_stream(dev) if stream is None else _given(stream, dev))
    if rc:
        capi.check(rc, "ple_rms_norm8")
    return codes, scales, residual_out


class W8Weight:
    """A [O][K] weight matrix in 8 bits, W[o][i] = codes[o][i] * scales[o]: a view of the caller's tensors, codes int8
    [O][K] and scales fp32 [O] (nothing is copied or laid out anew)."""

    def __init__(self, codes, scales):
        _req("codes", codes, (None, None), (_I8,))
        self.out_dim, self.k_dim = int(codes.shape[0]), int(codes.shape[1])
        _req("scales", scales, (self.out_dim,), _F32)
        _same_device(codes, scales)
        self.codes, self.scales = codes, scales
        self.device = codes.get_device()
        self.desc = capi.ple_w8_weight(_ptr(codes), _ptr(scales), self.out_dim, self.k_dim)


def ple_w8_linear(x, x_scales, w: W8Weight, *, out=None, stream=None):
    """x int8 [T][K] (rows may be strided) and its scales fp32 [T] -> out bf16 [T][O] = (x * x_scales) W^T."""
    shape = x.shape
    if len(shape) != 2 or shape[1] != w.k_dim or x.dtype is not _I8 or (shape[0] and x.stride(1) != 1):
        raise ValueError(f"x must be int8 [T][{w.k_dim}] with contiguous rows, got {tuple(shape)} {x.dtype}")
    T = shape[0]
    if not _fits(x_scales, _FLOAT, (T,), w.device):
        _req("x_scales", x_scales, (T,), _F32)
        _same_device(x, x_scales, w.codes)
    if out is None:
        if x.get_device() != w.device:
            _same_device(x, w.codes)
        out = _new((T, w.out_dim), _BF, x.device, stream)
    else:
        _req("out", out, (T, w.out_dim), _BF16)
        _same_device(x, w.codes, out)
    rc = capi.load().ple_w8_linear(x.data_ptr(), x.stride(0) if T > 1 else w.k_dim, _ptr(x_scales), ctypes.byref(w.desc), T,
                                   _ptr(out), _raw_stream(w.device) if stream is None else _given(stream, w.device))
    if rc:
        capi.check(rc, "ple_w8_linear")
    return out


class KV8Cache:
    """A paged 8-bit key/value cache: a view of the caller's tensors.

    k_codes e4m3fn [pages][heads][page_size/16][D/16][16 tokens][16], v_codes e4m3fn [pages][heads][page_size/16][D][16
    tokens], k_scales, v_scales fp32 [pages][heads][page_size/16] (codes as uint8 or float8_e4m3fn)."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        _req("k_codes", k_codes, (None, None, None, None, 16, 16), _FP8)
        pages, heads, blocks, pieces = k_codes.shape[:4]
        _req("v_codes", v_codes, (pages, heads, blocks, 16 * pieces, 16), _FP8)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            _req(name, t, (pages, heads, blocks), _F32)
        _same_device(k_codes, k_scales, v_codes, v_scales)
        self.tensors = (k_codes, k_scales, v_codes, v_scales)
        self.device = k_codes.get_device()
        self.num_pages, self.num_kv_heads, self.page_size, self.head_dim = pages, heads, 16 * blocks, 16 * pieces
        self.desc = capi.ple_kv8_cache(*(t.data_ptr() for t in self.tensors), pages, heads, 16 * blocks, 16 * pieces, 0)


def ple_kv8_append(cache: KV8Cache, k, v, query_start_loc, seq_lens, page_table, *, inv_freq=None,
                   interleaved: bool = False, q=None, q_out=None, max_request_tokens: int = 0, stream=None):
    """New keys and values bf16 [T][heads][D] into the cache, keys (and q, if given) rotated by their positions over
    the first 2 * len(inv_freq) elements.  max_request_tokens (0: unknown): no request has more new tokens, which sizes the
    launch (of one that has more, the last ones may not be stored).  Returns the rotated queries bf16 [T][q heads][D], or None without q."""
    return _append("ple_kv8_append", cache, k, v, query_start_loc, seq_lens, page_table, inv_freq, interleaved, q, q_out,
                   stream, max_request_tokens)


def ple_kv8_read(cache: KV8Cache, query_start_loc, seq_lens, page_table, num_tokens: int, *, k_out=None, v_out=None,
                 stream=None):
    """The new tokens' keys and values as the cache holds them: two bf16 [T][heads][D]."""
    return _read("ple_kv8_read", cache, query_start_loc, seq_lens, page_table, num_tokens, k_out, v_out, stream)


def ple_kv8_attention_workspace_bytes(cache: KV8Cache, num_q_heads: int, num_tokens: int, num_reqs: int,
                                      table_width: int, *, window: int = 0, max_request_tokens: int = 0,
                                      max_seq_len: int = 0) -> int:
    """Workspace of a call with these sizes and hints (0: none is needed)."""
    return _attention_workspace_bytes("ple_kv8_attention", cache, num_q_heads, num_tokens, num_reqs, table_width, window,
                                      max_request_tokens, max_seq_len)


def ple_kv8_attention(q, cache: KV8Cache, query_start_loc, seq_lens, page_table, *, window: int = 0, scale=None,
                      max_request_tokens: int = 0, max_seq_len: int = 0, want_lse: bool = False, out=None, lse=None,
                      workspace=None, stream=None):
    """Causal attention of the new tokens q bf16 [T][q heads][D] over the cache; arguments and results as for
    ple_kv4_attention, long prefills and single tokens better in two calls too."""
    return _attention("ple_kv8_attention", q, cache, query_start_loc, seq_lens, page_table, window, scale,
                      max_request_tokens, max_seq_len, want_lse, out, lse, workspace, stream)
