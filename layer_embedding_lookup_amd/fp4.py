"""The 4-bit decode operators (include/ple_fp4.h): products with 4-bit weights,
a paged 4-bit key/value cache and attention over it.

    w = W4Weight.nvfp4(codes, block_scales, tensor_scale)      # or W4Weight.int4(codes, scales, zeros)
    y = ple_w4_linear(x, w)
    cache = KV4Cache(k_codes, k_scales, v_codes, v_scales, k_scale, v_scale)
    q = ple_kv4_append(cache, k, v, query_start_loc, seq_lens, page_table, inv_freq=inv_freq, q=q)
    out, lse = ple_kv4_attention(q, cache, query_start_loc, seq_lens, page_table, want_lse=True)

Like the rest of the binding these only marshal tensors; the header states
formats, layouts and limits.  Outputs and workspaces that a call makes itself
belong to the stream it runs on (`stream`, or the current one).  Tensors are on
the current device, or on that of a `stream` that is not a default one.
"""
from __future__ import annotations

import ctypes

import torch

from . import capi
from . import _BF16, _BYTES, _F32, _I32, _nbytes, _ptr, _req, _req_bytes, _same_device, _stream

_FP8 = (torch.uint8, torch.float8_e4m3fn)
_MOST = 2 ** 31 - 1  # ctypes would pass the low 32 bits of a larger window or hint; all of them mean "no limit"
_BF, _INT = torch.bfloat16, torch.int32
_get_device, _get_raw_stream = (getattr(torch._C, n, None) for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))


def _current(device: int) -> None:
    """A default stream's handle is 0 on every device, which the library takes for the current one's: work on another
    device's tensors would run beside that device's own work, on memory that the current device may not reach."""
    now = _get_device()
    if now != device:
        raise ValueError(f"tensors are on cuda:{device}, the current device is cuda:{now}: call under "
                         f"torch.cuda.device({device})")


def _raw_stream(device: int) -> int:
    """The current stream's handle on the tensors' device, which has to be the current one (these calls are launch-bound at
    decode sizes, and building a torch.cuda.Stream object for it costs more than the call)."""
    if _get_device() != device:
        _current(device)
    return _get_raw_stream(device)


def _given(stream, device: int) -> int:
    """The handle of the caller's stream, a default one only of the current device."""
    if not isinstance(stream, int) and stream.cuda_stream == 0:
        _current(device)
    return _stream(stream)


def _on(stream, device):
    """The context for memory that work on `stream` writes.  The allocator hands out what was freed in the current
    stream's order, so a block from its pool may still be in use by work queued there, which `stream` does not wait
    for; memory taken on `stream` itself follows that stream's order, when it is taken and when it is given back."""
    if isinstance(stream, int):  # a handle; 0 is the default stream, which ExternalStream would not take it for
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _new(shape, dtype, device, stream=None):
    """torch.empty for one to three dimensions, in 1.3 us where that takes 2.0, for a call on `stream`."""
    n = len(shape)
    strides = (shape[1], 1) if n == 2 else (shape[1] * shape[2], shape[2], 1) if n == 3 else (1,)
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    with _on(stream, device):
        t = torch.empty_strided(shape, strides, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))  # where the caller most likely reads it before giving it up
    return t


def _fits(t, dtype, shape, device: int) -> bool:
    """A contiguous tensor of this type, shape and device: what most calls pass.  Anything else goes through the
    checks that name the fault."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device
            and t.is_contiguous())


class W4Weight:
    """A [O][K] weight matrix in 4 bits: a view of the caller's tensors (nothing is copied or laid out anew)."""

    def __init__(self, codes, scales, zeros, tensor_scale, fmt: int, group: int):
        self.codes, self.scales, self.zeros, self.tensor_scale = codes, scales, zeros, tensor_scale
        self.out_dim, self.k_dim = int(codes.shape[0]), 2 * int(codes.shape[1])
        _same_device(codes, scales, zeros, tensor_scale)
        self.device = codes.get_device()
        self.desc = capi.ple_w4_weight(_ptr(codes), _ptr(scales), _ptr(zeros), _ptr(tensor_scale), fmt, self.out_dim,
                                       self.k_dim, group)

    @classmethod
    def nvfp4(cls, codes, block_scales, tensor_scale) -> "W4Weight":
        """codes uint8 [O][K/2] (element 2i in the low nibble of byte i), block_scales e4m3fn [O][K/16],
        tensor_scale fp32 [1]."""
        _req("codes", codes, (None, None), _BYTES)
        O, half = codes.shape
        _req("block_scales", block_scales, (O, half // 8), _FP8)
        _req("tensor_scale", tensor_scale, (1,), _F32)
        return cls(codes, block_scales, None, tensor_scale, capi.PLE_W4_NVFP4, 16)

    @classmethod
    def int4(cls, codes, scales, zeros=None) -> "W4Weight":
        """codes uint8 [O][K/2], scales bf16 [O][K/group], zeros uint8 [O][K/group] or None (8 everywhere);
        the group (32, 64 or 128) follows from the shapes."""
        _req("codes", codes, (None, None), _BYTES)
        O, half = codes.shape
        _req("scales", scales, (O, None), _BF16)
        groups = int(scales.shape[1])
        if groups < 1 or (2 * half) % groups != 0:
            raise ValueError(f"scales has {groups} groups a row, which do not divide {2 * half} elements")
        _req("zeros", zeros, (O, groups), _BYTES, optional=True)
        return cls(codes, scales, zeros, None, capi.PLE_W4_INT4, 2 * half // groups)


def ple_w4_linear(x, w: W4Weight, *, out=None, stream=None):
    """x bf16 [T][K] (rows may be strided) -> out bf16 [T][O] = x W^T."""
    shape = x.shape
    if len(shape) != 2 or shape[1] != w.k_dim or x.dtype not in _BF16 or (shape[0] and x.stride(1) != 1):
        raise ValueError(f"x must be bf16 [T][{w.k_dim}] with contiguous rows, got {tuple(shape)} {x.dtype}")
    T = shape[0]
    if out is None:
        if x.get_device() != w.device:
            _same_device(x, w.codes)
        out = _new((T, w.out_dim), _BF, x.device, stream)
    else:
        _req("out", out, (T, w.out_dim), _BF16)
        _same_device(x, w.codes, out)
    rc = capi.load().ple_w4_linear(x.data_ptr(), x.stride(0) if T > 1 else w.k_dim, ctypes.byref(w.desc), T,
                                   _ptr(out), _raw_stream(w.device) if stream is None else _given(stream, w.device))
    if rc:
        capi.check(rc, "ple_w4_linear")
    return out


class KV4Cache:
    """A paged 4-bit key/value cache: a view of the caller's tensors.

    k_codes, v_codes uint8 [pages][heads][page_size][D/2]; k_scales, v_scales e4m3fn
    [pages][heads][page_size/16][D/16][16]; k_scale, v_scale fp32 [heads]."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_scale, v_scale):
        _req("k_codes", k_codes, (None, None, None, None), _BYTES)
        pages, heads, size, half = k_codes.shape
        _req("v_codes", v_codes, (pages, heads, size, half), _BYTES)
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            _req(name, t, (pages, heads, size // 16, half // 8, 16), _FP8)
        _req("k_scale", k_scale, (heads,), _F32)
        _req("v_scale", v_scale, (heads,), _F32)
        _same_device(k_codes, k_scales, v_codes, v_scales, k_scale, v_scale)
        self.tensors = (k_codes, k_scales, v_codes, v_scales, k_scale, v_scale)
        self.device = k_codes.get_device()
        self.num_pages, self.num_kv_heads, self.page_size, self.head_dim = pages, heads, size, 2 * half
        self.desc = capi.ple_kv4_cache(*(t.data_ptr() for t in self.tensors), pages, heads, size, 2 * half, 0)


def _heads(name: str, t, T, heads, cache) -> int:
    """A [T][heads][D] bf16 tensor whose tokens may be strided (a slice of a fused projection); its token stride."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _BF16:
        raise ValueError(f"{name} must be a bf16 tensor")
    D, shape = cache.head_dim, t.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != D or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected ({T}, {'*' if heads is None else heads}, {D})")
    stride = t.stride()
    if T and (stride[2] != 1 or (shape[1] > 1 and stride[1] != D)):
        raise ValueError(f"{name} must have contiguous heads and elements, got strides {stride}")
    return stride[0] if T > 1 else shape[1] * D


def _kv4_batch(cache, query_start_loc, seq_lens, page_table, T, max_request_tokens=0, max_seq_len=0):
    R = page_table.shape[0] if page_table.dim() == 2 else -1
    dev = cache.device
    if not (_fits(query_start_loc, _INT, (R + 1,), dev) and _fits(seq_lens, _INT, (R,), dev)
            and _fits(page_table, _INT, page_table.shape, dev)):
        _req("query_start_loc", query_start_loc, (None,), _I32)
        R = query_start_loc.shape[0] - 1
        if R < 0:
            raise ValueError("query_start_loc needs at least one entry")
        _req("seq_lens", seq_lens, (R,), _I32)
        _req("page_table", page_table, (R, None), _I32)
        _same_device(cache.tensors[0], query_start_loc, seq_lens, page_table)
    return capi.ple_kv4_batch(query_start_loc.data_ptr(), _ptr(seq_lens), page_table.data_ptr(), T, R,
                              page_table.shape[1], min(max_request_tokens, _MOST), min(max_seq_len, _MOST))


def _out(name, t, shape, dtypes, cache, stream):
    """An output of a call on `stream`: the caller's, checked, or a new one."""
    if t is None:
        return _new(shape, dtypes[0], cache.tensors[0].device, stream)
    _req(name, t, shape, dtypes)
    _same_device(cache.tensors[0], t)
    return t


def _append(name, cache, k, v, query_start_loc, seq_lens, page_table, inv_freq, interleaved, q, q_out, stream,
            max_request_tokens=0):
    """What the appends of the paged caches share; name: the library's call."""
    D, T, H = cache.head_dim, k.shape[0], cache.num_kv_heads
    ks, vs = _heads("k", k, T, H, cache), _heads("v", v, T, H, cache)
    qs = hq = rot = 0
    q_at = out_at = freq_at = None
    if q is not None:
        qs, hq = _heads("q", q, T, None, cache), q.shape[1]
        q_out = _out("q_out", q_out, (T, hq, D), _BF16, cache, stream)
        q_at, out_at = q.data_ptr(), _ptr(q_out)
    elif q_out is not None:
        raise ValueError("q_out given without q")
    if inv_freq is not None:
        _req("inv_freq", inv_freq, (None,), _F32)
        if inv_freq.get_device() != cache.device:
            _same_device(cache.tensors[0], inv_freq)
        rot, freq_at = 2 * inv_freq.shape[0], inv_freq.data_ptr()
    b = _kv4_batch(cache, query_start_loc, seq_lens, page_table, T, max_request_tokens)
    dev = cache.device
    if k.get_device() != dev or v.get_device() != dev or (q is not None and q.get_device() != dev):
        _same_device(cache.tensors[0], k, v, q)
    rc = getattr(capi.load(), name)(
        ctypes.byref(cache.desc), ctypes.byref(b), k.data_ptr(), ks, v.data_ptr(), vs, q_at, qs, hq, out_at, freq_at,
        rot, 1 if interleaved else 0, _raw_stream(cache.device) if stream is None else _given(stream, cache.device))
    if rc:
        capi.check(rc, name)
    return q_out


def ple_kv4_append(cache: KV4Cache, k, v, query_start_loc, seq_lens, page_table, *, inv_freq=None,
                   interleaved: bool = False, q=None, q_out=None, stream=None):
    """New keys and values bf16 [T][heads][D] into the cache, keys (and q, if given) rotated by their positions over
    the first 2 * len(inv_freq) elements.  Returns the rotated queries bf16 [T][q heads][D], or None without q."""
    return _append("ple_kv4_append", cache, k, v, query_start_loc, seq_lens, page_table, inv_freq, interleaved, q, q_out,
                   stream)


def _read(name, cache, query_start_loc, seq_lens, page_table, num_tokens, k_out, v_out, stream):
    T = int(num_tokens)
    shape = (T, cache.num_kv_heads, cache.head_dim)
    k_out = _out("k_out", k_out, shape, _BF16, cache, stream)
    v_out = _out("v_out", v_out, shape, _BF16, cache, stream)
    b = _kv4_batch(cache, query_start_loc, seq_lens, page_table, T)
    rc = getattr(capi.load(), name)(ctypes.byref(cache.desc), ctypes.byref(b), _ptr(k_out), _ptr(v_out),
                                    _raw_stream(cache.device) if stream is None else _given(stream, cache.device))
    if rc:
        capi.check(rc, name)
    return k_out, v_out


def ple_kv4_read(cache: KV4Cache, query_start_loc, seq_lens, page_table, num_tokens: int, *, k_out=None, v_out=None,
                 stream=None):
    """The new tokens' keys and values as the cache holds them: two bf16 [T][heads][D]."""
    return _read("ple_kv4_read", cache, query_start_loc, seq_lens, page_table, num_tokens, k_out, v_out, stream)


_WORKSPACE = {n: n + "_workspace_bytes" for n in ("ple_kv4_attention", "ple_kv8_attention")}


def _attention_workspace_bytes(name, cache, num_q_heads, num_tokens, num_reqs, table_width, window, max_request_tokens,
                               max_seq_len) -> int:
    any_ptr = cache.desc.k_codes  # sizes alone matter here
    b = capi.ple_kv4_batch(any_ptr, any_ptr, any_ptr, int(num_tokens), int(num_reqs), int(table_width),
                           min(int(max_request_tokens), _MOST), min(int(max_seq_len), _MOST))
    return int(getattr(capi.load(), _WORKSPACE[name])(int(num_q_heads), ctypes.byref(cache.desc), ctypes.byref(b),
                                                      min(int(window), _MOST)))


def ple_kv4_attention_workspace_bytes(cache: KV4Cache, num_q_heads: int, num_tokens: int, num_reqs: int,
                                      table_width: int, *, window: int = 0, max_request_tokens: int = 0,
                                      max_seq_len: int = 0) -> int:
    """Workspace of a call with these sizes and hints (0: none is needed)."""
    return _attention_workspace_bytes("ple_kv4_attention", cache, num_q_heads, num_tokens, num_reqs, table_width, window,
                                      max_request_tokens, max_seq_len)


def _attention(name, q, cache, query_start_loc, seq_lens, page_table, window, scale, max_request_tokens, max_seq_len, want_lse,
               out, lse, workspace, stream):
    """What the attentions over the paged caches share; name: the library's call."""
    D, T, window = cache.head_dim, q.shape[0], min(window, _MOST)
    qs, hq = _heads("q", q, T, None, cache), q.shape[1]
    out = _out("out", out, (T, hq, D), _BF16, cache, stream)
    if lse is not None or want_lse:
        lse = _out("lse", lse, (T, hq), _F32, cache, stream)
    b = _kv4_batch(cache, query_start_loc, seq_lens, page_table, T, max_request_tokens, max_seq_len)
    if q.get_device() != cache.device:
        _same_device(cache.tensors[0], q)
    lib = capi.load()
    desc, batch = ctypes.byref(cache.desc), ctypes.byref(b)
    need = getattr(lib, _WORKSPACE[name])(hq, desc, batch, window)
    if workspace is None:
        if need > 0:  # (given up on return, before the work has ended: taken in the order of the stream it runs on)
            if stream is None:
                workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
            else:
                with _on(stream, q.device):
                    workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
    else:
        _req_bytes("workspace", workspace, need)
        _same_device(cache.tensors[0], workspace)
    rc = getattr(lib, name)(
        q.data_ptr(), qs, hq, desc, batch, window,
        D ** -0.5 if scale is None else scale, _ptr(out), _ptr(lse),
        None if workspace is None else _ptr(workspace), 0 if workspace is None else _nbytes(workspace),
        _raw_stream(cache.device) if stream is None else _given(stream, cache.device))
    if rc:
        capi.check(rc, name)
    return out, lse


def ple_kv4_attention(q, cache: KV4Cache, query_start_loc, seq_lens, page_table, *, window: int = 0, scale=None,
                      max_request_tokens: int = 0, max_seq_len: int = 0, want_lse: bool = False, out=None, lse=None,
                      workspace=None, stream=None):
    """Causal attention of the new tokens q bf16 [T][q heads][D] over the cache (their own keys appended before).
    scale: 1/sqrt(D) if None.  window: tokens seen, the own one included (0: all).  max_request_tokens and
    max_seq_len (0: unknown) let the call size its launch; pass them (the launch is that of the longest requests: long
    prefills and many single tokens take less time in two calls).  Returns (out bf16 [T][q heads][D], lse fp32
    [T][q heads] or None)."""
    return _attention("ple_kv4_attention", q, cache, query_start_loc, seq_lens, page_table, window, scale,
                      max_request_tokens, max_seq_len, want_lse, out, lse, workspace, stream)
