"""Tensors of the 4-bit and 8-bit decode operators on another device than the current one: a call that would land on the
current device's default stream is refused by name.  On the CPU, with a library that notes its calls and tensors that say they
are on device 1."""
import pytest
import torch

import layer_embedding_lookup_amd as ple
from layer_embedding_lookup_amd import bits8, capi, fp4
from test_bits8_streams import Weight as Weight8
from test_bits8_streams import host_cache
from test_fp4_arguments import ARGS, K, Q, Weight, cache, calls  # noqa: F401  (fixtures)

BF, I8 = torch.bfloat16, torch.int8


class Default:
    """A device's default stream."""
    cuda_stream = 0


def operators(kv4):
    """Every operator with a stream, its outputs given."""
    kv8, x, w = host_cache(), torch.zeros((5, 128), dtype=BF), torch.zeros(128, dtype=BF)
    kv4.device = kv8.device = 1
    w4, w8 = type("W", (Weight,), dict(device=1)), type("W", (Weight8,), dict(device=1))
    out = dict(codes=8192, scales=12288, residual_out=4096)
    return {
        "ple_w4_linear": lambda s: ple.ple_w4_linear(x, w4, out=4096, stream=s),
        "ple_w8_linear": lambda s: ple.ple_w8_linear(torch.zeros((5, 128), dtype=I8), 8192, w8, out=4096, stream=s),
        "ple_kv4_append": lambda s: ple.ple_kv4_append(kv4, K, K, *ARGS, stream=s),
        "ple_kv8_append": lambda s: ple.ple_kv8_append(kv8, K, K, *ARGS, stream=s),
        "ple_kv4_read": lambda s: ple.ple_kv4_read(kv4, *ARGS, 3, k_out=4096, v_out=8192, stream=s),
        "ple_kv8_read": lambda s: ple.ple_kv8_read(kv8, *ARGS, 3, k_out=4096, v_out=8192, stream=s),
        "ple_kv4_attention": lambda s: ple.ple_kv4_attention(Q, kv4, *ARGS, out=4096, workspace=64, stream=s),
        "ple_kv8_attention": lambda s: ple.ple_kv8_attention(Q, kv8, *ARGS, out=4096, workspace=64, stream=s),
        "ple_rms_norm8": lambda s: ple.ple_rms_norm8(x, w, residual=4096, stream=s, **out),
    }


@pytest.mark.parametrize("stream", [None, Default], ids=["current", "default"])
def test_default_streams_of_other_devices(calls, cache, monkeypatch, stream):  # noqa: F811
    monkeypatch.setattr(bits8, "_same_device", lambda *t: None)
    monkeypatch.setattr(fp4, "_get_raw_stream", lambda device: 0)
    for now in (0, 1):
        monkeypatch.setattr(fp4, "_get_device", lambda: now)
        for name, call in operators(cache).items():
            if name == "ple_rms_norm8":                       # (goes by its tensors' own device, which is the CPU's -1 here)
                continue
            calls.clear()
            if now == 0:
                with pytest.raises(ValueError, match="tensors are on cuda:1, the current device is cuda:0"):
                    call(stream)
                assert name not in calls
            else:
                call(stream)
                assert name in calls
    with pytest.raises(ValueError, match="the current device is cuda:1"):
        operators(cache)["ple_rms_norm8"](stream)


def test_other_streams_know_their_device(calls, cache, monkeypatch):  # noqa: F811
    """A stream of one's own, or a handle, is taken as it is."""
    monkeypatch.setattr(bits8, "_same_device", lambda *t: None)
    monkeypatch.setattr(fp4, "_get_device", lambda: 0)
    for name, call in operators(cache).items():
        call(9)
        assert calls[name][-1] == 9
