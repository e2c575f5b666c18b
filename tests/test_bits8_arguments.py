"""What the binding of the 8-bit decode operators hands to the library: raw addresses as the other calls take them, and
numbers beyond 32 bits.  On the CPU, with a library that notes its arguments."""
import pytest
import torch

import layer_embedding_lookup_amd as ple
from layer_embedding_lookup_amd import bits8
from test_bits8_streams import Weight, host_cache
from test_fp4_arguments import ARGS, K, MOST, Q, calls  # noqa: F401  (the fixture)

BF, I8 = torch.bfloat16, torch.int8


@pytest.fixture(autouse=True)
def any_device(monkeypatch):
    monkeypatch.setattr(bits8, "_same_device", lambda *t: None)


def test_raw_addresses(calls):  # noqa: F811
    cache = host_cache()
    x, w = torch.zeros((5, 128), dtype=BF), torch.zeros(128, dtype=BF)
    assert ple.ple_rms_norm8(x, w, residual=4096, codes=8192, scales=12288, residual_out=4096, stream=9) == (8192, 12288, 4096)
    args = calls["ple_rms_norm8"]
    assert args[1:3] == [128, 4096] and args[7:10] == [8192, 12288, 4096]
    assert ple.ple_w8_linear(torch.zeros((5, 128), dtype=I8), 8192, Weight, out=4096, stream=9) == 4096
    assert calls["ple_w8_linear"][2] == 8192 and calls["ple_w8_linear"][5] == 4096
    assert ple.ple_kv8_append(cache, K, K, *ARGS, q=Q, q_out=4096, stream=9) == 4096
    assert calls["ple_kv8_append"][9] == 4096
    assert ple.ple_kv8_read(cache, *ARGS, 3, k_out=4096, v_out=8192, stream=9) == (4096, 8192)
    assert calls["ple_kv8_read"][2:4] == [4096, 8192]
    lens = (ARGS[0], 777 * 16, ARGS[2])
    assert ple.ple_kv8_attention(Q, cache, *lens, out=4096, lse=8192, workspace=64, stream=9) == (4096, 8192)
    args = calls["ple_kv8_attention"]
    assert args[7:10] == [4096, 8192, 64] and args[4].seq_lens == 777 * 16


def test_numbers_beyond_32_bits(calls):  # noqa: F811
    """A window, or a hint, wider than an int32 is the widest one, not what its low 32 bits say."""
    cache = host_cache()
    for big in (MOST, MOST + 1, 2 ** 32 + 5, 2 ** 63 - 1):
        ple.ple_kv8_attention(Q, cache, *ARGS, window=big, max_request_tokens=big, max_seq_len=big, out=Q, stream=9)
        args = calls["ple_kv8_attention"]
        assert args[5] == MOST and args[4].max_request_tokens == MOST and args[4].max_seq_len == MOST
        ple.ple_kv8_append(cache, K, K, *ARGS, max_request_tokens=big, stream=9)
        assert calls["ple_kv8_append"][1].max_request_tokens == MOST
        cache.desc.k_codes = 16
        ple.ple_kv8_attention_workspace_bytes(cache, 4, 3, 1, 2, window=big, max_request_tokens=big, max_seq_len=big)
        args = calls["ple_kv8_attention_workspace_bytes"]
        assert args[3] == MOST and args[2].max_request_tokens == MOST and args[2].max_seq_len == MOST
    ple.ple_kv8_attention(Q, cache, *ARGS, window=-1, out=Q, stream=9)
    assert calls["ple_kv8_attention"][5] == -1  # (refused by the library)


def test_a_growing_sequence_leaves_nothing_behind(calls):  # noqa: F811
    """A decode loop that passes its longest length as it grows: the cache object holds no more after it than before."""
    cache = host_cache()

    def held():
        return {name: len(v) for name, v in vars(cache).items() if hasattr(v, "__len__")}
    before = held()
    for n in range(1, 100):
        ple.ple_kv8_attention(Q, cache, *ARGS, max_request_tokens=3, max_seq_len=n, stream=9, out=Q)
    assert held() == before
