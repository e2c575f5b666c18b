"""What the binding of the 4-bit operators hands to the library: raw addresses as the other calls take them, and numbers
beyond 32 bits.  On the CPU, with a library that notes its arguments."""
import pytest
import torch

import layer_embedding_lookup_amd as ple
from layer_embedding_lookup_amd import capi, fp4

BF, I32 = torch.bfloat16, torch.int32
MOST = 2 ** 31 - 1


class Weight:
    k_dim, out_dim, codes, desc, device = 128, 64, None, capi.ple_w4_weight(), -1


@pytest.fixture
def calls(monkeypatch):
    log = {}

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                log[name] = [getattr(a, "_obj", a) for a in args]
                return 0
            return call

    monkeypatch.setattr(capi, "load", lambda: Lib())
    monkeypatch.setattr(fp4, "_same_device", lambda *t: None)
    return log


@pytest.fixture
def cache():
    c = object.__new__(ple.KV4Cache)
    c.tensors, c.device, c._workspaces = (torch.zeros((4, 2, 16, 64), dtype=torch.uint8),), -1, {}
    c.num_pages, c.num_kv_heads, c.page_size, c.head_dim, c.desc = 4, 2, 16, 128, capi.ple_kv4_cache()
    return c


ARGS = (torch.tensor([0, 3], dtype=I32), torch.tensor([3], dtype=I32), torch.zeros((1, 2), dtype=I32))
K, Q = torch.zeros((3, 2, 128), dtype=BF), torch.zeros((3, 4, 128), dtype=BF)


def test_raw_addresses(calls, cache):
    assert ple.ple_w4_linear(torch.zeros((5, 128), dtype=BF), Weight, out=4096, stream=9) == 4096
    assert calls["ple_w4_linear"][4] == 4096
    assert ple.ple_kv4_append(cache, K, K, *ARGS, q=Q, q_out=4096, stream=9) == 4096
    assert calls["ple_kv4_append"][9] == 4096
    assert ple.ple_kv4_read(cache, *ARGS, 3, k_out=4096, v_out=8192, stream=9) == (4096, 8192)
    assert calls["ple_kv4_read"][2:4] == [4096, 8192]
    lens = (ARGS[0], 777 * 16, ARGS[2])
    assert ple.ple_kv4_attention(Q, cache, *lens, out=4096, lse=8192, workspace=64, stream=9) == (4096, 8192)
    args = calls["ple_kv4_attention"]
    assert args[7:10] == [4096, 8192, 64] and args[4].seq_lens == 777 * 16


def test_numbers_beyond_32_bits(calls, cache):
    """A window, or a hint, wider than an int32 is the widest one, not what its low 32 bits say."""
    for big in (MOST, MOST + 1, 2 ** 32 + 5, 2 ** 63 - 1):
        ple.ple_kv4_attention(Q, cache, *ARGS, window=big, max_request_tokens=big, max_seq_len=big, out=Q, stream=9)
        args = calls["ple_kv4_attention"]
        assert args[5] == MOST and args[4].max_request_tokens == MOST and args[4].max_seq_len == MOST
        cache.desc.k_codes = 16
        ple.ple_kv4_attention_workspace_bytes(cache, 4, 3, 1, 2, window=big, max_request_tokens=big, max_seq_len=big)
        args = calls["ple_kv4_attention_workspace_bytes"]
        assert args[3] == MOST and args[2].max_request_tokens == MOST and args[2].max_seq_len == MOST
    ple.ple_kv4_attention(Q, cache, *ARGS, window=-1, out=Q, stream=9)
    assert calls["ple_kv4_attention"][5] == -1  # (refused by the library)


def test_a_growing_sequence_leaves_nothing_behind(calls, cache):
    """A decode loop that passes its longest length as it grows: the cache object holds no more after it than before."""
    def held():
        return {name: len(v) for name, v in vars(cache).items() if hasattr(v, "__len__")}
    before = held()
    for n in range(1, 100):
        ple.ple_kv4_attention(Q, cache, *ARGS, max_request_tokens=3, max_seq_len=n, stream=9, out=Q)
    assert held() == before
