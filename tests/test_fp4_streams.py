"""Memory that a call of the 4-bit operators makes itself, on a stream other than the current one."""
import contextlib

import pytest
import torch

import fp4_util as U
import layer_embedding_lookup_amd as ple
from layer_embedding_lookup_amd import capi, fp4

BF, I32 = torch.bfloat16, torch.int32


class Weight:
    k_dim, out_dim, codes, desc, device = 128, 64, None, capi.ple_w4_weight(), -1


@pytest.fixture
def made(monkeypatch):
    """The binding over host tensors with a library that does nothing; yields every allocation with the stream whose
    order it was made in."""
    log, at = [], [None]

    class Lib:
        def __getattr__(self, name):
            return lambda *args: 4096 if name.endswith("_bytes") else 0

    @contextlib.contextmanager
    def stream(s):
        at.append(s)
        yield
        at.pop()

    def noting(f):
        def g(*args, **kw):
            t = f(*args, **kw)
            log.append((tuple(t.shape), at[-1]))
            return t
        return g

    monkeypatch.setattr(capi, "load", lambda: Lib())
    monkeypatch.setattr(fp4, "_same_device", lambda *t: None)
    monkeypatch.setattr(fp4, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: None)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: None)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    monkeypatch.setattr(torch, "empty_strided", noting(torch.empty_strided))
    return log


class Side:
    cuda_stream = 77


@pytest.mark.parametrize("stream,order", [(None, None), (Side, Side), (77, 77), (0, "default")])
def test_made_in_the_order_of_the_call(made, stream, order):
    c = object.__new__(ple.KV4Cache)
    c.tensors, c.device, c._workspaces = (torch.zeros((4, 2, 16, 64), dtype=torch.uint8),), -1, {}
    c.num_pages, c.num_kv_heads, c.page_size, c.head_dim, c.desc = 4, 2, 16, 128, capi.ple_kv4_cache()
    k, q = torch.zeros((3, 2, 128), dtype=BF), torch.zeros((3, 4, 128), dtype=BF)
    args = (torch.tensor([0, 3], dtype=I32), torch.tensor([3], dtype=I32), torch.zeros((1, 2), dtype=I32))
    made.clear()
    ple.ple_w4_linear(torch.zeros((5, 128), dtype=BF), Weight, stream=stream)
    ple.ple_kv4_append(c, k, k, *args, q=q, stream=stream)
    ple.ple_kv4_read(c, *args, 3, stream=stream)
    ple.ple_kv4_attention(q, c, *args, want_lse=True, stream=stream)
    shapes = [(5, 64), (3, 4, 128), (3, 2, 128), (3, 2, 128), (3, 4, 128), (3, 4), (4096,)]
    assert [m for m in made if m[0] in shapes] == [(s, order) for s in shapes]


DEV = "cuda:0"


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("what", ["workspace", "out", "lse", "q_out", "read", "linear"])
def test_leaves_alone_what_the_current_stream_still_reads(what, handle):
    """Blocks given back to the current stream's pool while its queue still reads them: a call on another stream, which
    waits for nothing here, must not take them."""
    g = torch.Generator().manual_seed(31)
    cache = U.Cache(g, [2500], H=1, D=128, page=16)
    c = ple.KV4Cache(*cache.tensors(DEV))
    T = 64 if what in ("q_out", "read", "linear") else 1
    args = (torch.tensor([0, T], dtype=I32, device=DEV), torch.tensor([2500], dtype=I32, device=DEV), cache.table.to(DEV))
    q, k = (torch.randn((T, h, 128), generator=g).to(BF).to(DEV) for h in (8, 1))
    w = ple.W4Weight.nvfp4(torch.randint(0, 256, (192, 64), generator=g).to(torch.uint8).to(DEV),
                           torch.randint(0, 0x60, (192, 8), generator=g).to(torch.uint8).to(DEV), torch.ones(1, device=DEV))
    need = ple.ple_kv4_attention_workspace_bytes(c, 8, 1, 1, cache.width, max_request_tokens=1, max_seq_len=2500)
    assert need > 0
    size = {"workspace": need, "out": 8 * 128 * 2, "lse": 8 * 4, "q_out": T * 8 * 256, "read": T * 256, "linear": T * 384}[what]

    def call(**kw):
        if what == "q_out":
            return (ple.ple_kv4_append(c, k, k, *args, q=q, **kw),)
        if what == "read":
            return ple.ple_kv4_read(c, *args, T, **kw)
        if what == "linear":
            return (ple.ple_w4_linear(k.view(T, 128), w, **kw),)
        return ple.ple_kv4_attention(q, c, *args, max_request_tokens=1, max_seq_len=2500, want_lse=True, **kw)

    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    blocks = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(4)]
    copies = [torch.empty_like(b) for b in blocks]
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)  # about 25 ms
    for a, b in zip(copies, blocks):
        a.copy_(b)
    del a, b, blocks
    got = call(stream=side.cuda_stream if handle else side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in copies)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.gpu
def test_a_call_on_a_forked_stream_in_a_graph():
    """Captured on a stream that forks off the capturing one, workspace and outputs made by the calls; every replay
    against the eager result, with eager work of the same size between them."""
    g = torch.Generator().manual_seed(32)
    cache = U.Cache(g, [2500, 900], H=1, D=128, page=16)
    c = ple.KV4Cache(*cache.tensors(DEV))
    args = (torch.tensor([0, 1, 2], dtype=I32, device=DEV), torch.tensor([2500, 900], dtype=I32, device=DEV), cache.table.to(DEV))
    kw = dict(max_request_tokens=1, max_seq_len=2500, want_lse=True)
    q = torch.randn((2, 8, 128), generator=g).to(BF).to(DEV)
    w = ple.W4Weight.nvfp4(torch.randint(0, 256, (192, 512), generator=g).to(torch.uint8).to(DEV),
                           torch.randint(0, 0x60, (192, 64), generator=g).to(torch.uint8).to(DEV), torch.ones(1, device=DEV))

    def calls(stream):
        out, lse = ple.ple_kv4_attention(q, c, *args, stream=stream, **kw)
        return out, lse, ple.ple_w4_linear(out.view(2, 1024), w, stream=stream)

    calls(None)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = calls(side)
        torch.cuda.current_stream().wait_stream(side)
    for i in range(4):
        q.normal_(generator=torch.Generator(device=DEV).manual_seed(i))
        want = calls(None)
        graph.replay()
        calls(None)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
