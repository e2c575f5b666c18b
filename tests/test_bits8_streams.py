"""The 8-bit decode operators on streams and in graphs: memory that a call makes itself on a stream other than the current
one, captured and replayed calls, and a run of them all as a decode step uses them."""
import pytest
import torch

import bits8_util as U
import layer_embedding_lookup_amd as ple
from layer_embedding_lookup_amd import capi
from test_fp4_streams import Side, made  # noqa: F401  (the fixture)

BF, I8, I32 = torch.bfloat16, torch.int8, torch.int32
DEV = "cuda:0"


def host_cache():
    c = object.__new__(ple.KV8Cache)
    c.tensors, c.device, c._workspaces = (torch.zeros((4, 2, 1, 8, 16, 16), dtype=torch.uint8),), -1, {}
    c.num_pages, c.num_kv_heads, c.page_size, c.head_dim, c.desc = 4, 2, 16, 128, capi.ple_kv8_cache()
    return c


class Weight:
    k_dim, out_dim, codes, desc, device = 128, 64, None, capi.ple_w8_weight(), -1


@pytest.mark.parametrize("stream,order", [(None, None), (Side, Side), (77, 77), (0, "default")])
def test_made_in_the_order_of_the_call(made, monkeypatch, stream, order):  # noqa: F811
    from layer_embedding_lookup_amd import bits8
    monkeypatch.setattr(bits8, "_same_device", lambda *t: None)
    monkeypatch.setattr(bits8, "_raw_stream", lambda device: 0)
    k, q = torch.zeros((3, 2, 128), dtype=BF), torch.zeros((3, 4, 128), dtype=BF)
    args = (torch.tensor([0, 3], dtype=I32), torch.tensor([3], dtype=I32), torch.zeros((1, 2), dtype=I32))
    x, w = torch.zeros((7, 32), dtype=BF), torch.zeros(32, dtype=BF)
    codes, scales = torch.zeros((5, 128), dtype=I8), torch.zeros(5)
    c = host_cache()
    made.clear()
    ple.ple_rms_norm8(x, w, residual=x, stream=stream)
    ple.ple_w8_linear(codes, scales, Weight, stream=stream)
    ple.ple_kv8_append(c, k, k, *args, q=q, stream=stream)
    ple.ple_kv8_read(c, *args, 3, stream=stream)
    ple.ple_kv8_attention(q, c, *args, want_lse=True, stream=stream)
    shapes = [(7, 32), (7, 32), (7,), (5, 64), (3, 4, 128), (3, 2, 128), (3, 2, 128), (3, 4, 128), (3, 4), (4096,)]
    assert made == [(s, order) for s in shapes]


class Step:
    """A decode step's operators over small tensors: norm, projection, append, attention, norm, projection."""

    def __init__(self, seed, lens, D=128, Hq=8, H=2, hidden=512, page=16, room=64):
        g = torch.Generator().manual_seed(seed)
        self.D, self.Hq, self.H, self.R = D, Hq, H, len(lens)
        self.host = U.Cache(g, [n + room for n in lens], H=H, D=D, page=page, poison=False)
        self.cache = ple.KV8Cache(*self.host.tensors(DEV))
        self.kept = [t.clone() for t in self.cache.tensors]
        self.start = torch.arange(self.R + 1, dtype=I32, device=DEV)
        self.lens = torch.tensor(lens, dtype=I32, device=DEV)
        self.table = self.host.table.to(DEV)
        self.most = max(lens) + room
        self.inv = torch.logspace(0, -4, D // 2).to(DEV)
        weight = lambda o, k: ple.W8Weight(torch.randint(-127, 128, (o, k), generator=g).to(I8).to(DEV),  # noqa: E731
                                           (torch.rand(o, generator=g) * 2e-3).to(DEV))
        self.qkv, self.out = weight((Hq + 2 * H) * D, hidden), weight(hidden, Hq * D)
        self.norms = [torch.randn(n, generator=g).to(BF).to(DEV) for n in (hidden, Hq * D)]
        self.x, self.h = (torch.randn((self.R, hidden), generator=g).to(BF).to(DEV) for _ in range(2))

    def restore(self):
        for a, b in zip(self.cache.tensors, self.kept):
            a.copy_(b)

    def __call__(self, stream=None, workspace=None):
        kw = dict(stream=stream)
        codes, scales, h = ple.ple_rms_norm8(self.x, self.norms[0], residual=self.h, **kw)
        heads = ple.ple_w8_linear(codes, scales, self.qkv, **kw).view(self.R, -1, self.D)
        a, b = self.Hq, self.Hq + self.H
        where = (self.start, self.lens, self.table)
        q = ple.ple_kv8_append(self.cache, heads[:, a:b], heads[:, b:], *where, inv_freq=self.inv, q=heads[:, :a],
                               max_request_tokens=1, **kw)
        att, lse = ple.ple_kv8_attention(q, self.cache, *where, max_request_tokens=1, max_seq_len=self.most, want_lse=True,
                                         workspace=workspace, **kw)
        codes, scales, _ = ple.ple_rms_norm8(att.view(self.R, -1), self.norms[1], **kw)
        return (h, heads, q, att, lse, codes, scales, ple.ple_w8_linear(codes, scales, self.out, **kw))


@pytest.mark.gpu
def test_a_run_of_them_together():
    """Each operator's definition in 64 bits over what the one before it gave."""
    import test_bits8_gpu as G
    s = Step(50, [300, 1, 47, 1000])
    before = {k: s.host.codes[k].clone() for k in "kv"}
    h, heads, q, att, lse, codes, scales, y = s()
    norm = ple.ple_rms_norm8(s.x, s.norms[0], residual=s.h)
    G.check_norm(s.x.cpu(), s.norms[0].cpu(), s.h.cpu(), 1e-6, norm)
    assert torch.equal(norm[2], h)
    G.check_linear(norm[0].cpu(), norm[1].cpu(), s.qkv.codes.cpu(), s.qkv.scales.cpu(), heads.view(s.R, -1))
    hc, a, b, qsl, lens = heads.cpu(), s.Hq, s.Hq + s.H, list(range(s.R + 1)), s.lens.tolist()
    turned = U.rotate(hc[:, a:b], s.lens.cpu().long() - 1, s.inv.cpu(), False)
    got = {"k": s.host.append("k", turned, qsl, lens), "v": s.host.append("v", hc[:, b:].to(torch.float64), qsl, lens)}
    after = G.check_append(s.host, before, got, s.cache.tensors)
    want, want_lse, tol, tol_lse = U.attention(after, q.cpu(), qsl, s.lens.cpu())
    assert ((att.cpu().double() - want).abs() <= tol).all() and ((lse.cpu().double() - want_lse).abs() <= tol_lse).all()
    G.check_norm(att.view(s.R, -1).cpu(), s.norms[1].cpu(), None, 1e-6, (codes, scales, None))
    G.check_linear(codes.cpu(), scales.cpu(), s.out.codes.cpu(), s.out.scales.cpu(), y)


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [False, True])
def test_two_graphs_replayed_in_turn(shared):
    """Two captured steps, with workspaces of their own or one of the caller's for both, eager steps and synchronisation
    between replays, each replay against the eager result to the bit."""
    s, t = Step(51, [700, 2500]), Step(52, [1500, 40, 3])
    need = [ple.ple_kv8_attention_workspace_bytes(x.cache, x.Hq, x.R, x.R, x.table.shape[1], max_request_tokens=1, max_seq_len=x.most)
            for x in (s, t)]
    assert min(need) > 0
    ws = torch.empty(max(need), dtype=torch.uint8, device=DEV) if shared else None
    for x in (s, t):
        x(workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for x in (s, t):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = x(workspace=ws)
        graphs.append((x, graph, got))
    for i in range(4):
        for x, graph, got in graphs:
            x.x.normal_(generator=torch.Generator(device=DEV).manual_seed(i))
            x.restore()
            want = [y.clone() for y in x(workspace=ws)]
            held = [y.clone() for y in x.cache.tensors]
            x.restore()
            graph.replay()
            if i % 2:
                torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
            assert all(torch.equal(a.view(I8 if a.dtype == torch.uint8 else I32), b.view(I8 if b.dtype == torch.uint8 else I32))
                       for a, b in zip(x.cache.tensors, held))


@pytest.mark.gpu
def test_a_call_on_a_forked_stream_in_a_graph():
    """Captured on a stream that forks off the capturing one; a step moves the lengths on, so every replay appends one token
    more."""
    s = Step(53, [2500, 900])
    first = s.lens.clone()

    def calls(stream):
        with torch.cuda.stream(stream):
            s.lens.add_(1)
        return s(stream=stream)

    calls(torch.cuda.current_stream())
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = calls(side)
        torch.cuda.current_stream().wait_stream(side)
    want = []
    for _ in range(2):
        s.lens.copy_(first)
        s.restore()
        for i in range(20):                                   # more than a block of 16 tokens
            s.x.normal_(generator=torch.Generator(device=DEV).manual_seed(i))
            if len(want) < 20:
                want.append([y.clone() for y in calls(torch.cuda.current_stream())])
            else:
                graph.replay()
                torch.cuda.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i


@pytest.mark.gpu
def test_two_calls_at_once():
    """Steps over two caches on two streams at the same time, workspaces and outputs of their own."""
    pair = [Step(54, [2500, 900]), Step(55, [1300, 1300, 5])]
    streams = [torch.cuda.Stream() for _ in pair]
    want = [[y.clone() for y in s()] for s in pair]
    for s in pair:
        s.restore()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):                                        # (the second and later steps write the same token again)
        for s, stream in zip(pair, streams):
            got.append((s, s(stream=stream)))
    torch.cuda.synchronize()
    for i, (s, ys) in enumerate(got):
        # the first step finds the block as it was; a repeated one too, but for its grown scale
        if i < 2:
            assert all(torch.equal(a, b) for a, b in zip(ys, want[pair.index(s)]))
        assert all(torch.isfinite(y.float()).all() for y in ys)


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("what", ["workspace", "out", "lse", "q_out", "read", "linear", "codes", "residual_out"])
def test_leaves_alone_what_the_current_stream_still_reads(what, handle):
    """Blocks given back to the current stream's pool while its queue still reads them: a call on another stream, which
    waits for nothing here, must not take them."""
    g = torch.Generator().manual_seed(31)
    cache = U.Cache(g, [2500], H=1, D=128, page=16)
    c = ple.KV8Cache(*cache.tensors(DEV))
    T = 1 if what in ("workspace", "out", "lse") else 64
    args = (torch.tensor([0, T], dtype=I32, device=DEV), torch.tensor([2500], dtype=I32, device=DEV), cache.table.to(DEV))
    q, k = (torch.randn((T, h, 128), generator=g).to(BF).to(DEV) for h in (8, 1))
    codes, scales = torch.randint(-128, 128, (T, 128), generator=g).to(I8).to(DEV), torch.ones(T, device=DEV)
    w = ple.W8Weight(torch.randint(-128, 128, (192, 128), generator=g).to(I8).to(DEV), torch.ones(192, device=DEV))
    ones = torch.ones(128, dtype=BF, device=DEV)
    need = ple.ple_kv8_attention_workspace_bytes(c, 8, 1, 1, cache.width, max_request_tokens=1, max_seq_len=2500)
    assert need > 0
    size = {"workspace": need, "out": 8 * 128 * 2, "lse": 8 * 4, "q_out": T * 8 * 256, "read": T * 256, "linear": T * 384,
            "codes": T * 128, "residual_out": T * 256}[what]

    def call(**kw):
        if what == "q_out":
            return (ple.ple_kv8_append(c, k, k, *args, q=q, **kw),)
        if what == "read":
            return ple.ple_kv8_read(c, *args, T, **kw)
        if what == "linear":
            return (ple.ple_w8_linear(codes, scales, w, **kw),)
        if what in ("codes", "residual_out"):
            return [t for t in ple.ple_rms_norm8(k.view(T, 128), ones, residual=k.view(T, 128) if what != "codes" else None, **kw)
                    if t is not None]
        return ple.ple_kv8_attention(q, c, *args, max_request_tokens=1, max_seq_len=2500, want_lse=True, **kw)

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
