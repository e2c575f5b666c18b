"""The 8-bit decode operators as measured cases: the residual's addition and RMS
norm with an 8-bit output (ple_rms_norm8), products of 8-bit integers
(ple_w8_linear), appending rotated keys and values to a paged 8-bit cache
(ple_kv8_append, read back by ple_kv8_read) and attention over that cache
(ple_kv8_attention).

`own` false computes them in plain torch operations, true through the
framework's entry points; both on the same tensors, in the formats of
include/ple_8bit.h:

  inputs   codes int8 [T][K], one fp32 scale per token
  weights  codes int8 [O][K], one fp32 scale per output channel
  cache    e4m3fn codes uint8, keys [pages][heads][page_size/16][D/16]
           [16 tokens][16], values [pages][heads][page_size/16][D][16 tokens],
           and for each one fp32 scale per block of 16 tokens and head
           [pages][heads][page_size/16]
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
BLOCK = 16                   # tokens that share a scale
MOST, LEAST = 2.0 ** 32, 2.0 ** -32  # range of the cache's scales


# ---- cases ----

def listed():
    return [
        # one user's decode step: the token's residual stream normalised for the next projection, 4096 wide; latency
        dict(name="norm_1", kind="norm", T=1, N=4096, residual=True),
        # a prefill's tokens, ragged prompts together: bound by reading and writing the residual stream
        dict(name="norm_8k", kind="norm", T=7984, N=4096, residual=True),
        # one token through the key/value projection of a 4096-wide layer: bound by reading the weights
        dict(name="linear_1", kind="linear", T=1, K=4096, O=8192),
        # odd sizes: a token count and widths that fill no tile, rows that end inside a step
        dict(name="linear_odd", kind="linear", T=37, K=4112, O=5003),
        # the decode batch of 256 requests through its key/value projection (8 heads of 256 -> 2 x 2048)
        dict(name="linear_256", kind="linear", T=256, K=2048, O=4096),
        # a prefill of 8k tokens through the key/value projection: bound by the products
        dict(name="linear_8k", kind="linear", T=8192, K=4096, O=8192),
        # a decode step's new keys and values, one token of each of 256 requests, far positions, query rotated too
        dict(name="append_decode_256", kind="append", R=256, new=1, past=60000, Hq=32, Hkv=8, D=128, page=16, rot=128,
             interleaved=False),
        # a prefill's keys and values, ragged prompts behind cached ones, half of each head rotated, neighbouring pairs
        dict(name="append_prefill_8k", kind="append", R=5, new=1638, past=300, Hq=32, Hkv=8, D=128, page=64, rot=64,
             interleaved=True),
        # one user's long context: the work has to be split along the cache
        dict(name="attn_1x100k", kind="attention", R=1, new=1, past=100100, Hq=32, Hkv=8, D=128, page=64, window=0),
        # a full decode batch, ragged lengths up to 6000: bound by reading the cache
        dict(name="attn_256x6k", kind="attention", R=256, new=1, past=6000, Hq=32, Hkv=8, D=128, page=64, window=0),
        # verify windows of up to 4 drafts with a sliding window, 8 query heads to a key head
        dict(name="attn_spec_64x4", kind="attention", R=64, new=4, past=4090, Hq=32, Hkv=4, D=128, page=32, window=1024),
        # a chunk of a prefill behind cached context: bound by the products
        dict(name="attn_chunk_2x1500", kind="attention", R=2, new=1500, past=5000, Hq=32, Hkv=8, D=128, page=64, window=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "linear", "linear", "append", "attention", "attention"])
    if kind == "norm":
        N = 16 * _log(rng, 16, 512)
        return dict(kind=kind, T=_log(rng, 1, min(8192, 7984 * 4096 // N)), N=N, residual=rng.random() < 0.7)
    if kind == "linear":
        return dict(kind=kind, T=_log(rng, 1, 4096), K=16 * _log(rng, 32, 512), O=_log(rng, 300, 8192))
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8] if Hkv < 8 else [1, 2, 4])
    page = rng.choice([16, 32, 48, 64, 128])
    if kind == "append":
        R = _log(rng, 1, 256)
        new = max(1, min(_log(rng, 1, 4000), 8192 // R))
        rot = rng.choice([D, D // 2, D // 4])
        return dict(kind=kind, R=R, new=new, past=_log(rng, 1, 200000 // R), Hq=Hq, Hkv=Hkv, D=D, page=page, rot=rot,
                    interleaved=rng.random() < 0.5)
    form = rng.choice(["decode", "decode", "verify", "chunk"])
    R = _log(rng, 1, 200) if form == "decode" else _log(rng, 1, 64) if form == "verify" else rng.choice([1, 2, 3])
    new = 1 if form == "decode" else rng.choice([2, 3, 4, 5, 8]) if form == "verify" else _log(rng, 17, 1000)
    most = 500000 if form == "decode" else 200000 if form == "verify" else 12000
    past = _log(rng, 1, max(2, min(100000, most * 8 // (R * Hkv) * 128 // D // 4)) if form != "chunk" else 4000)
    return dict(kind=kind, R=R, new=new, past=past, Hq=Hq, Hkv=Hkv, D=D, page=page,
                window=rng.choice([0, 0, 128, 1000]))


# ---- formats ----

def _block_scale(top):
    """The power of two that a block's largest magnitude asks for: the least s with top <= 448 s, within the range."""
    m, e = torch.frexp(top.float())  # top = m 2^e, 1/2 <= m < 1;  448 = 7/8 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), LEAST).clamp(LEAST, MOST).float()


def _e4m3(x):
    """fp32 values to e4m3fn codes, to the nearest, ties to the even one."""
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _value(codes, dtype=torch.float32):
    return codes.view(torch.float8_e4m3fn).to(torch.float32).to(dtype)


def _laid_out(codes, name):
    """Blocks of codes [...][16 tokens][D] as the cache holds them."""
    return codes.unflatten(-1, (-1, 16)).transpose(-3, -2) if name == "k" else codes.transpose(-1, -2)


def _in_order(held, name):
    """And back."""
    return held.transpose(-3, -2).flatten(-2) if name == "k" else held.transpose(-1, -2)


def _tokens(s, name, page, place):
    """The codes of tokens at these places of these pages, [...][heads][D]."""
    codes = s[name + "_codes"][page, :, place // BLOCK, :, place % BLOCK]
    return codes.flatten(-2) if name == "k" else codes


# ---- states ----

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    if case["kind"] == "norm":
        T, N = case["T"], case["N"]
        # a residual stream: tokens of different size, a few channels much larger than the others
        wide = 1 + 20 * (torch.rand(N, generator=g, device=DEV) < 0.004)
        s = dict(case=case, x=(_randn((T, N), g) * 0.3).bfloat16(), weight=(1 + 0.2 * _randn((N,), g)).bfloat16())
        if case["residual"]:
            s["residual"] = (_randn((T, N), g) * wide * torch.exp(0.5 * _randn((T, 1), g))).bfloat16()
        return s
    if case["kind"] == "linear":
        T, K, O = case["T"], case["K"], case["O"]
        w = _randn((O, K), g) * K ** -0.5
        ws = w.abs().amax(-1) / 127
        x = _randn((T, K), g) * torch.exp(0.5 * _randn((T, 1), g))
        xs = x.abs().amax(-1) / 127
        return dict(case=case, codes=(w / ws[:, None]).round().to(torch.int8), scales=ws,
                    x=(x / xs[:, None]).round().to(torch.int8), x_scales=xs)
    return _prepare_cache(case, g)


def _lengths(c):
    """New tokens and whole length of each request, by the case alone: a decode or verify batch has ragged pasts (some of
    them near nothing), a prefill ragged prompts behind ragged cached context."""
    if c["R"] == 1:
        return [c["new"]], [c["past"] + c["new"]]
    rng = random.Random("%d %d %d" % (c["R"], c["new"], c["past"]))
    new = [1 if c["new"] == 1 else rng.randint(1, c["new"]) if c["new"] <= 8 else round(c["new"] * rng.uniform(0.5, 1.5))
           for _ in range(c["R"])]
    return new, [n + round(c["past"] * rng.random()) for n in new]


def _starts(counts):
    qsl = torch.zeros(len(counts) + 1, dtype=torch.int32)
    qsl[1:] = counts.cumsum(0)
    return qsl


def _prepare_cache(c, g):
    R, Hq, Hkv, D, page = c["R"], c["Hq"], c["Hkv"], c["D"], c["page"]
    new, seq = (torch.tensor(v, dtype=torch.int32) for v in _lengths(c))
    qsl = _starts(new)
    T = int(qsl[-1])
    need = (seq.long() + page - 1) // page
    width = int(need.max())
    pages = int(need.sum()) + 3
    where = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.zeros((R, width), dtype=torch.int32, device=DEV)
    live = torch.arange(width)[None, :] < need[:, None]
    table[live.to(DEV)] = where[:int(need.sum())]
    s = dict(case=c, T=T, most_new=int(new.max()), most_seq=int(seq.max()), qsl=qsl.to(DEV), seq=seq.to(DEV), table=table,
             unused=where[-1].long())
    for name in ("k", "v"):
        shape = (D // 16, BLOCK, 16) if name == "k" else (D, BLOCK)
        s[name + "_codes"] = torch.empty((pages, Hkv, page // BLOCK, *shape), dtype=torch.uint8, device=DEV)
        s[name + "_scales"] = torch.empty((pages, Hkv, page // BLOCK), device=DEV)
        step = max(1, (1 << 26) // (Hkv * page * D))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            # tokens of different size, so that a block's scale is that of its largest
            x = _randn((n, Hkv, page // BLOCK, BLOCK, D), g) * torch.exp(0.5 * _randn((n, Hkv, page // BLOCK, BLOCK, 1), g))
            scale = _block_scale(x.abs().amax((-2, -1)))
            codes = _e4m3(x / scale[..., None, None])
            s[name + "_codes"][p:p + n] = _laid_out(codes, name)
            s[name + "_scales"][p:p + n] = scale
    # what no token has been written to yet holds anything, codes that are no number and such scales among it
    filled = s["seq"] - (new.to(DEV) if c["kind"] == "append" else 0)
    t = torch.arange(width * page, device=DEV)
    r, j = torch.nonzero((t[None, :] >= filled[:, None]) & (t[None, :] < need.to(DEV)[:, None] * page), as_tuple=True)
    at, i = table[r, j // page].long(), j % page
    for name in ("k", "v"):
        s[name + "_codes"][at, :, i // BLOCK, :, i % BLOCK] = 0x7F
    first = i % BLOCK == 0
    for name in ("k", "v"):
        s[name + "_scales"][at[first], :, i[first] // BLOCK] = torch.nan
    if c["kind"] == "attention":
        s["q"] = (_randn((T, Hq, D), g) * 1.5).bfloat16()
        return s
    # the rows of one fused projection, as its user slices them
    s["qkv"] = (_randn((T, (Hq + 2 * Hkv) * D), g) * torch.exp(0.5 * _randn((T, 1), g))).bfloat16()
    s["inv_freq"] = (1e4 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device=DEV) / c["rot"])).float()
    # reading back takes the whole blocks that were written to: their earlier tokens may have changed with the scale
    touched = new + (seq - new) % BLOCK
    s["back_qsl"], s["back_T"] = _starts(touched).to(DEV), int(touched.sum())
    return s


# ---- one pass ----

def run(s):
    kind = s["case"]["kind"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "append": _own_append, "attention": _own_attention}[kind](s)
    return {"norm": _plain_norm, "linear": _plain_linear, "append": _plain_append, "attention": _plain_attention}[kind](s)


def _own_norm(s):
    import layer_embedding_lookup_amd as ple
    codes, scales, h = ple.ple_rms_norm8(s["x"], s["weight"], residual=s.get("residual"), eps=EPS)
    values = codes * scales[:, None]  # the codes as the values they stand for
    return values if h is None else (values, h)


def _own_linear(s):
    import layer_embedding_lookup_amd as ple
    w = s.get("handle")
    if w is None:  # the descriptor of the weights, which a program keeps beside them
        w = s["handle"] = ple.W8Weight(s["codes"], s["scales"])
    return ple.ple_w8_linear(s["x"], s["x_scales"], w)


def _own_cache(s):
    import layer_embedding_lookup_amd as ple
    cache = s.get("handle")
    if cache is None:  # the cache object that a program keeps
        cache = s["handle"] = ple.KV8Cache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    return ple, cache


def _split(s):
    c = s["case"]
    a, b = c["Hq"] * c["D"], (c["Hq"] + c["Hkv"]) * c["D"]
    x = s["qkv"]
    return [v.unflatten(-1, (-1, c["D"])) for v in (x[:, :a], x[:, a:b], x[:, b:])]


def _own_append(s):
    ple, cache = _own_cache(s)
    q, k, v = _split(s)
    q = ple.ple_kv8_append(cache, k, v, s["qsl"], s["seq"], s["table"], inv_freq=s["inv_freq"],
                           interleaved=s["case"]["interleaved"], q=q, max_request_tokens=s["most_new"])
    return (q, *ple.ple_kv8_read(cache, s["back_qsl"], s["seq"], s["table"], s["back_T"]))


def _own_attention(s):
    ple, cache = _own_cache(s)
    return ple.ple_kv8_attention(s["q"], cache, s["qsl"], s["seq"], s["table"], window=s["case"]["window"],
                                 max_request_tokens=s["most_new"], max_seq_len=s["most_seq"], want_lse=True)


def _plain_norm(s):
    h = s["x"]
    if "residual" in s:
        h = (h.float() + s["residual"].float()).bfloat16()
    x = h.float()
    t = x * s["weight"].float()
    top = t.abs().amax(-1, keepdim=True)
    scale = top * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) / 127
    values = torch.where(top > 0, (t * 127 / top).round(), 0.0) * scale
    return (values, h) if "residual" in s else values


def _plain_linear(s):
    acc = s["x"].float() @ s["codes"].float().t()
    return (acc * s["x_scales"][:, None] * s["scales"]).bfloat16()


def _places(s, qsl, T):
    """Request and position of each token of a batch."""
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(qsl[1:].contiguous(), t, right=True)
    return r, s["seq"][r].long() - (qsl[r + 1].long() - t)


def _rotate(x, pos, s):
    """The rotation of x [T][H][D] in 64 bits."""
    rot, half = s["case"]["rot"], s["case"]["rot"] // 2
    x = x.double()
    angle = (pos.double()[:, None] * s["inv_freq"].double()[None, :])[:, None, :]
    cos, sin = angle.cos(), angle.sin()
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_append(s):
    c = s["case"]
    R, H, D, page = c["R"], c["Hkv"], c["D"], c["page"]
    q, k, v = _split(s)
    r, pos = _places(s, s["qsl"], s["T"])
    q, k = _rotate(q, pos, s).float().bfloat16(), _rotate(k, pos, s).float()
    # the blocks that each request writes to, one after the other
    most = (s["most_new"] + BLOCK - 2) // BLOCK + 1
    begin = s["seq"].long() - (s["qsl"][1:] - s["qsl"][:-1]).long()
    block = (begin // BLOCK)[:, None] + torch.arange(most, device=DEV)
    live = block * BLOCK < s["seq"][:, None]
    first = (block * BLOCK).clamp(max=s["table"].shape[1] * page - 1)
    at = torch.where(live, s["table"].gather(1, first // page).long(), s["unused"]).flatten()  # (a page of no request)
    group = (first % page // BLOCK).flatten()
    kept = (begin[:, None] - block * BLOCK).clamp(0, BLOCK).flatten()         # earlier tokens of the block
    keep = (torch.arange(BLOCK, device=DEV) < kept[:, None])[:, None, :, None]
    mine = r * most + pos // BLOCK - begin[r] // BLOCK
    page_of, place = s["table"][r, pos // page].long(), pos % page
    for name, x in (("k", k), ("v", v.float())):
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        top = torch.zeros((R * most, H), device=DEV).scatter_reduce_(0, mine[:, None].expand(-1, H), x.abs().amax(-1), "amax")
        old = torch.where(kept[:, None] > 0, scales[at, :, group], 0.0)
        scale = torch.maximum(_block_scale(top), old)
        by = (old / scale)[:, :, None, None]
        held = _in_order(codes[at, :, group], name)                           # [blocks][H][16][D]
        codes[at, :, group] = _laid_out(torch.where(keep, _e4m3(_value(held) * by), held), name)
        scales[at, :, group] = scale
        new = _e4m3(x / scale[mine][..., None])
        codes[page_of, :, place // BLOCK, :, place % BLOCK] = new.unflatten(-1, (-1, 16)) if name == "k" else new
    r, pos = _places(s, s["back_qsl"], s["back_T"])
    page_of, place = s["table"][r, pos // page].long(), pos % page
    k, v = (_value(_tokens(s, n, page_of, place)) * s[n + "_scales"][page_of, :, place // BLOCK][..., None] for n in ("k", "v"))
    return q, k.bfloat16(), v.bfloat16()


def _rows(s, name):
    """Keys or values of every request in order, [R][Hkv][width * page][D], and whether a token stands there, [R][width * page]."""
    table = s["table"].long()
    x = _value(_in_order(s[name + "_codes"][table], name)).flatten(3, 4)          # [R][width][Hkv][page][D]
    x = x * s[name + "_scales"][table].repeat_interleave(BLOCK, -1)[..., None]
    x = x.transpose(1, 2).flatten(2, 3)
    live = torch.arange(x.shape[2], device=DEV)[None, :] < s["seq"][:, None]
    return torch.where(live[:, None, :, None], x, 0.0), live


def _plain_attention(s):
    c = s["case"]
    Hq, Hkv, D, G, R, most = c["Hq"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"], c["R"], s["most_new"]
    r, pos = _places(s, s["qsl"], s["T"])
    i = torch.arange(s["T"], device=DEV) - s["qsl"][r].long()
    q = torch.zeros((R, most, Hq, D), device=DEV)
    q[r, i] = s["q"].float() * D ** -0.5
    q = q.view(R, most, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(R, Hkv, G * most, D)
    k, live = _rows(s, "k")
    score = torch.matmul(q, k.transpose(-1, -2)).view(R, Hkv, G, most, -1)
    del k
    p = torch.full((R, most), -1, device=DEV)
    p[r, i] = pos
    j = torch.arange(live.shape[1], device=DEV)
    seen = live[:, None, :] & (j <= p[..., None])
    if c["window"]:
        seen &= j > p[..., None] - c["window"]
    score = score.masked_fill_(~seen[:, None, None], -torch.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    v, _ = _rows(s, "v")
    out = torch.matmul(score.view(R, Hkv, G * most, -1), v).view(R, Hkv, G, most, D)
    out = torch.where(total > 0, out / total, 0.0).permute(0, 3, 1, 2, 4).reshape(R, most, Hq, D)
    lse = (total.log() + top).squeeze(-1).permute(0, 3, 1, 2).reshape(R, most, Hq)
    return out[r, i].bfloat16(), lse[r, i]


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "linear": _exact_linear, "append": _exact_append, "attention": _exact_attention}[case["kind"]](s)


def _exact_norm(s):
    h = s["x"].double()
    if "residual" in s:
        # the residual stream is held in bf16, and what it holds is what is normalised
        h = (h + s["residual"].double()).bfloat16().double()
    t = h * s["weight"].double()
    size = torch.linalg.vector_norm(h, dim=-1, keepdim=True) / math.sqrt(h.shape[-1])
    top = t.abs().amax(-1, keepdim=True)
    step = torch.where(top > 0, top, 1.0) / 127
    values = torch.round(t / step) * step / torch.sqrt(size * size + EPS)
    return (values, h) if "residual" in s else values


def _exact_linear(s):
    return (s["x"].double() * s["x_scales"].double()[:, None]) @ (s["codes"].double() * s["scales"].double()[:, None]).t()


def _code_value(b):
    """An e4m3fn code's value from its fields (sign, four exponent bits with bias 7, three mantissa bits; 0x7F is no number)."""
    n = b.double()
    sign, e, m = torch.where(n >= 128, -1.0, 1.0).double(), (n % 128 / 8).floor(), n % 8
    v = sign * torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, e - 7))
    return torch.where(n % 128 == 127, torch.nan, v)


def _nearest(x):
    """The nearest e4m3fn value of x in 64 bits: three bits after the leading one, steps of 2^-9 below 2^-6."""
    _, e = torch.frexp(x)
    step = torch.pow(2.0, (e - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(s):
    """Each head of each token for itself: rotated as complex numbers, then block by block of each request."""
    c = s["case"]
    H, D, page = c["Hkv"], c["D"], c["page"]
    q, k, v = (x.double() for x in _split(s))
    r, pos = _places(s, s["qsl"], s["T"])
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[:, None] * s["inv_freq"].double())[:, None]
    rot, half = c["rot"], c["rot"] // 2

    def turned(x):
        x = x.clone()
        if c["interleaved"]:
            z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * turn
            x[..., 0:rot:2], x[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :half], x[..., half:rot]) * turn
            x[..., :half], x[..., half:rot] = z.real, z.imag
        return x

    got = []
    for name, x in (("k", turned(k)), ("v", v)):
        outs = []
        for i in range(c["R"]):
            a, b, n = int(s["qsl"][i]), int(s["qsl"][i + 1]), int(s["seq"][i])
            lo = (n - (b - a)) // BLOCK * BLOCK
            blocks = (n - lo + BLOCK - 1) // BLOCK
            kept = n - (b - a) - lo
            rows = torch.zeros((blocks * BLOCK, H, D), dtype=torch.float64, device=DEV)
            rows[kept:n - lo] = x[a:b]
            need = rows.view(blocks, BLOCK, H, D).abs().amax((1, 3))
            scale = torch.where(need > 0, torch.pow(2.0, torch.ceil(torch.log2(need / 448))), LEAST).clamp(LEAST, MOST)
            if kept:
                p, g = int(s["table"][i, lo // page]), lo % page // BLOCK
                old = s[name + "_scales"][p, :, g].double()
                codes = s["k_codes"][p, :, g, :, :kept].transpose(1, 2).flatten(2) if name == "k" else \
                    s["v_codes"][p, :, g, :, :kept].transpose(1, 2)
                scale[0] = torch.maximum(scale[0], old)
                rows[:kept] = (_code_value(codes) * old[:, None, None]).transpose(0, 1)
            scale = scale.repeat_interleave(BLOCK, 0)[..., None]
            outs.append((_nearest(rows / scale) * scale)[:n - lo])
        got.append(torch.cat(outs))
    return turned(q), *got


def _exact_attention(s):
    c = s["case"]
    D, G, Hkv, page = c["D"], c["Hq"] // c["Hkv"], c["Hkv"], c["page"]
    outs, lses = [], []
    for r in range(c["R"]):
        a, b, n = int(s["qsl"][r]), int(s["qsl"][r + 1]), int(s["seq"][r])
        at = s["table"][r, torch.arange(n, device=DEV) // page].long()
        i = torch.arange(n, device=DEV) % page
        k = _code_value(s["k_codes"][at, :, i // BLOCK, :, i % BLOCK].flatten(2)) * s["k_scales"][at, :, i // BLOCK].double()[..., None]
        v = _code_value(s["v_codes"][at, :, i // BLOCK, :, i % BLOCK]) * s["v_scales"][at, :, i // BLOCK].double()[..., None]
        k, v = (x.transpose(0, 1).contiguous() for x in (k, v))
        q = s["q"][a:b].double().view(b - a, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * (b - a), D)
        score = torch.bmm(q, k.transpose(1, 2).contiguous()).view(Hkv, G, b - a, n) / math.sqrt(D)
        p, j = torch.arange(n - (b - a), n, device=DEV)[:, None], torch.arange(n, device=DEV)[None, :]
        hidden = (j > p) | (j <= p - c["window"]) if c["window"] else j > p
        score.masked_fill_(hidden, -torch.inf)
        lses.append(torch.logsumexp(score, -1).permute(2, 0, 1).reshape(b - a, -1))
        weight = torch.softmax(score, -1).view(Hkv, G * (b - a), n)
        outs.append(torch.bmm(weight, v).view(Hkv, G, b - a, D).permute(2, 0, 1, 3).reshape(b - a, -1, D))
    return torch.cat(outs), torch.cat(lses)


# ---- what a pass cannot do without ----

def work(case):
    c = case
    if c["kind"] == "norm":
        T, N = c["T"], c["N"]
        # the rows in (and the residual in and out), the weight, the values of the codes out
        return {"bytes": T * N * (10 if c["residual"] else 6) + 2 * N, "flops": 6 * T * N}
    if c["kind"] == "linear":
        T, K, O = c["T"], c["K"], c["O"]
        return {"bytes": (T + O) * (K + 4) + 2 * T * O, "flops": 2 * T * K * O}
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    news, lengths = _lengths(c)
    T, token = sum(news), 2 * Hkv * D  # new tokens; a token's keys and values in the cache, and a block's scales
    block = 2 * Hkv * 4
    if c["kind"] == "append":
        # q, k and v in; q out; the cache's new rows and scales out; the written blocks read back as bf16
        back = sum(n + (m - n) % BLOCK for n, m in zip(news, lengths))
        blocks = sum((m - 1) // BLOCK - (m - n) // BLOCK + 1 for n, m in zip(news, lengths))
        return {"bytes": 2 * T * (2 * Hq + 2 * Hkv) * D + T * token + blocks * block + back * (token + 4 * Hkv * D),
                "flops": 6 * T * (Hq + Hkv) * c["rot"] // 2}
    read = pairs = 0
    for n, m in zip(news, lengths):
        w = c["window"] or m
        read += min(m, w + n - 1)
        pairs += sum(min(p + 1, w) for p in range(m - n, m))
    return {"bytes": read * token + read // BLOCK * block + 4 * T * Hq * D + 4 * T * Hq, "flops": 4 * Hq * D * pairs}
