"""Cases, plain forms and 64-bit values of the paged 8-bit KV cache and the rotation of positions.

Four operators: the rotation of queries and keys by their positions in any ring
layout, and its gradient (rope); storing new tokens, rotated on the way, in a
paged cache (kv8_append), and reading them back (kv8_read); attention of the
newest tokens, one or a whole chunk of a prompt, to that cache (attn_kv8).

A row of the table holds cos and sin of a position times each frequency, in
fp32. A pair (a, b) of channels becomes (a c - b s, b c + a s), both products
and their sum rounded to fp32; the pairs are (i, i + R/2) or, interleaved,
(2i, 2i+1) of the first R channels.

The cache is E4M3 codes [pages, Hkv, page size, D] and, for every 32 tokens of
a head, a power of two as its exponent, int8 [pages, Hkv, page size / 32]: the
smallest e >= -40 with max|x| <= 448 * 2^e over the block, at most 40, never
falling while the block has rows. A code is x / 2^e to the nearest, ties to
even. When an append raises a block's exponent, its older codes are rounded
once more. page_table [B, pages of a sequence] says where a sequence's rows are.

Sequence lengths follow from the case alone, so that work() knows them.
"""
import numpy as np
import torch

own = False

BLOCK = 32
DEV = "cuda"
F32, F64 = torch.float32, torch.float64


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step's new token of eight sequences: latency
        dict(name="append_step_b8", op="append", B=8, T=1, C=4096, page=64, Hq=32, Hkv=8, D=128,
             R=128, inter=False, dtype="bf16", packed=False, zero=False),
        # a prompt of the ring sweep's 32K tokens going into an empty cache
        dict(name="append_prompt_s32k", op="append", B=1, T=32768, C=32768, page=64, Hq=32,
             Hkv=8, D=128, R=128, inter=False, dtype="bf16", packed=False, zero=True),
        # a packed batch of prompts of odd lengths, fp32, half of the channels
        # rotated, in neighbouring pairs, behind what the cache already holds
        dict(name="append_packed_fp32", op="append", B=5, T=2501, C=4096, page=32, Hq=8, Hkv=4,
             D=64, R=32, inter=True, dtype="fp32", packed=True, zero=False),
        # one sequence of about a thousand tokens: latency
        dict(name="decode_latency", op="attn", B=1, T=1, C=1024, page=64, Hq=32, Hkv=8, D=128,
             causal=True, window=0, sink=0, ragged=True, zero=False, packed=False),
        # the decoding benchmark's batch: eight sequences of 128K tokens
        dict(name="decode_b8_s128k", op="attn", B=8, T=1, C=131072, page=64, Hq=32, Hkv=8,
             D=128, causal=True, window=0, sink=0, ragged=False, zero=False, packed=False),
        # sliding window with attention sinks, 32 KV heads, a ragged batch
        dict(name="decode_window_ragged", op="attn", B=16, T=1, C=8192, page=32, Hq=32, Hkv=32,
             D=128, causal=True, window=1000, sink=4, ragged=True, zero=False, packed=False),
        # three tokens at a time (speculative decoding), a ragged batch
        dict(name="decode_spec_ragged", op="attn", B=4, T=3, C=32768, page=128, Hq=32, Hkv=8,
             D=128, causal=True, window=0, sink=0, ragged=True, zero=False, packed=False),
        # the last chunk of 512 tokens of a 32K prompt
        dict(name="chunk_512_s32k", op="attn", B=1, T=512, C=32768, page=64, Hq=32, Hkv=8,
             D=128, causal=True, window=0, sink=0, ragged=False, zero=False, packed=False),
        # chunks of odd lengths and single tokens in one packed batch (a serving
        # step that mixes prompts and decoding)
        dict(name="chunk_packed_mixed", op="attn", B=7, T=1111, C=10016, page=32, Hq=32, Hkv=8,
             D=128, causal=True, window=0, sink=0, ragged=True, zero=False, packed=True),
        # a chunk of 4K tokens in the middle of a longer prompt
        dict(name="chunk_4k_s16k", op="attn", B=1, T=4096, C=16384, page=128, Hq=32, Hkv=8,
             D=128, causal=True, window=0, sink=0, ragged=False, zero=False, packed=False),
        # queries of the sliding-window training shape, a zigzag ring of 8
        dict(name="rope_zigzag_s8k", op="rope", B=2, S=8192, H=32, D=128, R=128, inter=False,
             inverse=False, dtype="bf16", cp=8, layout="zigzag", packed=0),
        # gradients of a packed batch's keys, odd lengths, fp32
        dict(name="rope_grad_packed_fp32", op="rope", B=1, S=5003, H=8, D=64, R=32, inter=True,
             inverse=True, dtype="fp32", cp=1, layout="contiguous", packed=4),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "chunk", "chunk", "rope"])
    D = rng.choice([64, 128, 128])
    page = rng.choice([32, 64, 128])
    Hkv = rng.choice([1, 2, 3, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
    R, inter = rng.choice([16, 32, D, D, D]), rng.random() < 0.3
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "append":
        B = rng.randint(1, 9)
        T = _log(rng, 1, 16384 // B)
        return dict(op=op, B=B, T=T, C=-(-(T + 600) // page) * page, page=page, Hq=Hq, Hkv=Hkv,
                    D=D, R=R, inter=inter, dtype=dtype, packed=rng.random() < 0.4,
                    zero=rng.random() < 0.3)
    if op == "rope":
        cp = rng.choice([1, 1, 2, 4])
        S = _log(rng, 8, 16384)
        if cp > 1:
            S = max(1, S // (2 * cp)) * 2 * cp
        packed = rng.choice([0, 0, 3, 7]) if S >= 16 else 0
        c = dict(op=op, B=1 if packed else rng.randint(1, 3), S=S, H=Hq, D=D, R=R, inter=inter,
                 inverse=rng.random() < 0.5, dtype=dtype, cp=cp,
                 layout=rng.choice(["contiguous", "zigzag", "stripe"]), packed=packed)
        if c["layout"] == "zigzag":  # two chunks per rank
            c["S"] -= S % (2 * cp)
        return c
    window = rng.choice([0, 0, _log(rng, 1, 4000)])
    sink = rng.choice([0, 1, 4]) if window else 0
    if op == "decode":
        B = rng.randint(1, 12)
        C = -(-_log(rng, 32, 400000 // B) // page) * page
        T, packed = rng.choice([1, 1, 1, 2, 3, 5]), False
    else:
        B = rng.randint(1, 5)
        T = _log(rng, 6, 2000 // B)
        packed = rng.random() < 0.5
        C = -(-max(_log(rng, 64, 24000 // B), T * (B if packed else 1)) // page) * page
    return dict(op="attn", B=B, T=T, C=C, page=page, Hq=Hq, Hkv=Hkv, D=D,
                causal=rng.random() < 0.8, window=window, sink=sink, ragged=rng.random() < 0.7,
                zero=rng.random() < 0.3, packed=packed)


def _lens(c):
    """Cached lengths of the B sequences: the capacity each, or spread below it;
    at least the new tokens where there are many (zero: none in the first)."""
    B, top = c["B"], c["C"]
    out = [top] * B
    if c["ragged"]:
        out = [max(1, min(top, top * (2 * ((5 * b + 3) % B) + 2) // (2 * B) - b)) for b in range(B)]
    if c["T"] > 8:
        out = [max(L, n) for L, n in zip(out, _new(c))]
    if c["zero"] and B > 1:
        out[0] = 0
    return out


def _spans(total, n):
    """Boundaries of n packed sequences of different odd lengths."""
    cut = [0]
    for i in range(1, n):
        cut.append(max(cut[-1], min(total, total * i * (i + 1) // (n * (n + 1)) + i % 3)))
    return cut + [total]


def _cuts(c):
    """Boundaries of a packed batch of new tokens: the first sequences bring one
    token each, the others chunks."""
    if c["op"] == "append":
        cut = [0]
        for e in _spans(c["B"] * c["T"], c["B"])[1:]:
            cut.append(min(e, cut[-1] + c["C"] - 600))  # no more than there is room for
        return cut
    B, T = c["B"], c["T"]
    single = min(B // 2, T)
    return list(range(single)) + [single + x for x in _spans(T - single, B - single)]


def _new(c):
    """New tokens of each sequence."""
    if c["packed"]:
        cut = _cuts(c)
        return [b - a for a, b in zip(cut, cut[1:])]
    return [c["T"]] * c["B"]


# -------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _keys(shape, g, dtype):
    """Keys and values as a model has them: some channels much larger."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=F32)
    gain = torch.ones(shape[-1], device=DEV)
    gain[1::17] = 4.0
    gain[3::29] = 0.1
    return (x * gain).to(dtype)


def _pages(c):
    """(pages of a sequence, pages in all)."""
    mp = c["C"] // c["page"]
    return mp, c["B"] * mp + 3


def _cache_bytes(c, seed):
    """Codes and exponents of random keys and values; some blocks of tokens much
    larger than others. A few pages at a time, which bounds the memory."""
    g = _gen(seed)
    H, D, page = c["Hkv"], c["D"], c["page"]
    n, nb = _pages(c)[1], c["page"] // BLOCK
    out = [torch.empty((n, H, page, D), dtype=torch.uint8, device=DEV),
           torch.empty((n, H, nb), dtype=torch.int8, device=DEV)]
    out += [torch.empty_like(t) for t in out]
    at = max(1, 1 << 27 >> (H * page * D).bit_length())
    for p in range(0, n, at):
        m = min(at, n - p)
        for i in (0, 2):
            x = _keys((m, H, nb, BLOCK, D), g, F32)
            x = x * torch.exp2(torch.randint(-2, 2, (m, H, nb, 1, 1), generator=g, device=DEV).to(F32))
            e = _exponent(x.abs().amax((-1, -2)))
            out[i][p:p + m] = _codes(x, e[..., None, None]).view(torch.uint8).view(m, H, page, D)
            out[i + 1][p:p + m] = e.to(torch.int8)
    return out


def _table(positions, R):
    """cos and sin of every position and frequency, fp32 [positions, R]."""
    f = 10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=F64) / R)
    a = torch.arange(positions, device=DEV, dtype=F64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], -1).to(F32)


def _positions(S, cp, layout):
    """Natural position of each rank-major position."""
    p = torch.arange(S, device=DEV)
    if layout == "stripe":
        return p.reshape(S // cp, cp).t().reshape(-1)
    if layout == "zigzag":
        ch = p.reshape(2 * cp, -1)
        return torch.cat([torch.cat([ch[r], ch[2 * cp - 1 - r]]) for r in range(cp)])
    return p


def prepare(case, seed):
    c = case
    st = dict(c=c)
    g = _gen(seed)
    dt = F32 if c.get("dtype") == "fp32" else torch.bfloat16
    if c["op"] == "rope":
        shape = (c["S"], c["H"], c["D"]) if c["packed"] else (c["B"], c["S"], c["H"], c["D"])
        st["x"] = _keys(shape, g, dt)
        st["table"] = _table(c["S"], c["R"])
        st["cu"] = None
        if c["packed"]:
            st["cu"] = torch.tensor(_spans(c["S"], c["packed"]), dtype=torch.int32, device=DEV)
        return st
    B, C, H, D = c["B"], c["C"], c["Hkv"], c["D"]
    st["bytes"] = _cache_bytes(c, seed + 1)
    mp, n = _pages(c)
    st["pages"] = torch.randperm(n, generator=g, device=DEV)[: B * mp].to(torch.int32).view(B, mp)
    new = _new(c)
    lead = (sum(new),) if c["packed"] else (B, c["T"])
    st["cu"], st["most"] = None, max(new)
    if c["packed"]:
        st["cu"] = torch.tensor(_cuts(c), dtype=torch.int32, device=DEV)
    st["q"] = torch.randn(lead + (c["Hq"], D), generator=g, device=DEV).to(dt)
    if c["op"] == "attn":
        st["lens"] = torch.tensor(_lens(c), dtype=torch.int32, device=DEV)
        return st
    st["k"], st["v"] = _keys(lead + (H, D), g, dt), _keys(lead + (H, D), g, dt) * 0.5
    room = C - max(new)
    at = [0 if c["zero"] and b == 0 else min(room, 100 + 77 * b % 450) for b in range(B)]
    st["starts"] = torch.tensor(at, dtype=torch.int32, device=DEV)
    # the rows to read back: from the first block that the new tokens touch
    st["first"] = torch.tensor([a // BLOCK * BLOCK for a in at], dtype=torch.int32, device=DEV)
    st["lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    st["table"] = _table(C, c["R"])
    return st


# ---------------------------------------------------------------- plain forms

def _exponent(amax):
    """Smallest e >= -40 with amax <= 448 * 2^e, at most 40."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875)
    return torch.where(amax > 0, e, -40).clamp(-40, 40)


def _codes(x, e):
    return (x * torch.exp2(-e.to(F32))).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _rotated(x, cs, c, inverse=False):
    """fp32: x [..., heads, D] rotated by cs [..., R] (cos, sin) of its tokens."""
    x, R = x.to(F32), c["R"]
    cos, sin = cs[..., None, : R // 2], cs[..., None, R // 2:]
    if inverse:
        sin = -sin
    y = x.clone()
    if c["inter"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        y[..., : R // 2], y[..., R // 2: R] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rope(st):
    c, x = st["c"], st["x"]
    pos = _positions(c["S"], c["cp"], c["layout"])
    if st["cu"] is not None:
        pos = pos - st["cu"][torch.searchsorted(st["cu"], pos.to(torch.int32), right=True) - 1]
    return dict(y=_rotated(x, st["table"][pos], c, c["inverse"]).to(x.dtype))


def _padded(st, t):
    """[B, most, ...] of the new tokens, and which of them there are."""
    n = torch.arange(st["most"], device=DEV)
    if st["cu"] is None:
        return t, torch.ones(t.shape[:2], dtype=torch.bool, device=DEV)
    cu = st["cu"].long()
    at = (cu[:-1, None] + n).clamp(max=max(0, t.shape[0] - 1))
    return t[at], n < (cu[1:] - cu[:-1])[:, None]


def _packed(st, t):
    """The tokens that there are of [B, most, ...]."""
    if st["cu"] is None:
        return t
    n = torch.arange(st["most"], device=DEV)
    return t[n < (st["cu"][1:] - st["cu"][:-1])[:, None]]


def _rows(st, t):
    """[B, Hkv, C, ...] of an array by pages."""
    t = t[st["pages"].long()].transpose(1, 2)
    return t.flatten(2, 3)


def _plain_append(st):
    c = st["c"]
    B, H, D, most = c["B"], c["Hkv"], c["D"], st["most"]
    start, first = st["starts"].long()[:, None], st["first"].long()[:, None]
    nblk = -(-(most + BLOCK) // BLOCK)
    row = first + torch.arange(nblk * BLOCK, device=DEV)  # the touched blocks' rows
    r = row.clamp(max=c["C"] - 1)
    page = st["pages"].gather(1, r // c["page"]).long()
    out = []
    for i, t in enumerate((st["k"], st["v"])):
        x, there = _padded(st, t)
        cs = st["table"][(start + torch.arange(most, device=DEV)).clamp(max=c["C"] - 1)]
        x = _rotated(x, cs, c) if i == 0 else x.to(F32)
        # new rows where they go; elsewhere 0
        at = row - start
        isnew = (at >= 0) & (at < there.sum(1, keepdim=True))
        x = x[torch.arange(B, device=DEV)[:, None], at.clamp(0, most - 1)]
        x = torch.where(isnew[..., None, None], x, 0.0).view(B, nblk, BLOCK, H, D)
        isold = (at < 0)[..., None, None].view(B, nblk, BLOCK, 1, 1)
        # what the blocks held
        code = st["bytes"][2 * i][page, :, r % c["page"]]
        code = code.view(torch.float8_e4m3fn).to(F32).view(B, nblk, BLOCK, H, D)
        old = st["bytes"][2 * i + 1][page, :, r % c["page"] // BLOCK]
        old = old.view(B, nblk, BLOCK, H)[:, :, 0].to(torch.int32)
        e = _exponent(x.abs().amax((2, 4)))
        e = torch.where(isold.any(2)[..., 0], torch.maximum(e, old), e)[:, :, None, :, None]
        old = old[:, :, None, :, None]
        code = (code * torch.exp2((old - e).to(F32))).to(torch.float8_e4m3fn).to(F32)
        code = torch.where(isold, code, _codes(x, e).to(F32))
        val = (code * torch.exp2(e.to(F32))).flatten(1, 2)
        val = torch.where((isnew | (at < 0))[..., None, None], val, 0.0)
        out.append(val[:, : most + BLOCK - 1].to(t.dtype))
    lens = st["starts"] + (c["T"] if st["cu"] is None else st["cu"][1:] - st["cu"][:-1])
    x, _ = _padded(st, st["q"])
    q = _packed(st, _rotated(x, cs, c)).to(st["q"].dtype)
    return dict(k=out[0], v=out[1], q=q, lens=lens.to(torch.int32))


def _seen(st):
    """[B, most, C]: cached key j is visible to new token t."""
    c = st["c"]
    j = torch.arange(c["C"], device=DEV)[None, None, :]
    L = st["lens"].long()[:, None, None]
    n = c["T"] if st["cu"] is None else (st["cu"][1:] - st["cu"][:-1]).long()[:, None, None]
    i = L - n + torch.arange(st["most"], device=DEV)[None, :, None]
    v = (j < L) & (i >= 0)
    if c["causal"]:
        v = v & (j <= i)
    if c["window"]:
        v = v & ((i - j < c["window"]) | (j < c["sink"]))
    return v


def _plain_attn(st):
    c = st["c"]
    B, Hq, H, D, C = c["B"], c["Hq"], c["Hkv"], c["D"], c["C"]
    G, N = Hq // H, st["most"]
    kc, ke, vc, ve = st["bytes"]
    k, v = (_rows(st, code).view(torch.float8_e4m3fn).to(F32) *
            torch.exp2(_rows(st, e).to(F32)).repeat_interleave(BLOCK, -1)[..., None]
            for code, e in ((kc, ke), (vc, ve)))
    q, _ = _padded(st, st["q"])
    q = q.to(F32).view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    s = (q @ k.transpose(-1, -2)).view(B, H, G, N, C) * (1.0 / D ** 0.5)
    s = s.masked_fill(~_seen(st)[:, None, None], -torch.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, H, G * N, C) @ v).view(B, H, G, N, D) / torch.where(l > 0, l, 1.0)
    lse = m + torch.log(l)
    o, lse = (_packed(st, t.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, -1)) for t in (o, lse))
    return dict(out=o.to(torch.bfloat16), lse=lse.squeeze(-1).contiguous())


# -------------------------------------------------- the framework's operators

def _own(st):
    import sequence_long_context_gb300 as usp

    c = st["c"]
    if c["op"] == "rope":
        return dict(y=usp.rope(st["x"], st["table"], interleaved=c["inter"], inverse=c["inverse"],
                               cu_seqlens=st["cu"], cp=c["cp"], layout=c["layout"]))
    kc, ke, vc, ve = st["bytes"]
    if c["op"] == "append":
        cache = usp.KV8Cache(kc, ke, vc, ve, st["pages"], st["starts"])
        lens, q = usp.kv8_append(cache, st["k"], st["v"], q=st["q"], rope=st["table"],
                                 interleaved=c["inter"], cu_seqlens=st["cu"],
                                 seq_lens_out=st["lens"])
        k, v = usp.kv8_read(cache._replace(seq_lens=lens), st["most"] + BLOCK - 1,
                            starts=st["first"], dtype=st["k"].dtype)
        return dict(k=k, v=v, q=q, lens=lens)
    cache = usp.KV8Cache(kc, ke, vc, ve, st["pages"], st["lens"])
    out, lse = usp.attn_kv8(st["q"], cache, causal=c["causal"], window=c["window"],
                            sink_tokens=c["sink"], cu_seqlens=st["cu"], max_new=st["most"])
    return dict(out=out, lse=lse)


def run(state):
    if own:
        return _own(state)
    return dict(append=_plain_append, attn=_plain_attn, rope=_plain_rope)[state["c"]["op"]](state)


# ----------------------------------------------------------------------- work

def work(case):
    c = case
    D = c["D"]
    el = 4 if c.get("dtype") == "fp32" else 2
    if c["op"] == "rope":
        n = c["B"] * c["S"]
        return dict(bytes=2 * n * c["H"] * D * el + 4 * c["S"] * c["R"], flops=3 * n * c["H"] * c["R"])
    H, Hq = c["Hkv"], c["Hq"]
    row = 2 * D + 2 / BLOCK  # a token's keys and values of one head in the cache
    if c["op"] == "append":
        n = sum(_new(c))
        # k, v and q in, the cache written and read, the values and q out
        return dict(bytes=n * H * (4 * D * el + 2 * row) + 2 * n * Hq * D * el + 4 * n * c["R"] + 8 * c["B"],
                    flops=n * (H * 4 * D + 3 * (H + Hq) * c["R"]))
    keys = pairs = 0
    for L, n in zip(_lens(c), _new(c)):
        i = np.arange(max(0, L - n), L)
        hi = i + 1 if c["causal"] else np.full_like(i, L)
        lo = np.maximum(0, i - c["window"] + 1) if c["window"] else np.zeros_like(i)
        sunk = np.minimum(lo, c["sink"])
        pairs += int((np.maximum(0, hi - lo) + sunk).sum())
        if len(i):
            keys += int(hi[-1] - lo[0] + sunk[0])
    rows = sum(_new(c)) * Hq
    return dict(bytes=keys * H * row + rows * (4 * D + 4), flops=4 * D * pairs * Hq)


# ---------------------------------------------------- the definition, 64 bits

def _e4m3_round(x):
    """x to the nearest e4m3 number, ties to the even one, at most 448."""
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return torch.round(a / step) * step * torch.sign(x)


def _e4m3_table():
    b = torch.arange(256, device=DEV)
    e, m = (b >> 3) & 15, (b & 7).to(F64)
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.to(F64) - 7), m / 8 * 2.0 ** -6)
    v[127] = v[255] = torch.nan
    return torch.where(b > 127, -v, v)


def _exact_turn(x, pos, st, sign=1.0, rounded=False):
    """x [n, heads, D] at positions pos; the table's fp32 numbers are an input."""
    c = st["c"]
    R = c["R"]
    j = torch.arange(R // 2, device=DEV)
    ia, ib = (2 * j, 2 * j + 1) if c["inter"] else (j, j + R // 2)
    turn = torch.index_select(st["table"], 0, pos).to(F64)
    co, si = turn[:, None, j], sign * turn[:, None, R // 2 + j]
    rnd = (lambda t: t.to(F32).to(F64)) if rounded else (lambda t: t)
    y = x.to(F64)
    a, b = y[..., ia], y[..., ib]
    y = y.clone()
    y[..., ia] = rnd(rnd(a * co) - rnd(b * si))
    y[..., ib] = rnd(rnd(b * co) + rnd(a * si))
    return y


def _exact_rope(st):
    c, x = st["c"], st["x"]
    pos = torch.empty(c["S"], dtype=torch.long, device=DEV)
    if c["layout"] == "zigzag":
        n = c["S"] // (2 * c["cp"])
        chunks = [k for r in range(c["cp"]) for k in (r, 2 * c["cp"] - 1 - r)]
        for at, k in enumerate(chunks):
            pos[at * n:(at + 1) * n] = torch.arange(k * n, (k + 1) * n, device=DEV)
    elif c["layout"] == "stripe":
        n = c["S"] // c["cp"]
        for r in range(c["cp"]):
            pos[r * n:(r + 1) * n] = torch.arange(r, c["S"], c["cp"], device=DEV)
    else:
        pos = torch.arange(c["S"], device=DEV)
    if c["packed"]:
        own_pos = torch.empty_like(pos)
        cut = _spans(c["S"], c["packed"])
        for a, e in zip(cut, cut[1:]):
            inside = (pos >= a) & (pos < e)
            own_pos[inside] = pos[inside] - a
        pos = own_pos
    sign = -1.0 if c["inverse"] else 1.0
    if c["packed"]:
        return dict(y=_exact_turn(x, pos, st, sign))
    return dict(y=torch.stack([_exact_turn(t, pos, st, sign) for t in x]))


def _exact_append(st):
    c = st["c"]
    B, H, D, most = c["B"], c["Hkv"], c["D"], st["most"]
    cut, new = (_cuts(c) if c["packed"] else None), _new(c)
    part = lambda t, b: t[cut[b]:cut[b + 1]] if c["packed"] else t[b]  # noqa: E731
    starts = st["starts"].tolist()
    tab = _e4m3_table()
    out = [torch.zeros((B, most + BLOCK - 1, H, D), dtype=F64, device=DEV) for _ in range(2)]
    q = []
    for b in range(B):
        pos = (starts[b] + torch.arange(new[b], device=DEV)).clamp(max=c["C"] - 1)
        q.append(_exact_turn(part(st["q"], b), pos, st))
        base = starts[b] // BLOCK * BLOCK
        for i, name in enumerate("kv"):
            x = part(st[name], b)
            # the definition rounds a rotated key's products and sums to fp32
            x = _exact_turn(x, pos, st, rounded=True) if i == 0 else x.to(F64)
            have = starts[b] - base  # rows that the first block holds
            pg = int(st["pages"][b, base // c["page"]])
            at, blk = base % c["page"], base % c["page"] // BLOCK
            held = tab[st["bytes"][2 * i][pg, :, at:at + have].long()].transpose(0, 1)
            was = st["bytes"][2 * i + 1][pg, :, blk].to(F64)
            done = 0
            while done < new[b]:
                n = min(new[b] - done, BLOCK - have)
                y = x[done:done + n]
                top = y.abs().amax((0, 2))
                e = torch.ceil(torch.log2(torch.where(top > 0, top, 1.0) / 448.0))
                e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)
                e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e)
                e = torch.where(top > 0, e, -40.0).clamp(-40.0, 40.0)
                rows = torch.empty((0, H, D), dtype=F64, device=DEV)
                if have:
                    e = torch.maximum(e, was)
                    rows = _e4m3_round(held * torch.exp2(was - e)[:, None])
                s = torch.exp2(e)[:, None]
                rows = torch.cat([rows, _e4m3_round(y / s)]) * s
                first = starts[b] + done - have - base
                out[i][b, first:first + have + n] = rows
                done, have = done + n, 0
            if new[b] == 0 and have:
                out[i][b, :have] = held * torch.exp2(was)[:, None]
    return dict(k=out[0], v=out[1], q=torch.cat(q) if c["packed"] else torch.stack(q), lens=None)


def _exact_attn(st):
    c = st["c"]
    Hq, H, D = c["Hq"], c["Hkv"], c["D"]
    G, tab = Hq // H, _e4m3_table()
    new = _new(c)
    cut = _cuts(c) if c["packed"] else [c["T"] * b for b in range(c["B"] + 1)]
    q = st["q"].reshape(-1, Hq, D)
    out = torch.zeros((q.shape[0], Hq, D), dtype=F64, device=DEV)
    lse = torch.full((q.shape[0], Hq), -torch.inf, dtype=F64, device=DEV)
    for b, (L, n) in enumerate(zip(_lens(c), new)):
        used = -(-L // c["page"])
        pg = st["pages"][b, :used].long()
        if L == 0 or n == 0:
            continue
        for h in range(H):
            k, v = ((tab[st["bytes"][i][pg, h].long()].view(used, -1, BLOCK, D) *
                     torch.exp2(st["bytes"][i + 1][pg, h].to(F64))[..., None, None]).view(-1, D)[:L]
                    for i in (0, 2))
            j = torch.arange(L, device=DEV)
            for t0 in range(0, n, 512):
                t = torch.arange(t0, min(n, t0 + 512), device=DEV)
                gap = (L - n + t)[:, None] - j[None, :]
                hide = gap + j < 0
                if c["causal"]:
                    hide |= gap < 0
                if c["window"]:
                    hide |= (gap >= c["window"]) & (j >= c["sink"])[None, :]
                rows = q[cut[b] + t][:, h * G:(h + 1) * G].to(F64)
                s = torch.einsum("tgd,kd->tgk", rows, k) / D ** 0.5
                s = s.masked_fill(hide[:, None], -torch.inf)
                z = torch.logsumexp(s, -1)
                p = torch.nan_to_num(torch.exp(s - z[..., None]), nan=0.0)
                out[cut[b] + t, h * G:(h + 1) * G] = torch.einsum("tgk,kd->tgd", p, v)
                lse[cut[b] + t, h * G:(h + 1) * G] = z
    if not c["packed"]:
        out, lse = out.view(c["B"], c["T"], Hq, D), lse.view(c["B"], c["T"], Hq)
    return dict(out=out, lse=lse)


def exact(case, seed):
    st = prepare(case, seed)
    return dict(append=_exact_append, attn=_exact_attn, rope=_exact_rope)[case["op"]](st)
