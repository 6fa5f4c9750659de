"""Cases, plain forms and 64-bit values of the operators around the 4-bit KV cache.

Five operators: filling the cache (kv4_append) and reading it back
(kv4_read), one decoding step over it (attn_decode_kv4), the attention
weight of every key of a prompt (attn_key_weights) and eviction by that
weight (kv4_evict).

The cache holds 4-bit integers. A token's D channels of one KV head are cut
into blocks of 32; with y = x / descale (one multiplication by the fp32
reciprocal, rounded to fp32), a block has the scale s = e4m3(max|y| / 7),
rounded to nearest even and saturating, and the codes
c = clamp(round_half_even(y / s), -7, 7), 0 where s = 0. It stands for
c * s * descale. A code is stored as the nibble c + 8, channel 2i in the low
nibble of byte i. Arrays: codes [B, Hkv, C, D/2], scales [B, Hkv, C, D/32].

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
        dict(name="append_step_b8", op="append", B=8, T=1, C=4096, Hkv=8, D=128,
             dtype="bf16", packed=False, descale=1.0, zero=False),
        # a prompt of the ring sweep's 32K tokens going into an empty cache
        dict(name="append_prompt_s32k", op="append", B=1, T=32768, C=32768, Hkv=8, D=128,
             dtype="bf16", packed=False, descale=1.0, zero=True),
        # a packed batch of prompts of odd lengths, fp32 keys and values
        dict(name="append_packed_fp32", op="append", B=5, T=2501, C=4096, Hkv=4, D=64,
             dtype="fp32", packed=True, descale=0.37, zero=False),
        # one sequence of about a thousand tokens: latency
        dict(name="decode_latency", op="decode", B=1, Tq=1, C=1024, Hq=32, Hkv=8, D=128,
             causal=True, window=0, sink=0, ragged=True, zero=False, weights=False,
             descale=1.0),
        # the decoding benchmark's batch: eight sequences of 128K tokens
        dict(name="decode_b8_s128k", op="decode", B=8, Tq=1, C=131072, Hq=32, Hkv=8, D=128,
             causal=True, window=0, sink=0, ragged=False, zero=False, weights=False,
             descale=1.0),
        # sliding window with attention sinks, 32 KV heads, a ragged batch
        dict(name="decode_window_ragged", op="decode", B=16, Tq=1, C=8192, Hq=32, Hkv=32, D=128,
             causal=True, window=1000, sink=4, ragged=True, zero=False, weights=False,
             descale=0.5),
        # three tokens at a time (speculative decoding), a ragged batch, the keys'
        # attention weights accumulated for a later eviction
        dict(name="decode_spec_weights", op="decode", B=4, Tq=3, C=32768, Hq=32, Hkv=8, D=128,
             causal=True, window=0, sink=0, ragged=True, zero=False, weights=True,
             descale=1.0),
        # weights of a prompt's keys over all its queries, zigzag ring of 8
        dict(name="weights_zigzag_s8k", op="weights", B=1, S=8192, Hq=32, Hkv=8, D=128,
             causal=True, window=0, sink=0, cp=8, layout="zigzag", observe=0, packed=0,
             dtype="bf16"),
        # weights of a long prompt's keys over its last 64 queries
        dict(name="weights_last64_s32k", op="weights", B=1, S=32768, Hq=32, Hkv=8, D=128,
             causal=True, window=0, sink=0, cp=1, layout="contiguous", observe=64, packed=0,
             dtype="bf16"),
        # a packed batch of prompts, odd lengths, one query head per KV head
        dict(name="weights_packed_odd", op="weights", B=1, S=5003, Hq=8, Hkv=8, D=64,
             causal=True, window=0, sink=0, cp=1, layout="contiguous", observe=0, packed=4,
             dtype="bf16"),
        # a serving batch that has outgrown its budget by 64 tokens
        dict(name="evict_step_b8", op="evict", B=8, C=1104, Hkv=8, D=128, keep=1024,
             recent=64, sink=4, ragged=False, zero=False, ties=False),
        # eight prompts of 128K tokens brought down to 8K keys each
        dict(name="evict_prompt_s128k", op="evict", B=8, C=131072, Hkv=8, D=128, keep=8192,
             recent=1024, sink=4, ragged=True, zero=False, ties=False),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "weights", "evict"])
    D = rng.choice([64, 128])
    if op == "append":
        packed = rng.random() < 0.4
        B = rng.randint(1, 9)
        T = _log(rng, 1, 16384 // B)
        return dict(op=op, B=B, T=T, C=-(-(T + 600) // 16) * 16, Hkv=rng.choice([1, 2, 3, 8]), D=D,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), packed=packed,
                    descale=rng.choice([1.0, 0.25, 0.37, 2.0]), zero=rng.random() < 0.3)
    if op == "decode":
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        B = rng.randint(1, 12)
        C = -(-_log(rng, 16, 400000 // B) // 16) * 16
        window = rng.choice([0, 0, _log(rng, 1, 4000)])
        return dict(op=op, B=B, Tq=rng.choice([1, 1, 1, 2, 3, 5]), C=C, Hq=Hq, Hkv=Hkv, D=D,
                    causal=rng.random() < 0.8, window=window,
                    sink=rng.choice([0, 1, 4]) if window else 0, ragged=rng.random() < 0.7,
                    zero=rng.random() < 0.3, weights=rng.random() < 0.5,
                    descale=rng.choice([1.0, 0.5, 0.37]))
    if op == "weights":
        Hkv = rng.choice([1, 2, 4])
        cp = rng.choice([1, 1, 2, 4])
        layout = rng.choice(["contiguous", "zigzag", "stripe"])
        S = _log(rng, 8, 6000)
        packed = rng.choice([0, 0, 3, 7]) if S >= 16 else 0
        if cp > 1:
            S = max(1, S // (2 * cp)) * 2 * cp
        window = rng.choice([0, 0, _log(rng, 8, 2000)])
        return dict(op=op, B=1 if packed else rng.randint(1, 3), S=S, Hq=Hkv * rng.choice([1, 2, 4]),
                    Hkv=Hkv, D=D, causal=rng.random() < 0.8, window=window,
                    sink=rng.choice([0, 4]) if window else 0, cp=cp,
                    layout=layout if cp > 1 else "contiguous",
                    observe=rng.choice([0, 0, 1, _log(rng, 1, 300)]), packed=packed, dtype="bf16")
    B = rng.randint(1, 8)
    C = -(-_log(rng, 32, 200000 // B) // 16) * 16
    keep = _log(rng, 8, C)
    sink = rng.choice([0, 0, 4])
    return dict(op=op, B=B, C=C, Hkv=rng.choice([1, 2, 8]), D=D, keep=keep,
                recent=rng.randint(0, keep - sink), sink=sink, ragged=rng.random() < 0.6,
                zero=rng.random() < 0.2, ties=rng.random() < 0.4)


def _lens(c, top):
    """Cached lengths of the B sequences: `top` each, or spread below it."""
    B = c["B"]
    out = [top] * B
    if c.get("ragged"):
        out = [max(1, min(top, top * (2 * ((5 * b + 3) % B) + 2) // (2 * B) - b)) for b in range(B)]
    if c.get("zero") and B > 1:
        out[0] = 0
    return out


def _spans(total, n):
    """Boundaries of n packed sequences of different odd lengths."""
    cut = [0]
    for i in range(1, n):
        cut.append(max(cut[-1], min(total, total * i * (i + 1) // (n * (n + 1)) + i % 3)))
    return cut + [total]


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


def _quantize(x, descale):
    """(codes, scales) of [..., D] values: the cache's bytes."""
    c, s = _quantized(x, descale)
    u = (c + 8).to(torch.uint8).flatten(-2)
    return u[..., 0::2] | (u[..., 1::2] << 4), s.to(torch.float8_e4m3fn).view(torch.uint8)


def _cache_bytes(c, seed):
    """codes and scales [B, Hkv, C, ..] of random keys and values; one
    sequence at a time, which bounds the memory it takes."""
    g = _gen(seed)
    B, C, H, D = c["B"], c["C"], c["Hkv"], c["D"]
    out = [torch.empty((B, H, C, n), dtype=torch.uint8, device=DEV)
           for n in (D // 2, D // BLOCK, D // 2, D // BLOCK)]
    for b in range(B):
        for i in (0, 2):
            out[i][b], out[i + 1][b] = _quantize(_keys((H, C, D), g, F32), c.get("descale", 1.0))
    return out


def _positions(S, cp, layout):
    """Natural position of each rank-major position."""
    p = torch.arange(S, device=DEV)
    if layout == "stripe":
        return p.reshape(S // cp, cp).t().reshape(-1)
    if layout == "zigzag":
        ch = p.reshape(2 * cp, -1)
        return torch.cat([torch.cat([ch[r], ch[2 * cp - 1 - r]]) for r in range(cp)])
    return p


def _case_lse(c, q, k, vis_rows, dtype=F64):
    """Log-sum-exp of the observed queries (0 where nothing reads it), a head at
    a time and in blocks of queries."""
    B, S, Hq, D = q.shape
    G = Hq // c["Hkv"]
    lse = torch.zeros((B, Hq, S), dtype=F32, device=DEV)
    pos, seg = vis_rows
    rows = torch.nonzero(_observed(c, pos, seg)).flatten()
    for r in rows.split(1024):
        m = _visible(c, pos, seg, r)
        for b in range(B):
            for h in range(Hq):
                s = q[b, r, h].to(dtype) @ k[b, :, h // G].to(dtype).t() / D ** 0.5
                lse[b, h, r] = torch.logsumexp(s.masked_fill(~m, -torch.inf), -1).to(F32)
    return lse


def _segments(c):
    """(natural position, (first, end) of the own sequence) of each
    rank-major position of a prompt batch."""
    S = c["S"]
    pos = _positions(S, c["cp"], c["layout"])
    cut = torch.tensor(_spans(S, c["packed"]) if c["packed"] else [0, S], device=DEV)
    n = torch.searchsorted(cut, pos, right=True) - 1
    return pos, (cut[n], cut[n + 1])


def _observed(c, pos, seg):
    return pos >= seg[1] - c["observe"] if c["observe"] else torch.ones_like(pos, dtype=torch.bool)


def _visible(c, pos, seg, rows):
    """[rows, S]: key j is visible to query i."""
    i, j, first = pos[rows, None], pos[None, :], seg[0]
    v = first[rows, None] == first[None, :]
    if c["causal"]:
        v = v & (j <= i)
    if c["window"]:
        v = v & ((i - j < c["window"]) | (j - first[None, :] < c["sink"]))
    return v


def prepare(case, seed):
    c = case
    st = dict(c=c)
    if c["op"] == "append":
        g = _gen(seed)
        B, C, H, D, T = c["B"], c["C"], c["Hkv"], c["D"], c["T"]
        dt = torch.bfloat16 if c["dtype"] == "bf16" else F32
        shape = (B * T, H, D) if c["packed"] else (B, T, H, D)
        st["k"], st["v"] = _keys(shape, g, dt), _keys(shape, g, dt) * 0.5
        at = [0 if c["zero"] and b == 0 else min(C - T, 100 + 77 * b % 450) for b in range(B)]
        if C == T:
            at = [0] * B
        st["starts"] = torch.tensor(at, dtype=torch.int32, device=DEV)
        st["lens"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        if c["packed"]:
            cut = [min(C - 600, b) for b in _spans(B * T, B)]
            # no sequence longer than the room that is left in the cache
            for b in range(B):
                cut[b + 1] = min(_spans(B * T, B)[b + 1], cut[b] + C - 600)
            st["cut"] = cut
            st["k"], st["v"] = st["k"][: cut[-1]].contiguous(), st["v"][: cut[-1]].contiguous()
            st["cu"] = torch.tensor(cut, dtype=torch.int32, device=DEV)
            st["tokens"] = max(b - a for a, b in zip(cut, cut[1:]))
        else:
            st["cu"], st["tokens"] = None, T
        st["bytes"] = [torch.zeros((B, H, C, n), dtype=torch.uint8, device=DEV)
                       for n in (D // 2, D // BLOCK, D // 2, D // BLOCK)]
    elif c["op"] == "decode":
        st["bytes"] = _cache_bytes(c, seed)
        g = _gen(seed + 1)
        st["q"] = torch.randn((c["B"], c["Tq"], c["Hq"], c["D"]), generator=g, device=DEV).to(torch.bfloat16)
        st["lens"] = torch.tensor(_lens(c, c["C"]), dtype=torch.int32, device=DEV)
        st["weight"] = None
        if c["weights"]:
            st["weight"] = torch.rand((c["B"], c["Hkv"], c["C"]), generator=g, device=DEV) * 0.01
    elif c["op"] == "weights":
        g = _gen(seed)
        q = torch.randn((c["B"], c["S"], c["Hq"], c["D"]), generator=g, device=DEV).to(torch.bfloat16)
        k = _keys((c["B"], c["S"], c["Hkv"], c["D"]), g, torch.bfloat16)
        k = (k * 0.7).to(torch.bfloat16)
        st["place"] = _segments(c)
        st["lse"] = _case_lse(c, q, k, st["place"], F32 if c["S"] > 2000 else F64)
        st["q"], st["k"], st["cu"] = q, k, None
        if c["packed"]:
            st["q"], st["k"], st["lse"] = q[0], k[0], st["lse"][0]
            st["cu"] = torch.tensor(_spans(c["S"], c["packed"]), dtype=torch.int32, device=DEV)
    else:
        st["bytes"] = _cache_bytes(c, seed)
        g = _gen(seed + 1)
        # a few keys take most of the attention
        w = torch.rand((c["B"], c["Hkv"], c["C"]), generator=g, device=DEV)
        w = w ** 4 * 3.0
        st["weight"] = (w * 16).round() / 16 if c["ties"] else w
        st["lens"] = torch.tensor(_lens(c, c["C"]), dtype=torch.int32, device=DEV)
        Cd = -(-c["keep"] // 16) * 16
        st["dst"] = [torch.zeros(t.shape[:2] + (Cd,) + t.shape[3:], dtype=t.dtype, device=DEV)
                     for t in st["bytes"] + [st["weight"]]]
        st["dst_lens"] = torch.zeros(c["B"], dtype=torch.int32, device=DEV)
    if c["op"] in ("decode", "evict"):
        st["cache"] = tuple(st["bytes"])
    return st


# ---------------------------------------------------------------- plain forms

def _quantized(x, descale):
    """(integer codes as fp32 [..., n, 32], scales as fp32 [..., n])."""
    y = x.to(F32) * torch.tensor(1.0 / np.float32(descale), dtype=F32, device=x.device)
    y = y.unflatten(-1, (-1, BLOCK))
    # a tensor as the divisor: a scalar one becomes a product with its reciprocal
    seven = torch.full((), 7.0, dtype=F32, device=x.device)
    s = (y.abs().amax(-1) / seven).clamp(max=448.0).to(torch.float8_e4m3fn).to(F32)
    q = y / torch.where(s > 0, s, 1.0)[..., None]
    return torch.where(s[..., None] > 0, q.round().clamp(-7, 7), 0.0), s


def _values(codes, scales, descale):
    """fp32 values [..., D] of the cache's bytes."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(F32) - 8
    s = scales.view(torch.float8_e4m3fn).to(F32)
    return (c.unflatten(-1, (-1, BLOCK)) * s[..., None]).flatten(-2) * descale


def _seen(c, L):
    """[B, Tq, C]: cached key j is visible to new token t."""
    j = torch.arange(c["C"], device=DEV)[None, None, :]
    L = L.long()[:, None, None]
    i = L - c["Tq"] + torch.arange(c["Tq"], device=DEV)[None, :, None]
    v = (j < L) & (i >= 0)
    if c["causal"]:
        v = v & (j <= i)
    if c["window"]:
        v = v & ((i - j < c["window"]) | (j < c["sink"]))
    return v


def _plain_append(st):
    c = st["c"]
    B, H, D, n = c["B"], c["Hkv"], c["D"], st["tokens"]
    if st["cu"] is not None:
        count = st["cu"][1:] - st["cu"][:-1]
        at = (st["cu"][:-1, None] + torch.arange(n, device=DEV)).clamp(max=max(0, st["k"].shape[0] - 1))
        there = torch.arange(n, device=DEV) < count[:, None]
        rows = [t[at.long()] for t in (st["k"], st["v"])]
    else:
        count = torch.full((B,), n, device=DEV, dtype=torch.int32)
        there = torch.ones((B, n), dtype=torch.bool, device=DEV)
        rows = [st["k"], st["v"]]
    out = []
    for x in rows:
        q, s = _quantized(x, c["descale"])
        val = (q * s[..., None]).flatten(-2) * c["descale"]
        out.append(torch.where(there[..., None, None], val, 0.0).to(x.dtype))
    return dict(k=out[0], v=out[1], lens=st["starts"] + count.to(torch.int32))


def _plain_decode(st):
    c = st["c"]
    B, Tq, Hq, H, D = c["B"], c["Tq"], c["Hq"], c["Hkv"], c["D"]
    kc, ks, vc, vs = st["cache"]
    k, v = _values(kc, ks, c["descale"]), _values(vc, vs, c["descale"])
    q = st["q"].to(F32).reshape(B, Tq, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    s = (q @ k.transpose(-1, -2)) * (1.0 / D ** 0.5)
    vis = _seen(c, st["lens"])[:, None, None].expand(B, H, Hq // H, Tq, c["C"]).reshape(B, H, -1, c["C"])
    s = s.masked_fill(~vis, -torch.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, 1.0)
    o = p @ v
    lse = (m + torch.log(l)).squeeze(-1)
    back = lambda t: t.reshape((B, H, Hq // H, Tq) + t.shape[3:]).permute(  # noqa: E731
        *([0, 3, 1, 2] + list(range(4, t.dim() + 1)))).reshape((B, Tq, Hq) + t.shape[3:])
    out = dict(out=back(o).to(torch.bfloat16), lse=back(lse).contiguous())
    if c["weights"]:
        st["weight"] += p.sum(2)
        out["weight"] = st["weight"]
    return out


def _plain_weights(st):
    c = st["c"]
    q, k, lse = st["q"], st["k"], st["lse"]
    if c["packed"]:
        q, k, lse = q[None], k[None], lse[None]
    B, S, Hq, D = q.shape
    H = c["Hkv"]
    rows = torch.nonzero(_observed(c, *st["place"])).flatten()
    qh = q[:, rows].to(F32).permute(0, 2, 1, 3).reshape(B, H, -1, D)
    s = (qh @ k.to(F32).permute(0, 2, 3, 1)) * (1.0 / D ** 0.5)
    s = s.reshape(B, H, Hq // H, len(rows), S) - lse[:, :, rows].reshape(B, H, Hq // H, -1, 1)
    p = torch.where(_visible(c, *st["place"], rows), torch.exp(s), 0.0)
    w = p.sum((2, 3))
    return dict(weight=w[0] if c["packed"] else w)


def _plain_evict(st):
    c = st["c"]
    L = st["lens"].long()[:, None, None]
    j = torch.arange(c["C"], device=DEV)[None, None, :]
    w = st["weight"]
    w = torch.where((j < c["sink"]) | (j >= L - c["recent"]), torch.inf, w)
    w = torch.where(j < L, w, -torch.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., : c["keep"]]
    n = L.clamp(max=c["keep"])
    t = torch.arange(c["keep"], device=DEV)
    order = torch.where(t < n, order, c["C"]).sort(-1).values
    there = t < n
    kept = torch.where(there, order, -1).to(torch.int32)
    out = []
    for src, dst in zip(st["bytes"] + [st["weight"]], st["dst"]):
        at = order.clamp(max=c["C"] - 1)
        keep = there
        if src.dim() == 4:
            at, keep = at[..., None].expand(*at.shape, src.shape[-1]), keep[..., None]
        dst[:, :, : c["keep"]] = torch.where(keep, src.gather(2, at), dst[:, :, : c["keep"]])
        out.append(dst)
    return dict(kept=kept, k=out[0], k_scale=out[1], v=out[2], v_scale=out[3], weight=out[4],
                lens=n.reshape(-1).to(torch.int32))


# -------------------------------------------------- the framework's operators

def _own(st):
    import sequence_long_context_gb300 as usp

    c = st["c"]
    if c["op"] == "append":
        cache = usp.KV4Cache(*st["bytes"], seq_lens=st["starts"], key_weight=None,
                             k_descale=c["descale"], v_descale=c["descale"])
        lens = usp.kv4_append(cache, st["k"], st["v"], cu_seqlens=st["cu"], seq_lens_out=st["lens"])
        k, v = usp.kv4_read(cache._replace(seq_lens=lens), st["tokens"], starts=st["starts"],
                            dtype=st["k"].dtype)
        return dict(k=k, v=v, lens=lens)
    if c["op"] == "decode":
        cache = usp.KV4Cache(*st["bytes"], seq_lens=st["lens"], key_weight=st["weight"],
                             k_descale=c["descale"], v_descale=c["descale"])
        out, lse = usp.attn_decode_kv4(st["q"], cache, causal=c["causal"], window=c["window"],
                                       sink_tokens=c["sink"], accumulate=c["weights"])
        r = dict(out=out, lse=lse)
        if c["weights"]:
            r["weight"] = st["weight"]
        return r
    if c["op"] == "weights":
        return dict(weight=usp.attn_key_weights(
            st["q"], st["k"], st["lse"], causal=c["causal"], window=c["window"],
            sink_tokens=c["sink"], cu_seqlens=st["cu"], cp=c["cp"], layout=c["layout"],
            observe=c["observe"]))
    src = usp.KV4Cache(*st["bytes"], seq_lens=st["lens"], key_weight=st["weight"],
                       k_descale=1.0, v_descale=1.0)
    dst = usp.KV4Cache(*st["dst"][:4], seq_lens=st["dst_lens"], key_weight=st["dst"][4],
                       k_descale=1.0, v_descale=1.0)
    dst, kept = usp.kv4_evict(src, c["keep"], recent=c["recent"], sink_tokens=c["sink"], out=dst)
    # the moved codes and scales are bytes copied as they are
    return dict(kept=kept, k=dst.k, k_scale=dst.k_scale, v=dst.v, v_scale=dst.v_scale,
                weight=dst.key_weight, lens=dst.seq_lens)


def run(state):
    if own:
        return _own(state)
    return dict(append=_plain_append, decode=_plain_decode, weights=_plain_weights,
                evict=_plain_evict)[state["c"]["op"]](state)


# ----------------------------------------------------------------------- work

def _pairs(c):
    """Visible (observed query, key) pairs of one head, and observed queries."""
    cut = _spans(c["S"], c["packed"]) if c["packed"] else [0, c["S"]]
    pairs = rows = 0
    for a, e in zip(cut, cut[1:]):
        n = e - a
        i = np.arange(max(0, n - c["observe"]) if c["observe"] else 0, n)
        hi = i + 1 if c["causal"] else np.full_like(i, n)
        seen = hi
        if c["window"]:
            lo = np.maximum(0, i - c["window"] + 1)
            seen = hi - lo + np.minimum(lo, c["sink"])
        pairs += int(seen.sum())
        rows += len(i)
    return pairs, rows


def work(case):
    c = case
    D, H = c["D"], c["Hkv"]
    row = D + 2 * D // BLOCK  # a token's keys and values of one head in the cache
    if c["op"] == "append":
        el = 2 if c["dtype"] == "bf16" else 4
        n = c["B"] * c["T"]
        if c["packed"]:
            cut = [0]
            for e in _spans(n, c["B"])[1:]:
                cut.append(min(e, cut[-1] + c["C"] - 600))
            n = cut[-1]
        # k and v in, the cache written and read, the values out
        return dict(bytes=n * H * (2 * D * el * 2 + 2 * row) + 8 * c["B"], flops=n * H * 2 * D * 4)
    if c["op"] == "decode":
        keys = 0
        pairs = 0
        for L in _lens(c, c["C"]):
            i = np.arange(max(0, L - c["Tq"]), L)
            hi = i + 1 if c["causal"] else np.full_like(i, L)
            lo = np.maximum(0, i - c["window"] + 1) if c["window"] else np.zeros_like(i)
            sunk = np.minimum(lo, c["sink"])
            pairs += int((np.maximum(0, hi - lo) + sunk).sum())
            if len(i):
                keys += int(hi[-1] - lo[0] + sunk[0])
        rows = c["B"] * c["Tq"] * c["Hq"]
        return dict(bytes=keys * H * (row + (8 if c["weights"] else 0)) + rows * (4 * D + 4),
                    flops=4 * D * pairs * c["Hq"])
    if c["op"] == "weights":
        pairs, rows = _pairs(c)
        return dict(bytes=c["B"] * (c["S"] * H * (2 * D + 4) + rows * c["Hq"] * (2 * D + 4)),
                    flops=2 * D * pairs * c["Hq"] * c["B"])
    lens = _lens(c, c["C"])
    kept = sum(min(L, c["keep"]) for L in lens)
    return dict(bytes=H * (4 * sum(lens) + kept * (2 * (row + 4) + 4)), flops=H * sum(lens))


# ---------------------------------------------------- the definition, 64 bits

def _e4m3_round(x):
    """x >= 0 to the nearest e4m3 number, ties to the even one, at most 448."""
    x = x.clamp(max=448.0)
    e = torch.floor(torch.log2(torch.where(x > 0, x, 1.0))).clamp(min=-6.0)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def _e4m3_table():
    b = torch.arange(256, device=DEV)
    e, m = (b >> 3) & 15, (b & 7).to(F64)
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.to(F64) - 7), m / 8 * 2.0 ** -6)
    v[127] = v[255] = torch.nan
    return torch.where(b > 127, -v, v)


def _exact_values(codes, scales, descale):
    B, H, C, half = codes.shape
    out = torch.empty((B, H, C, 2 * half), dtype=F64, device=DEV)
    out[..., 0::2] = (codes % 16).to(F64) - 8
    out[..., 1::2] = (codes // 16).to(F64) - 8
    s = _e4m3_table()[scales.long()] * float(np.float32(descale))
    return out * s.repeat_interleave(BLOCK, dim=-1)


def _exact_append(st):
    c = st["c"]
    n, B = st["tokens"], c["B"]
    inv = float(np.float32(1.0) / np.float32(c["descale"]))
    got = []
    for x in (st["k"], st["v"]):
        # the definition rounds the product with the reciprocal once, to fp32
        y = (x.to(F64) * inv).to(F32).to(F64).reshape(x.shape[:-1] + (-1, BLOCK))
        s = _e4m3_round(y.abs().max(dim=-1, keepdim=True).values / 7)
        code = torch.round(y / torch.where(s == 0, 1.0, s)).clamp(-7, 7) * (s != 0)
        val = (code * s).reshape(x.shape) * float(np.float32(c["descale"]))
        if st["cu"] is not None:
            full = torch.zeros((B, n) + tuple(val.shape[1:]), dtype=F64, device=DEV)
            for b in range(B):
                a, e = st["cut"][b], st["cut"][b + 1]
                full[b, : e - a] = val[a:e]
            val = full
        got.append(val)
    return dict(k=got[0], v=got[1], lens=None)


def _exact_decode(st):
    c = st["c"]
    kc, ks, vc, vs = st["cache"]
    B, Tq, Hq, H = c["B"], c["Tq"], c["Hq"], c["Hkv"]
    G, D = Hq // H, c["D"]
    out = torch.zeros((B, Tq, Hq, D), dtype=F64, device=DEV)
    lse = torch.full((B, Tq, Hq), -torch.inf, dtype=F64, device=DEV)
    weight = st["weight"].to(F64) if c["weights"] else None
    for b, L in enumerate(_lens(c, c["C"])):
        if L == 0:
            continue
        k = _exact_values(kc[b:b + 1, :, :L], ks[b:b + 1, :, :L], c["descale"])[0]
        v = _exact_values(vc[b:b + 1, :, :L], vs[b:b + 1, :, :L], c["descale"])[0]
        j = torch.arange(L, device=DEV)
        for t in range(Tq):
            i = L - Tq + t
            if i < 0:
                continue
            ok = torch.ones(L, dtype=torch.bool, device=DEV)
            if c["causal"]:
                ok &= j <= i
            if c["window"]:
                ok &= (i - j < c["window"]) | (j < c["sink"])
            q = st["q"][b, t].to(F64).reshape(H, G, D)
            s = torch.einsum("hgd,hkd->hgk", q, k) / D ** 0.5
            s[..., ~ok] = -torch.inf
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[..., None])
            out[b, t] = torch.einsum("hgk,hkd->hgd", p, v).reshape(Hq, D)
            lse[b, t] = z.reshape(Hq)
            if weight is not None:
                weight[b, :, :L] += p.sum(1)
    r = dict(out=out, lse=lse)
    if weight is not None:
        r["weight"] = weight
    return r


def _exact_weights(st):
    c = st["c"]
    lead = c["packed"] > 0
    q, k, lse = (t[None] if lead else t for t in (st["q"], st["k"], st["lse"]))
    B, S, Hq, D = q.shape
    G = Hq // c["Hkv"]
    pos, (first, end) = st["place"]
    w = torch.zeros((B, c["Hkv"], S), dtype=F64, device=DEV)
    take = torch.arange(S, device=DEV)
    if c["observe"]:
        take = take[end - pos <= c["observe"]]
    for r in take.split(2048):
        gap = pos[r][:, None] - pos[None, :]
        hide = first[r][:, None] != first[None, :]
        if c["causal"]:
            hide |= gap < 0
        if c["window"]:
            hide |= (gap >= c["window"]) & (pos - first >= c["sink"])[None, :]
        for b in range(B):
            for h in range(Hq):
                s = torch.mm(q[b, r, h].to(F64), k[b, :, h // G].to(F64).t()) / D ** 0.5
                p = torch.exp(s - lse[b, h, r].to(F64)[:, None])
                w[b, h // G] += p.masked_fill(hide, 0.0).sum(0)
    return dict(weight=w[0] if lead else w)


def _exact_evict(st):
    # whole numbers, moved bytes and moved weights: only the weights are
    # floating, and they are the ones at the kept places
    c = st["c"]
    full = torch.zeros(st["dst"][4].shape, dtype=F64, device=DEV)
    for b, L in enumerate(_lens(c, c["C"])):
        w = st["weight"][b, :, :L].to(F64)
        if L > c["keep"]:
            rest = c["keep"] - c["sink"] - c["recent"]
            mid = w[:, c["sink"]: L - c["recent"]]
            # a place before counts first among equals
            rank = torch.argsort(-mid, dim=-1, stable=True)[:, :rest]
            at = torch.cat([torch.arange(c["sink"], device=DEV).expand(c["Hkv"], -1), rank + c["sink"],
                            torch.arange(L - c["recent"], L, device=DEV).expand(c["Hkv"], -1)], 1)
            w = torch.take_along_dim(w, at.sort(-1).values, 1)
        full[b, :, : w.shape[1]] = w
    return dict(kept=None, k=None, k_scale=None, v=None, v_scale=None, weight=full, lens=None)


def exact(case, seed):
    st = prepare(case, seed)
    return dict(append=_exact_append, decode=_exact_decode, weights=_exact_weights,
                evict=_exact_evict)[case["op"]](st)
