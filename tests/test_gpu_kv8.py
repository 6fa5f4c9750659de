"""GPU parity of the rotation of positions and the paged 8-bit KV cache against the
oracle.

Rotations, codes, exponents and lengths are compared exactly: products, sums and
roundings are those of the definition. Tolerances of the attention (bf16 output,
|ds| the error of a score, n keys, u = 2^-24):
  |ds| <= D u max_ij sum_d |q_d k_d| scale  (fp32 accumulation of exact products)
          + 2^-22 (1 + max|s|)  (scaling, maximum, exp2's argument and result)
  LSE:    |ds| + n u + 4 u |LSE|
  O:      A (2^-11 + 2 |ds| + 2 n u) + 2^-32 n V + 2^-8 |O|
          with A = sum_j P_j |v_j|: P is rounded to fp16 (2^-11), whose subnormal
          step (half of 2^-24) counts against a reference at least 2^7 below the
          largest contribution, each key's value at most V = 448 * 2^max(e_v);
          O is rounded to bf16"""
import numpy as np
import pytest
import torch

import sequence_long_context_gb300 as usp
from oracle import fp8, kv8, layouts
from tests._gpu import device

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------------- rope

ROPE = [
    # shape, dtype, R, interleaved, cp, layout
    ((1, 1, 1, 64), BF, 16, False, 1, "contiguous"),
    ((2, 5, 3, 64), F32, 64, True, 1, "contiguous"),
    ((2, 96, 32, 128), BF, 128, False, 4, "zigzag"),
    ((3, 48, 8, 128), F32, 128, False, 8, "stripe"),
    ((1, 333, 5, 128), BF, 96, True, 3, "contiguous"),
    ((1, 64, 1, 128), F32, 32, True, 2, "zigzag"),
    ((1, 1000, 33, 64), BF, 32, False, 1, "contiguous"),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("shape,dtype,R,inter,cp,layout", ROPE)
def test_rope_is_the_definition_bit_for_bit(shape, dtype, R, inter, cp, layout, inverse):
    dev = device()
    x = torch.randn(shape, generator=gen(R)).to(dtype)
    S = shape[1]
    table = usp.rope_table(S + 3, R, device=dev)
    pos = layouts.extract(np.arange(S), layout, cp, axis=0)
    want = np.stack([kv8.rotate(b.float().numpy(), pos, table.cpu().numpy(), inter, inverse) for b in x])
    want = torch.from_numpy(want).to(dtype)
    got = usp.rope(x.to(dev), table, interleaved=inter, inverse=inverse, cp=cp, layout=layout)
    assert torch.equal(got.cpu(), want)
    y = x.to(dev)
    assert usp.rope(y, table, interleaved=inter, inverse=inverse, cp=cp, layout=layout, out=y) is y
    assert torch.equal(y, got)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope_packed_restarts_and_leaves_padding(dtype):
    dev = device()
    cut = [3, 3, 40, 41, 90]
    x = torch.randn(96, 6, 64, generator=gen(1)).to(dtype)
    table = usp.rope_table(96, 64, device=dev)
    for layout, cp in (("contiguous", 1), ("zigzag", 4), ("stripe", 3)):
        pos = layouts.extract(np.arange(96), layout, cp, axis=0)
        want = x.clone()
        for a, e in zip(cut, cut[1:]):
            at = np.nonzero((pos >= a) & (pos < e))[0]
            want[at] = torch.from_numpy(kv8.rotate(x[at].float().numpy(), pos[at] - a,
                                                   table.cpu().numpy())).to(dtype)
        got = usp.rope(x.to(dev), table, cu_seqlens=i32(cut, dev), cp=cp, layout=layout)
        assert torch.equal(got.cpu(), want), layout


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient_is_the_inverse(inter):
    """<g, rope(x + h) - rope(x - h)> / 2 = <rope^-1(g), h>: the rotation is linear, so
    central differences have no error but rounding (2^-24 of each of 3 sums, twice)."""
    dev = device()
    B, S, H, D = 2, 24, 3, 64
    x, h, g = (torch.randn(B, S, H, D, generator=gen(s)).to(dev) for s in (1, 2, 3))
    table = usp.rope_table(S, 48, device=dev)
    kw = dict(interleaved=inter, cp=2, layout="zigzag")
    up, down = usp.rope(x + h, table, **kw), usp.rope(x - h, table, **kw)
    d = (g.double() * (up.double() - down.double())).sum() / 2
    back = (usp.rope(g, table, inverse=True, **kw).double() * h.double()).sum()
    tol = 8 * U * float((g.abs() * (x.abs() + h.abs())).double().sum()) * 2
    assert abs(float(d - back)) < tol


# ------------------------------------------------------------------ append, read

def shuffled_cache(dev, B, cap, H, D, page, seed=0, spare=3, fill=0xAB):
    """A cache whose sequences' pages lie in no order, every byte set."""
    c = usp.kv8_cache(B, cap, H, D, page_size=page, num_pages=B * -(-cap // page) + spare, device=dev)
    perm = torch.randperm(c.k.shape[0], generator=gen(seed))[: c.page_table.numel()]
    c.page_table.copy_(perm.to(torch.int32).view(c.page_table.shape))
    for t in (c.k, c.v):
        t.fill_(fill)
    for t in (c.k_exp, c.v_exp):
        t.fill_(17)
    return c


def host(c):
    return [t.cpu().numpy().copy() for t in c[:4]] + [c.page_table.cpu().numpy()]


APPEND = [
    # B, T, cap, H, Hq, D, page, dtype, R, interleaved, starts
    (1, 1, 64, 1, 1, 64, 32, BF, 64, False, [0]),
    (3, 1, 128, 2, 8, 128, 64, BF, 128, False, [0, 17, 127]),
    (4, 1, 256, 3, 3, 128, 128, F32, 32, True, [31, 32, 33, 256]),   # the last is full
    (2, 7, 64, 3, 6, 128, 32, F32, 128, False, [5, 60]),             # no room behind 64
    (4, 100, 256, 2, 4, 128, 64, BF, 64, True, [0, 3, 150, 255]),
    (2, 333, 384, 1, 5, 64, 128, BF, 16, False, [1, 50]),
    (1, 64, 128, 2, 2, 64, 32, F32, 64, False, [31]),                # one CTA group each ..
    (1, 65, 128, 2, 2, 64, 32, F32, 64, False, [31]),                # .. and blocks shared out
    (1, 65, 128, 5, 10, 128, 32, F32, 0, False, [-7]),               # a negative length counts as 0
    (9, 2, 32, 8, 8, 64, 32, BF, 0, False, list(range(24, 33))),
]


@pytest.mark.parametrize("B,T,cap,H,Hq,D,page,dtype,R,inter,starts", APPEND)
def test_append_stores_the_definitions_bytes(B, T, cap, H, Hq, D, page, dtype, R, inter, starts):
    dev = device()
    g = gen(T)
    k = (torch.randn(B, T, H, D, generator=g) * torch.logspace(-3, 2, D)).to(dtype)
    v = torch.randn(B, T, H, D, generator=g).to(dtype)
    q = torch.randn(B, T, Hq, D, generator=g).to(dtype)
    v[0, 0, 0, :8] = torch.tensor([float("nan"), float("inf"), -float("inf"), 0, -0.0, 1e-30, 7, 3.5])
    v[-1, -1, -1] = 0
    c = shuffled_cache(dev, B, cap, H, D, page)
    # rows that the blocks hold already: a first append of random ones
    have = [min(max(s, 0), cap) for s in starts]
    old = [torch.randn(B, cap, H, D, generator=g) * s for s in (3.0, 1e-3)]
    # (row by row where they end inside a block: any exponent may be there)
    want = host(c)
    for b in range(B):
        for i in (0, 1):
            kv8.append(want[2 * i], want[2 * i + 1], want[4][b], 0, old[i][b, : have[b]].numpy())
    for t, w in zip(c[:4], want):
        t.copy_(torch.from_numpy(w))
    c.seq_lens.copy_(torch.tensor(starts, dtype=torch.int32))
    table = usp.rope_table(c.page_table.shape[1] * page, R, device=dev) if R else None
    lens, qr = usp.kv8_append(c, k.to(dev), v.to(dev), q=q.to(dev), rope=table, interleaved=inter)
    cap = c.page_table.shape[1] * page
    assert lens is c.seq_lens and lens.tolist() == [min(cap, a + T) for a in have]
    for b in range(B):
        pos = have[b] + np.arange(T)
        kr, qw = k[b].float().numpy(), q[b].float().numpy()
        if R:
            tab = table.cpu().numpy()
            kr, qw = kv8.rotate(kr, pos, tab, inter), kv8.rotate(qw, pos, tab, inter)
        kv8.append(want[0], want[1], want[4][b], have[b], kr)
        kv8.append(want[2], want[3], want[4][b], have[b], v[b].float().numpy())
        assert torch.equal(qr[b].cpu(), torch.from_numpy(qw).to(dtype)), b
    for name, t, w in zip(c._fields, c[:4], want):
        assert np.array_equal(t.cpu().numpy(), w), name


@pytest.mark.parametrize("H,D,cut,pad", [(2, 128, [0, 5, 5, 70, 71], 0), (3, 64, [2, 2, 40, 300, 300], 7)])
@pytest.mark.parametrize("inplace", [False, True])
def test_append_packed_is_each_sequence_alone(H, D, cut, pad, inplace):
    dev = device()
    g = gen(9)
    B, T = len(cut) - 1, cut[-1] + pad
    k, v = (torch.randn(T, H, D, generator=g).to(BF).to(dev) for _ in "kv")
    q = torch.randn(T, 2 * H, D, generator=g).to(BF).to(dev)
    starts = i32([3, 0, 32, 9], dev)
    table = usp.rope_table(320, D, device=dev)
    a = shuffled_cache(dev, B, 320, H, D, 64)._replace(seq_lens=starts)
    b = shuffled_cache(dev, B, 320, H, D, 64)
    out = starts if inplace else torch.full((B,), -1, dtype=torch.int32, device=dev)
    want_lens = [s + cut[i + 1] - cut[i] for i, s in enumerate(starts.tolist())]
    first = starts.clone()
    q_out = torch.full_like(q, 5.0)
    got, qr = usp.kv8_append(a, k, v, q=q, q_out=q_out, rope=table, seq_lens_out=out,
                             cu_seqlens=i32(cut, dev))
    assert got is out and qr is q_out and out.tolist() == want_lens
    assert inplace or starts.tolist() == first.tolist()
    for i in range(B):
        s = slice(cut[i], cut[i + 1])
        one = b._replace(page_table=b.page_table[i:i + 1].contiguous(), seq_lens=first[i:i + 1].clone())
        _, q1 = usp.kv8_append(one, k[None, s].contiguous(), v[None, s].contiguous(),
                               q=q[None, s].contiguous(), rope=table)
        assert torch.equal(q1[0], q_out[s])
    for x, y in zip(a[:4], b[:4]):
        assert torch.equal(x, y)
    assert not q_out[: cut[0]].any() and not q_out[cut[-1]:].any()  # padding


def test_append_at_given_positions_and_in_place():
    dev = device()
    B, T, H, D = 2, 40, 2, 64
    g = gen(4)
    k, v = (torch.randn(B, T, H, D, generator=g).to(dev) for _ in "kv")
    q = torch.randn(B, T, 3, D, generator=g).to(dev)
    pos = torch.randint(-2, 60, (B, T), generator=g).to(torch.int32)  # 50 and up, and below 0: the nearest
    table = usp.rope_table(50, 64, device=dev)
    c = shuffled_cache(dev, B, 64, H, D, 32)
    want = host(c)
    q0 = q.cpu().numpy()
    lens, qr = usp.kv8_append(c, k, v, q=q, q_out=q, rope=table, positions=pos.to(dev))
    assert qr is q
    for b in range(B):
        tab = table.cpu().numpy()
        kv8.append(want[0], want[1], want[4][b], 0, kv8.rotate(k[b].cpu().numpy(), pos[b].numpy(), tab))
        kv8.append(want[2], want[3], want[4][b], 0, v[b].cpu().numpy())
        assert np.array_equal(q[b].cpu().numpy(), kv8.rotate(q0[b], pos[b].numpy(), tab))
    for t, w in zip(c[:4], want):
        assert np.array_equal(t.cpu().numpy(), w)


def test_append_one_at_a_time_is_the_oracles():
    """Exponents that rise in the middle of a block, rows rounded again each time."""
    dev = device()
    B, H, D = 2, 2, 64
    x = torch.randn(B, 70, H, D, generator=gen(5)) * torch.logspace(-4, 3, 70)[:, None, None]
    c = shuffled_cache(dev, B, 96, H, D, 32)
    want = host(c)
    for t in range(70):
        usp.kv8_append(c, x[:, t:t + 1].contiguous().to(dev), x[:, t:t + 1].contiguous().to(dev))
        for b in range(B):
            for i in (0, 1):
                kv8.append(want[2 * i], want[2 * i + 1], want[4][b], t, x[b, t:t + 1].numpy())
    for t, w in zip(c[:4], want):
        assert np.array_equal(t.cpu().numpy(), w)
    assert c.seq_lens.tolist() == [70, 70]


def test_append_without_pages_or_tokens():
    dev = device()
    c = shuffled_cache(dev, 3, 128, 2, 64, 32)
    c.page_table[0, 1] = -1
    c.page_table[1, :] = c.k.shape[0]
    c.seq_lens.copy_(i32([20, 0, 5], dev))
    before = [t.clone() for t in c]
    k = torch.randn(3, 50, 2, 64, generator=gen(6)).to(dev)
    want = host(c)
    usp.kv8_append(c, k, k)
    for b in range(3):
        for i in (0, 1):
            kv8.append(want[2 * i], want[2 * i + 1], want[4][b], [20, 0, 5][b], k[b].cpu().numpy())
    for t, w in zip(c[:4], want):
        assert np.array_equal(t.cpu().numpy(), w)
    assert c.seq_lens.tolist() == [70, 50, 55]
    lens = usp.kv8_append(c._replace(seq_lens=before[5]), k[:, :0].contiguous(), k[:, :0].contiguous(),
                          seq_lens_out=c.seq_lens)
    assert lens.tolist() == [20, 0, 5]
    e = usp.kv8_cache(2, 64, 2, 64, num_pages=0, device=dev)  # a pool of none
    usp.kv8_append(e, k[:2].contiguous(), k[:2].contiguous())
    assert e.seq_lens.tolist() == [50, 50] and not usp.kv8_read(e, 50)[0].any()
    out, lse = usp.attn_kv8(k[:2, :1].to(BF).contiguous(), e)
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,page", [(64, 128), (128, 32)])
def test_read_gives_the_values(D, page, dtype):
    dev = device()
    B, H, cap = 4, 3, 256
    c = random_cache(dev, B, cap, H, D, page, [256, 100, 0, 33])
    c.page_table[0, 1] = -5
    starts = [-3, 90, 0, 30]
    k, v = usp.kv8_read(c, 70, starts=i32(starts, dev), dtype=dtype)
    h = host(c)
    for b in range(B):
        for i, got in ((0, k), (1, v)):
            val, _ = kv8.values(h[2 * i], h[2 * i + 1], h[4][b], int(c.seq_lens[b]))
            want = np.zeros((70, H, D))
            for t in range(70):
                if 0 <= starts[b] + t < val.shape[0]:
                    want[t] = val[starts[b] + t]
            assert np.array_equal(np64(got[b]), want)


# --------------------------------------------------------------------- attention

def random_cache(dev, B, cap, H, D, page, lens, seed=0, exps=(-3, 3)):
    """Random codes and exponents; behind the lengths, in the rest of the last block
    too, and in pages of no sequence NaN codes: nothing may read them as keys."""
    c = shuffled_cache(dev, B, cap, H, D, page, seed, fill=0x7F)
    g = gen(seed + 1)
    h = host(c)
    for b in range(B):
        n = min(max(lens[b], 0), h[4].shape[1] * page)
        for r in range(0, n, 32):
            p, at = h[4][b, r // page], r % page
            for i in (0, 1):
                x = torch.randn(H, min(32, n - r), D, generator=g).numpy()
                h[2 * i][p, :, at: at + x.shape[1]] = fp8.e4m3_encode(x * 100)
                h[2 * i + 1][p, :, at // 32] = torch.randint(*exps, (H,), generator=g).numpy() - 6
    for t, w in zip(c[:4], h):
        t.copy_(torch.from_numpy(w))
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    return c


def check_attn(q, c, out, lse, causal=True, window=0, sink=0, cut=None, scale=None):
    """Compares with the oracle, sequence by sequence."""
    h = host(c)
    B = len(c.seq_lens)
    Hq, D = q.shape[-2:]
    scale = D ** -0.5 if scale is None else scale
    flat = [t.reshape((-1,) + tuple(t.shape[-2:] if t is not lse else t.shape[-1:])) for t in (q, out)]
    qf, of, lf = np64(flat[0]), np64(flat[1]), np64(lse.reshape(-1, Hq))
    assert np.isfinite(of).all()
    T = q.shape[1] if cut is None else 0
    for b in range(B):
        a, e = (cut[b], cut[b + 1]) if cut is not None else (b * T, (b + 1) * T)
        n = min(max(int(c.seq_lens[b]), 0), h[4].shape[1] * c.k.shape[2])
        k, there = kv8.values(h[0], h[1], h[4][b], n)
        v, _ = kv8.values(h[2], h[3], h[4][b], n)
        O, L = kv8.attend(qf[a:e], k, v, there, scale, causal, window, sink)
        A, _ = kv8.attend(qf[a:e], k, np.abs(v), there, scale, causal, window, sink)
        assert np.array_equal(np.isneginf(lf[a:e]), np.isneginf(L)), b
        fine = np.isfinite(L)
        if not fine.any():
            assert not of[a:e].any()
            continue
        G = Hq // k.shape[1]
        dot = np.einsum("thd,jhd->thj", np.abs(qf[a:e]), np.abs(np.repeat(k, G, 1))).max()
        ds = D * U * dot * scale + 2.0 ** -22 * (1 + dot * scale)
        big = 448.0 * 2.0 ** max(int(h[3].max()), -40)
        dL = np.abs(np.where(fine, lf[a:e] - np.where(fine, L, 0), 0))
        assert (dL <= ds + n * U + 4 * U * np.abs(np.where(fine, L, 0))).all(), (b, dL.max(), ds)
        tol = A * (2.0 ** -11 + 2 * ds + 2 * n * U) + 2.0 ** -32 * n * big + 2.0 ** -8 * np.abs(O)
        assert (np.abs(of[a:e] - O) <= tol).all(), (b, (np.abs(of[a:e] - O) / np.maximum(tol, 1e-300)).max())


ATTN = [
    # B, T, cap, H, G, D, page, lens, causal, window, sink
    (1, 1, 32, 1, 1, 64, 32, [1], True, 0, 0),
    (1, 1, 128, 1, 1, 128, 64, [128], True, 0, 0),
    (3, 1, 512, 2, 4, 128, 64, [500, 33, 0], True, 0, 0),
    (2, 3, 256, 2, 4, 128, 32, [256, 2], True, 0, 0),             # a sequence shorter than its new tokens
    (2, 2, 1024, 3, 8, 64, 128, [1000, 97], False, 0, 0),
    (2, 1, 2048, 1, 5, 128, 128, [2047, 1024], True, 100, 4),
    (2, 4, 640, 2, 3, 64, 64, [639, 64], True, 33, 70),           # sinks over the window's start
    (1, 5, 512, 2, 2, 128, 64, [512], False, 64, 1),
    (40, 1, 96, 2, 2, 64, 32, [(7 * b) % 97 for b in range(40)], True, 0, 0),
    (1, 1, 32768, 2, 4, 128, 128, [32700], True, 0, 0),
    # room for more keys than a cluster of CTAs takes per unit: units on one line
    (3, 1, 20480, 2, 4, 128, 64, [500, 33, 0], True, 0, 0),
    (2, 3, 32768, 2, 5, 64, 32, [20000, 2], True, 0, 0),
    (2, 2, 65536, 3, 8, 64, 128, [1000, 97], False, 0, 0),
    (2, 1, 20480, 1, 5, 128, 128, [2047, 1024], True, 100, 4),
    (2, 4, 33024, 2, 3, 128, 64, [639, 64], True, 33, 70),
    (40, 1, 4096, 4, 2, 64, 32, [(7 * b) % 97 for b in range(40)], True, 0, 0),
    (40, 5, 96, 4, 4, 64, 32, [(7 * b) % 97 for b in range(40)], True, 0, 0),
    # clusters of 6, 5, 4, 3, 2 CTAs
    (2, 1, 12288, 8, 4, 64, 64, [12288, 31], True, 0, 0),
    (3, 1, 1024, 8, 4, 128, 128, [1024, 0, 97], True, 0, 0),
    (3, 2, 8192, 10, 4, 64, 64, [8191, 700, 1], True, 0, 0),
    (9, 4, 256, 4, 4, 128, 32, [(31 * b) % 257 for b in range(9)], True, 50, 3),
    (5, 3, 320, 4, 5, 64, 32, [64, 320, 0, 289, 5], False, 0, 0),
    (5, 1, 2048, 10, 2, 128, 64, [2048, 1, 65, 1999, 512], True, 0, 0),
    # whole chunks
    (1, 33, 64, 1, 4, 128, 32, [33], True, 0, 0),
    (2, 100, 384, 2, 2, 128, 64, [380, 100], True, 0, 0),
    (2, 129, 512, 1, 1, 64, 32, [129, 500], True, 0, 0),
    (1, 70, 256, 3, 5, 64, 128, [200], False, 0, 0),
    (2, 90, 700, 2, 3, 128, 64, [650, 40], True, 50, 3),          # shorter than its new tokens
    (1, 257, 1024, 1, 8, 128, 128, [1000], True, 200, 200),
    (2, 65, 300, 2, 4, 64, 32, [0, 299], False, 37, 5),
    (1, 600, 2048, 2, 4, 128, 64, [2048], True, 0, 0),
    # more units than the GPU takes at once
    (5, 150, 768, 16, 4, 64, 64, [160, 700, 0, 333, 150], True, 0, 0),
    (70, 9, 384, 8, 3, 128, 128, [(37 * b) % 385 for b in range(70)], True, 0, 0),
]


@pytest.mark.parametrize("B,T,cap,H,G,D,page,lens,causal,window,sink", ATTN)
def test_attention_is_the_oracles(B, T, cap, H, G, D, page, lens, causal, window, sink):
    dev = device()
    c = random_cache(dev, B, cap, H, D, page, lens, seed=T)
    q = torch.randn(B, T, H * G, D, generator=gen(T + 1)).to(BF).to(dev)
    before = [t.clone() for t in c]
    out, lse = usp.attn_kv8(q, c, causal=causal, window=window, sink_tokens=sink)
    check_attn(q, c, out, lse, causal, window, sink)
    for a, b in zip(before, c):
        assert torch.equal(a, b)
    again, lse2 = usp.attn_kv8(q, c, causal=causal, window=window, sink_tokens=sink)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    usp.usp_device_status()


@pytest.mark.parametrize("cut,lens,kw", [
    ([0, 1, 2, 5, 5, 30], [40, 1, 100, 64, 29], dict(window=0)),
    ([2, 3, 4, 140, 141, 300], [70, 0, 250, 129, 300], dict(window=0)),
    ([0, 40, 41, 41, 90, 91], [200, 33, 10, 49, 320], dict(window=40, sink_tokens=2)),
    ([1, 2, 3, 4, 5, 6], [320, 1, 0, 63, 64], dict(causal=False)),
    ([0, 1, 2, 3, 200, 500], [320, 1, 150, 197, 320], dict(window=0, heads=12)),
    # units of few rows and many steps, in which half of the tensor core's rows have no
    # part, before units in which they have
    ([0, 1, 2, 3, 200, 500], [8000, 5000, 3000, 2500, 1800], dict(window=0, heads=8, cap=8192)),
])
@pytest.mark.parametrize("hint", [False, True])
def test_packed_attention_is_the_oracles(cut, lens, kw, hint):
    dev = device()
    kw = dict(kw)
    B, H, G, D = 5, kw.pop("heads", 2), 4, 128
    c = random_cache(dev, B, kw.pop("cap", 320), H, D, 32, lens, seed=cut[-1])
    T = cut[-1] + 3
    q = torch.randn(T, H * G, D, generator=gen(T)).to(BF).to(dev)
    out, lse = usp.attn_kv8(q, c, cu_seqlens=i32(cut, dev),
                            max_new=max(b - a for a, b in zip(cut, cut[1:])) if hint else 0, **kw)
    check_attn(q, c, out, lse, kw.get("causal", True), kw.get("window", 0), kw.get("sink_tokens", 0), cut=cut)
    for s in (slice(0, cut[0]), slice(cut[-1], T)):  # padding
        assert not out[s].any() and torch.isneginf(lse[s]).all()


@pytest.mark.parametrize("first,T", [(0, 700), (100, 400), (695, 700)])
def test_padding_around_single_tokens(first, T):
    dev = device()
    cut = [first + i for i in range(6)]
    c = random_cache(dev, 5, 320, 2, 128, 32, [320, 1, 0, 63, 64])
    q = torch.randn(T, 8, 128, generator=gen(T)).to(BF).to(dev)
    out, lse = usp.attn_kv8(q, c, cu_seqlens=i32(cut, dev), max_new=1)
    check_attn(q, c, out, lse, True, 0, 0, cut=cut)
    for s in (slice(0, cut[0]), slice(cut[-1], T)):
        assert not out[s].any() and torch.isneginf(lse[s]).all()


@pytest.mark.parametrize("T", [1, 40])
def test_rows_without_a_page_are_no_keys(T):
    dev = device()
    c = random_cache(dev, 3, 512, 2, 128, 64, [500, 300, 64], seed=3)
    c.page_table[0, 0] = -1
    c.page_table[0, 3:5] = 1 << 30
    c.page_table[1, :] = -7
    q = torch.randn(3, T, 4, 128, generator=gen(8)).to(BF).to(dev)
    out, lse = usp.attn_kv8(q, c)
    check_attn(q, c, out, lse)
    assert torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("exps", [(-34, 46), (-34, -33), (40, 46)])
def test_blocks_of_very_different_exponents(T, exps):
    """K's exponents up to 2^80 apart are scores of one key alone; V's as far apart."""
    dev = device()
    c = random_cache(dev, 1, 512, 1, 128, 64, [512], seed=3, exps=exps)
    c.k_exp.copy_(torch.randint(-9, -3, c.k_exp.shape, generator=gen(1)).to(torch.int8))
    q = torch.randn(1, T, 2, 128, generator=gen(8)).to(BF).to(dev)
    out, lse = usp.attn_kv8(q, c)
    check_attn(q, c, out, lse)


@pytest.mark.parametrize("T", [1, 33, 130])
def test_many_small_keys_beside_a_sink_count(T):
    """A first key that takes nearly all the attention, with a value of next to nothing,
    and 8191 keys of 2^-24 of its weight: O is theirs."""
    dev = device()
    c = random_cache(dev, 1, 8192, 1, 128, 128, [8192], seed=4)
    h = host(c)
    for p in h[4][0]:
        h[0][p], h[1][p] = 0, 0
        h[2][p], h[3][p] = fp8.e4m3_encode(np.full((1,), 256.0))[0], -2   # V = 64
    p0 = h[4][0, 0]
    h[0][p0, 0, 0] = fp8.e4m3_encode(np.full((128,), 1.0))
    h[2][p0, 0, 0] = 0
    for t, w in zip(c[:4], h):
        t.copy_(torch.from_numpy(w))
    q = torch.full((1, T, 1, 128), 24 * np.log(2.0) / 128 ** 0.5).to(BF).to(dev)
    out, lse = usp.attn_kv8(q, c, causal=False)
    check_attn(q, c, out, lse, causal=False)
    assert float(out.float().min()) > 0.5 * 8191 / 2 ** 24 * 64


@pytest.mark.parametrize("T", [1, 33])
@pytest.mark.parametrize("scale", [1e-30, 4.0])
def test_scales_and_extreme_queries(T, scale):
    dev = device()
    c = random_cache(dev, 2, 128, 1, 64, 64, [128, 50], seed=5)
    q = torch.randn(2, T, 4, 64, generator=gen(9))
    q[0, 0, 0] = 0
    q[0, 0, 1] *= 1e-30
    q[0, 0, 2] *= 1e20 if scale < 1 else 1
    q = q.to(BF).to(dev)
    out, lse = usp.attn_kv8(q, c, softmax_scale=scale)
    check_attn(q, c, out, lse, scale=scale)


@pytest.mark.parametrize("T", [1, 33])
def test_a_nan_query_is_its_own(T):
    dev = device()
    c = random_cache(dev, 1, 128, 2, 64, 64, [100], seed=5)
    q = torch.randn(1, T, 4, 64, generator=gen(9)).to(BF).to(dev)
    want, lse = usp.attn_kv8(q, c)
    q2 = q.clone()
    q2[0, 0, 1, 5] = float("nan")
    got, lse2 = usp.attn_kv8(q2, c)
    assert torch.isnan(got[0, 0, 1]).all()
    got[0, 0, 1], lse2[0, 0, 1] = want[0, 0, 1], lse[0, 0, 1]
    assert torch.equal(got, want) and torch.equal(lse2, lse)


def test_offsets_beyond_32_bits():
    """Pages behind the first 4 GB of a pool."""
    dev = device()
    H, D, page = 8, 128, 128
    n = (1 << 32) // (H * D * page) + 40
    c = usp.kv8_cache(2, 1024, H, D, page_size=page, num_pages=n, device=dev)
    c.page_table.copy_(torch.arange(n - 16, n, dtype=torch.int32).view(2, 8).flip(1))
    small = usp.kv8_cache(2, 1024, H, D, page_size=page, device=dev)
    k, v = (torch.randn(2, 900, H, D, generator=gen(s)).to(BF).to(dev) for s in (1, 2))
    for x in (c, small):
        usp.kv8_append(x, k, v)
    for T in (1, 50, 130):
        q = torch.randn(2, T, H, D, generator=gen(T)).to(BF).to(dev)
        a, b = usp.attn_kv8(q, c), usp.attn_kv8(q, small)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for x, y in zip(usp.kv8_read(c, 900), usp.kv8_read(small, 900)):
        assert torch.equal(x, y)


# ----------------------------------------------------------- together, as served

def serve(dev, c, table, prompts, steps, Hq, D, H, seed):
    """Prompts in two chunks, then single tokens; (outputs, q, k, v of all tokens)."""
    g = gen(seed)
    B = len(prompts)
    tot = [n + steps for n in prompts]
    q = [torch.randn(n, Hq, D, generator=g).to(BF).to(dev) for n in tot]
    k, v = ([torch.randn(n, H, D, generator=g).to(BF).to(dev) for n in tot] for _ in "kv")
    outs = [[] for _ in range(B)]
    at = [0] * B
    for part in range(2):
        n = [p // 2 if part == 0 else p - p // 2 for p in prompts]
        cut = np.concatenate([[0], np.cumsum(n)]).tolist()
        cat = lambda x: torch.cat([x[b][at[b]: at[b] + n[b]] for b in range(B)])  # noqa: E731
        cu = i32(cut, dev)
        _, qr = usp.kv8_append(c, cat(k), cat(v), q=cat(q), rope=table, cu_seqlens=cu)
        o, _ = usp.attn_kv8(qr, c, cu_seqlens=cu)
        for b in range(B):
            outs[b].append(o[cut[b]: cut[b + 1]])
            at[b] += n[b]
    for _ in range(steps):
        one = lambda x: torch.stack([x[b][at[b]: at[b] + 1] for b in range(B)])  # noqa: E731
        _, qr = usp.kv8_append(c, one(k), one(v), q=one(q), rope=table)
        o, _ = usp.attn_kv8(qr, c)
        for b in range(B):
            outs[b].append(o[b])
            at[b] += 1
    return [torch.cat(o) for o in outs], q, k, v


def test_serving_follows_training():
    """Chunks of prompts and decoding steps over the cache against the training path's
    rotation and forward on the same tokens. The cache rounds keys and values to E4M3
    (2^-4 of each at most): against attn_forward of the values read back, which differ
    from the chunks' by codes rounded again as exponents rise, the outputs agree as two
    bf16 roundings of them do; against the unrounded ones within the format's error."""
    dev = device()
    Hq, H, D, prompts, steps = 8, 2, 128, [200, 33], 5
    table = usp.rope_table(512, D, device=dev)
    c = shuffled_cache(dev, 2, 512, H, D, 64)
    outs, q, k, v = serve(dev, c, table, prompts, steps, Hq, D, H, 3)
    for b in range(2):
        n = prompts[b] + steps
        qr, kr = (usp.rope(x[b][None], table) for x in (q, k))
        want, _ = usp.attn_forward(qr, kr, v[b][None].contiguous())
        err = (outs[b].float() - want[0].float()).norm() / want[0].float().norm()
        # |dk| <= 2^-4 |k| moves a score by about 2^-4 |s| / sqrt(12): P and V each off
        # by a few percent of their own size, averaged over the keys
        assert float(err) < 0.1
        kc, vc = usp.kv8_read(c._replace(page_table=c.page_table[b:b + 1].contiguous(),
                                         seq_lens=c.seq_lens[b:b + 1].clone()), n)
        same, _ = usp.attn_forward(qr, kc, vc)
        # the last block's codes may have been rounded again since: 2^-9 of the block's largest
        err = (outs[b].float() - same[0].float()).norm() / same[0].float().norm()
        assert float(err) < 2.0 ** -6


def test_captured_step_replays_as_the_cache_grows():
    dev = device()
    B, H, Hq, D = 3, 2, 8, 128
    table = usp.rope_table(256, D, device=dev)
    g = gen(11)
    k, v = (torch.randn(B, 6, H, D, generator=g).to(BF).to(dev) for _ in "kv")
    q = torch.randn(B, 6, Hq, D, generator=g).to(BF).to(dev)
    caches = [random_cache(dev, B, 256, H, D, 64, [30, 64, 0], seed=2) for _ in "ab"]
    kb, vb, qb = k[:, :1].clone(), v[:, :1].clone(), q[:, :1].clone()
    ws = torch.empty(max(1, usp.usp_attn_kv8_workspace_size(B, 1, 0, False, 256, Hq, H, D)), dtype=torch.uint8, device=dev)

    def step(c):
        _, qr = usp.kv8_append(c, kb, vb, q=qb, rope=table)
        return usp.attn_kv8(qr, c, workspace=ws)

    s = torch.cuda.Stream(device=dev)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(random_cache(dev, B, 256, H, D, 64, [1, 2, 3], seed=2))
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(caches[0])
    for t in range(6):
        for dst, src in ((kb, k), (vb, v), (qb, q)):
            dst.copy_(src[:, t:t + 1])
        graph.replay()
        got = (out.clone(), lse.clone())
        want = step(caches[1])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), t
    assert caches[0].seq_lens.tolist() == [36, 70, 6]
    for a, b in zip(caches[0][:4], caches[1][:4]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 80])
def test_other_streams(T):
    """Every call on a stream of its own choosing, and two attentions at once with a
    workspace each."""
    dev = device()
    c = random_cache(dev, 2, 1024, 2, 128, 64, [900, 1000], seed=6)
    q = torch.randn(2, T, 8, 128, generator=gen(1)).to(BF).to(dev)
    want = usp.attn_kv8(q, c)
    kv = usp.kv8_read(c, 100)
    table = usp.rope_table(1024, 128, device=dev)
    x = usp.rope(q, table)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=dev) for _ in range(2)]
    got = [usp.attn_kv8(q, c, stream=s) for s in streams for _ in range(3)]
    kv2 = usp.kv8_read(c, 100, stream=streams[0])
    x2 = usp.rope(q, table, stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    assert torch.equal(kv2[0], kv[0]) and torch.equal(kv2[1], kv[1]) and torch.equal(x, x2)


def test_a_small_workspace_is_refused():
    dev = device()
    c = random_cache(dev, 2, 65536, 2, 64, 64, [100, 50])
    q = torch.zeros(2, 1, 4, 64, dtype=BF, device=dev)
    with pytest.raises(ValueError):
        usp.attn_kv8(q, c, workspace=torch.empty(128, dtype=torch.uint8, device=dev))
    with pytest.raises(usp.UspError):
        usp.attn_kv8(q[:, :0].contiguous(), c)
