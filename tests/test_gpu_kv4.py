"""GPU parity of the 4-bit KV cache's calls against the oracle.

Codes, scales, moved rows and lengths are compared exactly: the format's
quotients and roundings are those of the definition. Tolerances of the
attention (bf16 output, |ds| the error of a score, n keys, u = 2^-24):
  |ds| <= D u max_ij sum_d |q_d k_d| scale  (fp32 accumulation of exact
          products) + 2^-22 (scaling, maximum, exp2)
  LSE:    |ds| + n u + 4 u |LSE|
  O:      A (2^-11 + 2 |ds| + 2 n u) + 2^-25 n max|v| + 2^-8 |O|
          with A = sum_j P_j |v_j|: P is rounded to fp16 (2^-11, and 2^-25
          where it is subnormal, against a sum of at least 1), O to bf16
  weight: w (2 |ds| + 2 n u + 8 u) + u |total|"""
import numpy as np
import pytest
import torch

import sequence_long_context_gb300 as usp
from oracle import kv4, layouts
from tests._gpu import device

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FIELDS = ("k", "k_scale", "v", "v_scale")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def random_cache(dev, B, C, H, D, lens, seed=0, descale=1.0, weight=True):
    """A cache whose rows hold quantized normal values, behind the lengths
    rows of all-ones bytes (NaN scales, codes 7): nothing may read them."""
    g = gen(seed)
    c = usp.kv4_cache(B, C, H, D, device=dev, key_weight=weight, k_descale=descale,
                      v_descale=descale)
    C = c.k.shape[2]
    for a, b in (("k", "k_scale"), ("v", "v_scale")):
        x = torch.randn(B, H, C, D, generator=g) * (2.0 if a == "k" else 1.0)
        codes, sb = kv4.quantize(x, descale)
        for i, n in enumerate(lens):
            codes[i, :, max(n, 0):] = 255
            sb[i, :, max(n, 0):] = 255
        getattr(c, a).copy_(torch.from_numpy(codes))
        getattr(c, b).copy_(torch.from_numpy(sb))
    if weight:
        c.key_weight.copy_(torch.rand(B, H, C, generator=g))
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    return c


def cache_values(c):
    return [kv4.values(getattr(c, a).cpu().numpy(), getattr(c, b).cpu().numpy(), d)
            for a, b, d in (("k", "k_scale", c.k_descale), ("v", "v_scale", c.v_descale))]


def snapshot(c):
    return [None if t is None else t.clone() for t in c[:6]]


# ------------------------------------------------------------------ append, read

APPEND = [
    # B, T, C, H, D, dtype, starts
    (1, 1, 16, 1, 64, torch.bfloat16, [0]),
    (3, 1, 64, 2, 128, torch.bfloat16, [0, 17, 63]),
    (2, 7, 48, 3, 128, torch.float32, [5, 41]),      # exactly to the end
    (2, 9, 32, 2, 64, torch.float32, [0, 28]),       # the second runs out of room
    (4, 100, 256, 2, 128, torch.bfloat16, [0, 3, 150, 256]),  # and one is full
    (2, 333, 400, 1, 64, torch.bfloat16, [1, 50]),
    (1, 65, 128, 5, 128, torch.float32, [-7]),       # a negative length counts as 0
]


@pytest.mark.parametrize("descale", [1.0, 0.37])
@pytest.mark.parametrize("B,T,C,H,D,dtype,starts", APPEND)
def test_append_stores_the_definitions_bytes(B, T, C, H, D, dtype, starts, descale):
    dev = device()
    g = gen(T)
    k = (torch.randn(B, T, H, D, generator=g) * torch.logspace(-3, 2, D)).to(dtype)
    v = torch.randn(B, T, H, D, generator=g).to(dtype)
    k[0, 0, 0, :8] = torch.tensor([float("nan"), float("inf"), -float("inf"), 0, -0.0, 1e-30, 7, 3.5])
    v[0, 0, 0, :32] = 0
    c = usp.kv4_cache(B, C, H, D, device=dev, key_weight=True, k_descale=descale, v_descale=descale)
    for t in c[:4]:
        t.fill_(0xAB)
    c.key_weight.fill_(5)
    c.seq_lens.copy_(torch.tensor(starts, dtype=torch.int32))
    w = torch.rand(B, H, T, generator=g)
    lens = usp.kv4_append(c, k.to(dev), v.to(dev), key_weight=w.to(dev))
    assert lens is c.seq_lens
    at = [min(max(s, 0), C) for s in starts]
    assert lens.tolist() == [min(C, a + T) for a in at]
    for x, name in ((k, "k"), (v, "v")):
        codes, sb = kv4.quantize(x, descale)
        want = np.full(getattr(c, name).shape, 0xAB, np.uint8)
        want_s = np.full(getattr(c, name + "_scale").shape, 0xAB, np.uint8)
        for b in range(B):
            n = min(T, C - at[b])
            want[b, :, at[b]:at[b] + n] = codes[b, :n].swapaxes(0, 1)
            want_s[b, :, at[b]:at[b] + n] = sb[b, :n].swapaxes(0, 1)
        assert np.array_equal(getattr(c, name).cpu().numpy(), want), name
        assert np.array_equal(getattr(c, name + "_scale").cpu().numpy(), want_s), name
    want_w = np.full(c.key_weight.shape, 5, np.float32)
    for b in range(B):
        n = min(T, C - at[b])
        want_w[b, :, at[b]:at[b] + n] = w[b, :, :n]
    assert np.array_equal(c.key_weight.cpu().numpy(), want_w)


@pytest.mark.parametrize("H,D,cut", [(2, 128, [0, 5, 5, 70, 71]), (3, 64, [0, 0, 40, 300, 300])])
def test_append_packed_is_each_sequence_alone(H, D, cut):
    dev = device()
    g = gen(9)
    B, T = len(cut) - 1, cut[-1]
    k, v = (torch.randn(T, H, D, generator=g).to(torch.bfloat16).to(dev) for _ in "kv")
    w = torch.rand(H, T, generator=g).to(dev)
    starts = torch.tensor([3, 0, 16, 9], dtype=torch.int32, device=dev)
    a = usp.kv4_cache(B, 320, H, D, device=dev, key_weight=True)._replace(seq_lens=starts)
    b = usp.kv4_cache(B, 320, H, D, device=dev, key_weight=True)
    out = torch.full((B,), -1, dtype=torch.int32, device=dev)
    got = usp.kv4_append(a, k, v, key_weight=w, seq_lens_out=out,
                         cu_seqlens=torch.tensor(cut, dtype=torch.int32, device=dev))
    assert got is out and starts.tolist() == [3, 0, 16, 9]
    assert out.tolist() == [s + cut[i + 1] - cut[i] for i, s in enumerate(starts.tolist())]
    for i in range(B):
        one = usp.KV4Cache(*[t[i:i + 1] for t in b[:4]], seq_lens=starts[i:i + 1].clone(),
                           key_weight=b.key_weight[i:i + 1])
        s = slice(cut[i], cut[i + 1])
        usp.kv4_append(one, k[None, s].contiguous(), v[None, s].contiguous(),
                       key_weight=w[None, :, s].contiguous())
    for x, y in zip(a[:4] + (a.key_weight,), b[:4] + (b.key_weight,)):
        assert torch.equal(x, y)


def test_append_packed_leaves_tokens_outside_the_boundaries():
    """A padded batch: tokens before the first boundary and behind the last
    belong to no sequence, and no row behind a sequence's end is written."""
    dev = device()
    g = gen(10)
    k, v = (torch.randn(60, 2, 64, generator=g).to(torch.bfloat16).to(dev) for _ in "kv")
    w = torch.rand(2, 60, generator=g).to(dev)
    c = usp.kv4_cache(2, 64, 2, 64, device=dev, key_weight=True)
    for t in c[:4]:
        t.fill_(0xAB)
    c.key_weight.fill_(5)
    cu = torch.tensor([4, 20, 41], dtype=torch.int32, device=dev)
    assert usp.kv4_append(c, k, v, key_weight=w, cu_seqlens=cu).tolist() == [16, 21]
    for b, n in enumerate((16, 21)):
        for t in c[:4]:
            assert (t[b, :, n:] == 0xAB).all()
        assert (c.key_weight[b, :, n:] == 5).all()
        s = slice(int(cu[b]), int(cu[b]) + n)
        assert torch.equal(c.key_weight[b, :, :n], w[:, s])
        codes, sb = kv4.quantize(k[s].cpu(), 1.0)
        assert np.array_equal(c.k[b, :, :n].cpu().numpy(), codes.swapaxes(0, 1))
        assert np.array_equal(c.k_scale[b, :, :n].cpu().numpy(), sb.swapaxes(0, 1))


def test_append_without_weights_starts_new_keys_at_zero():
    dev = device()
    c = usp.kv4_cache(1, 32, 2, 64, device=dev, key_weight=True)
    c.key_weight.fill_(float("nan"))
    x = torch.ones(1, 5, 2, 64, device=dev, dtype=torch.bfloat16)
    usp.kv4_append(c, x, x)
    assert (c.key_weight[:, :, :5] == 0).all() and c.key_weight[:, :, 5:].isnan().all()
    before = snapshot(c)
    usp.kv4_append(c, x[:, :0], x[:, :0])  # no token
    for x, y in zip(before[:4], c[:4]):
        assert torch.equal(x, y)
    assert c.seq_lens.tolist() == [5]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,C,H,D,lens,tokens,starts,descale", [
    (1, 16, 1, 64, [1], 1, None, 1.0),
    (3, 64, 2, 128, [0, 64, 33], 64, None, 0.37),
    (2, 160, 3, 128, [150, 20], 37, [120, 5], 2.0),
    (2, 48, 2, 64, [48, 9], 60, [-3, 8], 1.0),       # before 0 and behind the capacity
])
def test_read_gives_the_values(B, C, H, D, lens, tokens, starts, descale, dtype):
    dev = device()
    c = random_cache(dev, B, C, H, D, lens, seed=C, descale=descale)
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device=dev)
    k, v = usp.kv4_read(c, tokens, starts=st, dtype=dtype)
    for got, want in zip((k, v), cache_values(c._replace(k_descale=1.0, v_descale=1.0))):
        # fp32 product with the descale, then the output's rounding
        want = torch.from_numpy((want.astype(np.float32) * np.float32(descale))).to(dtype)
        full = torch.zeros(B, tokens, H, D, dtype=dtype)
        for b in range(B):
            for t in range(tokens):
                p = (starts[b] if starts else 0) + t
                if 0 <= p < lens[b]:
                    full[b, t] = want[b, :, p]
        assert torch.equal(got.cpu(), full)


# ------------------------------------------------------------------------ decode

DECODE = [
    # B, Tq, C, Hq, H, D, lens, causal, window, sink, descale
    (1, 1, 16, 1, 1, 64, [1], True, 0, 0, 1.0),
    (1, 1, 16, 4, 1, 128, [16], True, 0, 0, 1.0),
    (4, 1, 112, 8, 2, 128, [0, 1, 33, 100], True, 0, 0, 0.5),
    (3, 2, 64, 6, 3, 64, [0, 1, 64], True, 0, 0, 1.0),     # a token without a position
    (2, 3, 256, 8, 2, 128, [255, 31], True, 0, 0, 0.37),   # 12 rows per KV head
    (2, 3, 64, 8, 2, 64, [2, 40], False, 0, 0, 1.0),
    (1, 5, 320, 16, 2, 128, [301], True, 0, 0, 1.0),       # 40 rows: three blocks
    (2, 1, 512, 32, 1, 64, [500, 17], True, 0, 0, 1.0),    # multi-query
    (5, 1, 96, 4, 4, 128, [96, 95, 65, 64, 63], True, 0, 0, 1.0),
    (2, 1, 1024, 8, 2, 128, [1000, 300], True, 100, 4, 1.0),
    (2, 2, 1024, 4, 2, 64, [1024, 37], True, 1, 0, 1.0),   # sees itself alone
    (2, 2, 512, 4, 2, 128, [512, 200], False, 40, 70, 1.0),
    (1, 1, 512, 4, 2, 128, [400], True, 1000, 4, 1.0),     # a window past the start
    (40, 1, 48, 2, 1, 64, [(7 * i) % 49 for i in range(40)], True, 0, 0, 1.0),
    (2, 1, 20000, 8, 2, 128, [19999, 12345], True, 0, 0, 1.0),
    (3, 16, 144, 2, 2, 128, [144, 15, 16], True, 0, 0, 1.0),
]


def check_decode(c, q, out, lse, weight, old, lens, causal, window, sink):
    B, Tq, Hq, D = q.shape
    H, C = c.k.shape[1], c.k.shape[2]
    lens = [min(max(n, 0), C) for n in lens]
    kv, vv = cache_values(c)
    for b, n in enumerate(lens):
        kv[b, :, n:] = 0
        vv[b, :, n:] = 0
    scale = 1 / np.sqrt(D)
    O, L, W = kv4.decode(q, kv, vv, lens, scale, causal, window, sink)
    A, _, _ = kv4.decode(q, kv, np.abs(vv), lens, scale, causal, window, sink)
    n = max(lens + [1])
    qa = np.abs(q.double().cpu().numpy()).max(axis=(0, 1, 2))
    ds = D * U * scale * (qa * np.abs(kv).max(axis=(0, 1, 2))).sum() + 2.0 ** -22
    got = out.double().cpu().numpy()
    bound = A * (2.0 ** -11 + 2 * ds + 2 * n * U) + 2.0 ** -25 * n * np.abs(vv).max() \
        + 2.0 ** -8 * np.abs(O)
    assert (np.abs(got - O) <= bound + 1e-30).all(), np.abs(got - O).max()
    gl = lse.double().cpu().numpy()
    assert np.array_equal(np.isfinite(gl), np.isfinite(L))
    assert (got[~np.isfinite(L)] == 0).all() and (gl[~np.isfinite(L)] == -np.inf).all()
    f = np.isfinite(L)
    assert (np.abs(gl[f] - L[f]) <= ds + n * U + 4 * U * np.abs(L[f])).all()
    if weight is not None:
        total = old.double().cpu().numpy() + W
        gw = weight.double().cpu().numpy()
        assert (np.abs(gw - total) <= W * (2 * ds + 2 * n * U + 8 * U) + U * np.abs(total)).all()
        for b, m in enumerate(lens):  # rows behind the sequence stay as they were
            assert torch.equal(weight[b, :, m:], old[b, :, m:])


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("B,Tq,C,Hq,H,D,lens,causal,window,sink,descale", DECODE)
def test_decode_matches_oracle(B, Tq, C, Hq, H, D, lens, causal, window, sink, descale, accumulate):
    dev = device()
    c = random_cache(dev, B, C, H, D, lens, seed=C + Tq, descale=descale)
    q = (torch.randn(B, Tq, Hq, D, generator=gen(B)) * 1.5).to(torch.bfloat16)
    before = snapshot(c)
    ws = torch.full((usp.usp_attn_decode_kv4_workspace_size(B, Tq, c.k.shape[2], Hq, H, D, accumulate),),
                    255, dtype=torch.uint8, device=dev)  # NaNs: entry contents do not matter
    out, lse = usp.attn_decode_kv4(q.to(dev), c, causal=causal, window=window, sink_tokens=sink,
                                   accumulate=accumulate, workspace=ws)
    usp.usp_device_status()
    for x, y in zip(before[:5], c[:5]):
        assert torch.equal(x, y)
    if not accumulate:
        assert torch.equal(before[5], c.key_weight)
    check_decode(c, q, out, lse, c.key_weight if accumulate else None, before[5], lens, causal,
                 window, sink)
    again, lse2 = usp.attn_decode_kv4(q.to(dev), c, causal=causal, window=window, sink_tokens=sink)
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # and the same every time


def test_decode_lengths_out_of_range_are_clamped():
    dev = device()
    c = random_cache(dev, 2, 48, 2, 64, [48, 48], seed=1)
    q = torch.randn(2, 1, 4, 64, generator=gen(2)).to(torch.bfloat16).to(dev)
    want = usp.attn_decode_kv4(q, c)
    c.seq_lens.copy_(torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32))
    got = usp.attn_decode_kv4(q, c)
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[1][0], want[1][0])
    assert (got[0][1] == 0).all() and (got[1][1] == -float("inf")).all()


def test_decode_large_scores_and_equal_keys():
    """Scores in the thousands (one key takes all), and one value throughout:
    the output is that value."""
    dev = device()
    c = random_cache(dev, 1, 4096, 1, 128, [4000], seed=3, descale=4.0)
    q = (torch.randn(1, 1, 4, 128, generator=gen(3)) * 40).to(torch.bfloat16)
    out, lse = usp.attn_decode_kv4(q.to(dev), c)
    kv, vv = cache_values(c)
    kv[:, :, 4000:] = vv[:, :, 4000:] = 0
    O, L, _ = kv4.decode(q, kv, vv, [4000], 1 / np.sqrt(128))
    ds = 128 * U * np.abs(q.double().numpy()).max() * 128 * np.abs(kv).max() / np.sqrt(128)
    assert (np.abs(lse.cpu().numpy() - L) <= ds + 4 * U * np.abs(L)).all()
    assert np.isfinite(out.float().cpu().numpy()).all()
    c.v.fill_(0xCC)        # code 4
    c.v_scale.fill_(0x38)  # 1
    out, _ = usp.attn_decode_kv4(q.to(dev), c)
    assert torch.allclose(out.float(), torch.full_like(out.float(), 16.0), rtol=2.0 ** -8 + 2.0 ** -10)


@pytest.mark.parametrize("descale", [1e-30, 1e-37])
def test_decode_zero_queries_with_a_tiny_descale(descale):
    """Scores too small for fp32 are 0, and masked keys stay masked: the output
    is the mean of the visible values (2^-8 of it, and of the mean of the
    values' magnitudes 2^-11 and n u for the sums)."""
    dev = device()
    c = random_cache(dev, 1, 112, 1, 64, [100], seed=12)._replace(k_descale=descale)
    q = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16, device=dev)
    out, lse = usp.attn_decode_kv4(q, c)
    vv = cache_values(c)[1]
    for t in range(3):
        n = 98 + t
        x = vv[0, 0, :n].astype(np.float64)
        bound = 2.0 ** -8 * np.abs(x.mean(0)) + np.abs(x).mean(0) * (2.0 ** -11 + 2 * n * U)
        for h in range(2):
            assert (np.abs(out[0, t, h].double().cpu().numpy() - x.mean(0)) <= bound).all()
            assert abs(float(lse[0, t, h]) - np.log(n)) <= n * U + 4 * U * np.log(n) + 2.0 ** -22


def test_decode_nan_query_stays_in_its_rows():
    dev = device()
    c = random_cache(dev, 2, 64, 2, 64, [60, 40], seed=4)
    q = torch.randn(2, 2, 4, 64, generator=gen(4)).to(torch.bfloat16).to(dev)
    want, wl = usp.attn_decode_kv4(q, c)
    q[0, 1, 2, 5] = float("nan")
    got, gl = usp.attn_decode_kv4(q, c)
    hit = torch.zeros(2, 2, 4, dtype=torch.bool)
    hit[0, 1, 2] = True
    assert got[hit.to(dev)].isnan().all() and gl[hit.to(dev)].isnan().all()
    assert torch.equal(got[~hit.to(dev)], want[~hit.to(dev)])
    assert torch.equal(gl[~hit.to(dev)], wl[~hit.to(dev)])


@pytest.mark.parametrize("D,Tq,lens,window,sink", [
    (128, 1, [1007 - 61 * i for i in range(16)], 0, 0),     # 32 down to 3 steps
    (128, 1, [5000 - 37 * i for i in range(16)], 1000, 4),  # 33 steps: one warp in the last round
    (64, 1, [513 + 32 * i for i in range(16)], 0, 0),
    (128, 9, [300 + 33 * i for i in range(16)], 0, 0),      # two tiles of query rows
])
def test_decode_many_units_whose_last_rounds_are_partial(D, Tq, lens, window, sink):
    """512 units (or twice that) of 3 to 34 steps: each CTA passes several unit ends at which some
    warps have no step, while the copies of the next units are under way. A warp
    that releases such a round's stage early lets it be overwritten while another
    reads it: outputs then differ between runs, or from the oracle's."""
    dev = device()
    B, H = len(lens), 32
    c = random_cache(dev, B, max(lens), H, D, lens, seed=D + Tq)
    q = torch.randn(B, Tq, H, D, generator=gen(Tq)).to(torch.bfloat16)
    qd = q.to(dev)
    out, lse = usp.attn_decode_kv4(qd, c, window=window, sink_tokens=sink)
    usp.usp_device_status()
    for _ in range(20):
        again, lse2 = usp.attn_decode_kv4(qd, c, window=window, sink_tokens=sink)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
    usp.usp_device_status()
    for b in (0, 7, 15):  # whole sequences against the oracle
        one = c._replace(**{n: getattr(c, n)[b:b + 1] for n in FIELDS + ("seq_lens", "key_weight")})
        check_decode(one, q[b:b + 1], out[b:b + 1], lse[b:b + 1], None, one.key_weight,
                     lens[b:b + 1], True, window, sink)


@pytest.mark.parametrize("B,Tq,C,G,H,D", [(1, 1, 131072, 1, 64, 64), (1, 1, 2 ** 20, 1, 16, 128),
                                          (2, 3, 131072, 4, 16, 128)])
def test_decode_long_rows_lose_nothing_but_the_roundings(B, Tq, C, G, H, D):
    """Random values, whose weighted mean is some hundred times smaller than they
    are. bf16 rounds O by at most 2^-8 of it, each evenly spread: 2^-8 / sqrt 3 rms
    at most; P's roundings (2^-11 each, independent) add 2^-11 / sqrt 3 of O; the
    rest of the error, of sums in fp32, may be a tenth of that of bf16."""
    dev = device()
    c = usp.kv4_cache(B, C, H, D, device=dev)
    torch.manual_seed(B + C)
    for _ in range(C // 8192):
        k, v = (torch.randn(B, 8192, H, D, device=dev, dtype=torch.bfloat16) for _ in "kv")
        usp.kv4_append(c, k, v)
    q = torch.randn(B, Tq, G * H, D, device=dev).to(torch.bfloat16)
    out, _ = usp.attn_decode_kv4(q, c, causal=False)
    err = ref = 0.0
    for h in range(0, H, H // 4):
        one = usp.KV4Cache(*(t[:1, h:h + 1].contiguous() for t in c[:4]), c.seq_lens[:1])
        kv, vv = (t[0, :, 0].double() for t in usp.kv4_read(one, C, dtype=torch.float32))
        s = q[0, :, h * G:(h + 1) * G].double() @ kv.T / D ** 0.5
        o = torch.softmax(s, -1) @ vv
        err += float(((out[0, :, h * G:(h + 1) * G].double() - o) ** 2).sum())
        ref += float((o ** 2).sum())
    assert (err / ref) ** 0.5 <= (1.1 * 2.0 ** -8 + 2.0 ** -11) / 3 ** 0.5


@pytest.mark.parametrize("sink_scale", [0.0, 0.25])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 1), (128, 12)])
def test_decode_keys_far_below_the_dominant_ones(D, G, sink_scale):
    """304 units of 4096 keys, so that a CTA has one or two; eight keys, one in
    each warp's share, outweigh every other by 2^23.4 and have V = 0. O is then
    what the others give, each p = 1.57 2^-24 of the largest. Bound: bf16 (2^-8),
    the rounding of p, held in steps of at most 2^-24 of 2^-7 of the largest
    (2^-32 / p = 0.26 %), and the sums (2 n u). A block of zeros is stored with the
    scale 0. Zero codes under a scale s (of a block with other numbers) stand in the
    step's two sums as 8 s p_max and cancel: each of the step's 32 keys may lose an
    ulp, 2^-23 of that, in each sum, so against l >= p_max 2^-17 8 s are added."""
    dev = device()
    B, H, L = 16, 19, 4096
    c = usp.kv4_cache(B, L, H, D, device=dev)
    c.k.fill_(0x88)          # codes 0
    c.k_scale.fill_(0x38)    # 1
    c.v.fill_(0xCC)          # code 4
    c.v_scale.fill_(0x28)    # 1/4
    c.k[:, :, 0:256:32, 0] = 0x8F  # channel 0: 7
    c.v[:, :, 0:256:32] = 0x88
    c.v_scale[:, :, 0:256:32] = 0x28 if sink_scale else 0
    c.seq_lens.fill_(L)
    q = torch.zeros(B, 1, G * H, D, dtype=torch.bfloat16, device=dev)
    q[..., 0] = 2.3125
    out, lse = usp.attn_decode_kv4(q, c, softmax_scale=1.0)
    p, n = np.exp(-7 * 2.3125), L - 8
    want = n * p / (8 + n * p)
    bound = want * (2.0 ** -8 + 2.0 ** -32 / p + 2 * L * U + 2.0 ** -20) \
        + 2.0 ** -17 * 8 * sink_scale
    assert float((out.double() - want).abs().max()) <= bound
    assert float((lse.double() - np.log(8 / p + n)).abs().max()) <= L * U + 20 * 4 * U + 2.0 ** -20


@pytest.mark.parametrize("D,Tq", [(64, 1), (128, 3)])
@pytest.mark.parametrize("which,descale", [("v", 3e37), ("v", 3.4e38), ("k", 3e37), ("k", 3.4e38)])
def test_decode_with_the_largest_descales(which, descale, D, Tq):
    """The smallest scales under descales up to fp32's largest number: the values
    and the scores are ordinary numbers (k: under queries near 2^-121)."""
    dev = device()
    c = random_cache(dev, 2, 112, 2, D, [100, 57], seed=15)._replace(**{which + "_descale": descale})
    for b, n in enumerate((100, 57)):
        getattr(c, which + "_scale")[b, :, :n] = 1  # 2^-9
    q = torch.randn(2, Tq, 8, D, generator=gen(16)) * (2.0 ** -121 if which == "k" else 1.0)
    q = q.to(torch.bfloat16)
    out, lse = usp.attn_decode_kv4(q.to(dev), c)
    check_decode(c, q, out, lse, None, None, [100, 57], True, 0, 0)


def test_decode_long_cache_offsets_pass_32_bits():
    """Codes of the last head start behind 4 GiB; only its rows are filled."""
    dev = device()
    B, H, C, D = 1, 9, 8 * 2 ** 20, 128
    if torch.cuda.mem_get_info()[0] < 30 * 2 ** 30:
        pytest.skip("needs 30 GB")
    c = usp.kv4_cache(B, C, H, D, device=dev, key_weight=True)
    small = random_cache(dev, 1, 4096, 1, D, [4096], seed=6)
    L = C - 5
    lo = L - 4096
    for a in FIELDS:
        getattr(c, a)[:, 8:, lo:L] = getattr(small, a)
    c.seq_lens.fill_(L)
    q = torch.randn(1, 1, 9, D, generator=gen(5)).to(torch.bfloat16).to(dev)
    # the window shows the filled rows alone
    out, lse = usp.attn_decode_kv4(q, c, window=4096, accumulate=True)
    want, wl = usp.attn_decode_kv4(q[:, :, 8:].contiguous(), small, accumulate=False)
    assert torch.allclose(out[:, :, 8:].float(), want.float(), atol=2.0 ** -8, rtol=2.0 ** -7)
    assert torch.allclose(lse[:, :, 8:], wl, rtol=1e-5)
    assert abs(float(c.key_weight[0, 8].double().sum()) - 1) < 1e-4
    x = torch.ones(1, 3, 9, D, device=dev, dtype=torch.bfloat16)
    usp.kv4_append(c, x, x)
    k, v = usp.kv4_read(c, 4, starts=torch.tensor([L - 1], dtype=torch.int32, device=dev))
    # e4m3(1 / 7) is 9/64 and the code 7, so a 1 stands for 63/64
    assert (k[0, 1:] == 63 / 64).all() and (v[0, 1:] == 63 / 64).all()
    assert c.seq_lens.item() == L + 3


# ------------------------------------------------------------------- key weights

WEIGHTS = [
    # B, S, Hq, H, D, causal, window, sink, cp, layout, observe, cut
    (1, 1, 1, 1, 64, True, 0, 0, 1, "contiguous", 0, None),
    (2, 3, 4, 2, 128, True, 0, 0, 1, "contiguous", 0, None),
    (1, 129, 4, 1, 128, True, 0, 0, 1, "contiguous", 0, None),
    (2, 300, 2, 2, 64, False, 0, 0, 1, "contiguous", 0, None),
    (1, 513, 6, 2, 64, True, 0, 0, 1, "contiguous", 7, None),
    (1, 700, 4, 2, 128, True, 50, 3, 1, "contiguous", 0, None),
    (1, 520, 4, 2, 128, False, 33, 0, 1, "contiguous", 100, None),
    (1, 1024, 4, 2, 128, True, 0, 0, 4, "zigzag", 0, None),
    (1, 1024, 4, 2, 64, True, 0, 0, 2, "stripe", 90, None),
    (2, 776, 4, 2, 64, True, 100, 4, 4, "zigzag", 0, None),     # chunks of 97
    (1, 390, 2, 1, 128, True, 0, 0, 3, "stripe", 0, None),
    (1, 380, 2, 1, 128, True, 64, 0, 2, "contiguous", 33, None),
    (1, 601, 4, 2, 128, True, 0, 0, 1, "contiguous", 0, [0, 1, 1, 200, 455, 601]),
    (1, 640, 4, 4, 64, True, 40, 2, 2, "zigzag", 30, [0, 5, 300, 640]),
    (1, 512, 2, 1, 64, False, 0, 0, 4, "stripe", 10, [0, 100, 512]),
    (1, 4096, 8, 2, 128, True, 0, 0, 1, "contiguous", 0, None),  # several parts
    # one tile of at most 64 observed rows: two heads share it (an odd group: not)
    (2, 700, 8, 2, 128, True, 0, 0, 1, "contiguous", 64, None),
    (1, 130, 4, 2, 64, False, 0, 0, 1, "contiguous", 33, None),
    (1, 1100, 3, 1, 128, True, 0, 0, 1, "contiguous", 1, None),
    (1, 50, 2, 1, 64, True, 0, 0, 1, "contiguous", 0, None),
    (2, 640, 4, 1, 128, True, 70, 2, 1, "contiguous", 40, None),
]


@pytest.mark.parametrize("path", ["bf16", "simt", "fp32"])
@pytest.mark.parametrize("B,S,Hq,H,D,causal,window,sink,cp,layout,observe,cut", WEIGHTS)
def test_key_weights_match_oracle(B, S, Hq, H, D, causal, window, sink, cp, layout, observe, cut, path):
    from oracle import attention
    dev = device()
    dt = torch.float32 if path == "fp32" else torch.bfloat16
    g = gen(S)
    q = torch.randn(B, S, Hq, D, generator=g).to(dt)
    k = torch.randn(B, S, H, D, generator=g).to(dt)
    if cut:
        q, k = q[0], k[0]
    scale = 1 / np.sqrt(D)
    cu = None if cut is None else np.array(cut)
    _, lse = attention.attn_fwd(q, k, k, scale, causal, window, sink, cu_seqlens=cu)
    lse32 = lse.astype(np.float32)
    want = kv4.key_weights(q, k, lse32, scale, causal, window, sink, cut, observe)
    ax = 0 if cut else 1
    qp, kp = (torch.from_numpy(layouts.extract(t.float().numpy(), layout, cp, axis=ax)).to(dt).to(dev)
              for t in (q, k))
    lp = torch.from_numpy(layouts.extract(lse32, layout, cp, axis=lse.ndim - 1)).to(dev)
    got = usp.attn_key_weights(
        qp, kp, lp.contiguous(), causal=causal, window=window, sink_tokens=sink,
        cu_seqlens=None if cut is None else torch.tensor(cut, dtype=torch.int32, device=dev),
        cp=cp, layout=layout, observe=observe, flags=usp.FLAG_FORCE_SIMT if path == "simt" else 0)
    usp.usp_device_status()
    w = layouts.restore(got.double().cpu().numpy(), layout, cp, axis=got.dim() - 1)
    ds = D * U * scale * (np.abs(q.double().numpy()).max() * np.abs(k.double().numpy()).max()) * D
    bound = want * (2 * ds + 4 * U * np.abs(lse32[np.isfinite(lse32)]).max() + 2 * S * U + 2.0 ** -20)
    assert w.shape == want.shape
    assert (np.abs(w - want) <= bound + 1e-37).all(), (np.abs(w - want) / np.maximum(want, 1e-30)).max()


@pytest.mark.parametrize("B,S,Hq,H,D,observe,window,sink", [
    (1, 33333, 4, 2, 128, 64, 0, 0),       # two tiles of two heads each
    (1, 20011, 8, 1, 64, 17, 0, 0),        # four
    (2, 9000, 2, 1, 128, 130, 0, 0),       # two heads of two tiles
    (1, 30000, 6, 2, 128, 90, 0, 0),       # three heads
    (2, 9000, 3, 1, 128, 130, 0, 0),       # six tiles: no longer kept
    (1, 16385, 2, 2, 128, 1, 0, 0),        # one query; one key in the last block
    (1, 40000, 4, 4, 64, 100, 5000, 300),  # blocks between that nobody sees
    (1, 70001, 1, 1, 64, 3, 0, 0),
])
def test_key_weights_of_few_queries_over_long_prompts(B, S, Hq, H, D, observe, window, sink):
    """Runs of key blocks pass by an item's queries; the bound is that of the
    comparison with the oracle."""
    dev = device()
    torch.manual_seed(S)
    q = torch.randn(B, S, Hq, D, device=dev).to(torch.bfloat16)
    k = torch.randn(B, S, H, D, device=dev).to(torch.bfloat16)
    scale = 1 / np.sqrt(D)
    i = torch.arange(S - observe, S, device=dev)[:, None]
    j = torch.arange(S, device=dev)[None]
    see = j <= i
    if window:
        see &= (i - j < window) | (j < sink)
    lse = torch.full((B, Hq, S), float("nan"), device=dev)  # of the others: not read
    want = torch.zeros(B, H, S, dtype=torch.float64, device=dev)
    for b in range(B):
        for h in range(Hq):
            s = q[b, S - observe:, h].double() @ k[b, :, h // (Hq // H)].double().T * scale
            s.masked_fill_(~see, -float("inf"))
            lse[b, h, S - observe:] = s.logsumexp(-1).float()
            want[b, h // (Hq // H)] += torch.exp(s - lse[b, h, S - observe:, None].double()).sum(0)
    got = usp.attn_key_weights(q, k, lse, window=window, sink_tokens=sink, observe=observe)
    usp.usp_device_status()
    ds = D * U * scale * float(q.abs().max() * k.abs().max()) * D
    top = float(lse[:, :, S - observe:].abs().max())
    bound = want * (2 * ds + 4 * U * top + 2 * observe * Hq * U + 2.0 ** -20)
    assert ((got.double() - want).abs() <= bound + 1e-37).all()
    again = usp.attn_key_weights(q, k, lse, window=window, sink_tokens=sink, observe=observe)
    assert torch.equal(got, again)


def check_weights_of_many_items(B, S, Hq, H, D, observe):
    """The last `observe` queries of B prompts, against 64 bits (the bound of the
    comparison with the oracle), and the same bits every time. With B H items of one
    or more runs, above 152, a CTA takes several, one behind the other."""
    dev = device()
    torch.manual_seed(S + Hq)
    q = torch.randn(B, S, Hq, D, device=dev).to(torch.bfloat16)
    k = torch.randn(B, S, H, D, device=dev).to(torch.bfloat16)
    scale, n = 1 / np.sqrt(D), min(observe, S) or S
    see = torch.arange(S, device=dev)[None] <= torch.arange(S - n, S, device=dev)[:, None]
    lse = torch.full((B, Hq, S), float("nan"), device=dev)  # of the others: not read
    want = torch.zeros(B, H, S, dtype=torch.float64, device=dev)
    for h in range(Hq):
        s = torch.einsum("bqd,bkd->bqk", q[:, S - n:, h].double(), k[:, :, h // (Hq // H)].double())
        s = (s * scale).masked_fill_(~see, -float("inf"))
        lse[:, h, S - n:] = s.logsumexp(-1).float()
        want[:, h // (Hq // H)] += torch.exp(s - lse[:, h, S - n:, None].double()).sum(1)
    got = usp.attn_key_weights(q, k, lse, observe=observe)
    usp.usp_device_status()
    ds = D * U * scale * float(q.abs().max() * k.abs().max()) * D
    top = float(lse[:, :, S - n:].abs().max())
    bound = want * (2 * ds + 4 * U * top + 2 * n * Hq * U + 2.0 ** -20)
    assert ((got.double() - want).abs() <= bound + 1e-37).all()
    for _ in range(20):
        assert torch.equal(got, usp.attn_key_weights(q, k, lse, observe=observe))
    usp.usp_device_status()


@pytest.mark.parametrize("B,S,Hq,H,D,observe", [
    (32, 1280, 8, 8, 128, 64),   # one query tile per block of a run
    (32, 1100, 8, 8, 64, 64),
    (32, 1100, 24, 8, 64, 64),   # three
    (40, 700, 8, 8, 64, 300),    # three of one head
])
def test_key_weights_of_odd_tile_counts_over_many_items(B, S, Hq, H, D, observe):
    """An odd number of query tiles per block of keys: which group of softmax warps
    has a block's first tile changes from block to block and item to item."""
    check_weights_of_many_items(B, S, Hq, H, D, observe)


@pytest.mark.parametrize("B,S,Hq,H,D,observe", [
    (32, 1100, 8, 8, 128, 400),  # four query tiles: two slots of keys
    (32, 1025, 32, 8, 64, 100),  # four, of two heads
    (32, 1152, 24, 8, 128, 33),  # three
])
def test_key_weights_of_short_last_blocks_over_many_items(B, S, Hq, H, D, observe):
    """One key tile in a run's last block: the next item's keys go on in the other
    MMA warp's slot of the ring."""
    check_weights_of_many_items(B, S, Hq, H, D, observe)


@pytest.mark.parametrize("B,S,Hq,H,D,observe", [
    (32, 2100, 32, 8, 128, 64),  # two tiles of two heads
    (32, 2049, 16, 8, 64, 64),   # one
    (32, 2176, 16, 8, 128, 120), # two
])
def test_key_weights_of_shared_queries_over_many_items(B, S, Hq, H, D, observe):
    """The queries that a run's blocks shared make room for the next item's while
    the last products are under way, and the run ends with one key tile."""
    check_weights_of_many_items(B, S, Hq, H, D, observe)


@pytest.mark.parametrize("B,S,Hq,H,D,observe", [
    (16, 2100, 8, 8, 64, 0),     # nine blocks, the last of one tile
    (40, 1100, 8, 8, 128, 0),
    (64, 900, 16, 8, 64, 0),
    (160, 300, 24, 8, 128, 0),
])
def test_key_weights_of_all_queries_over_many_items(B, S, Hq, H, D, observe):
    """Many query tiles per block: the ring of their statistics goes round while one
    key tile's groups are behind and the other's block has begun."""
    check_weights_of_many_items(B, S, Hq, H, D, observe)


@pytest.mark.parametrize("causal,window,sink,observe", [(False, 0, 0, 64), (False, 3000, 9, 128),
                                                        (True, 0, 0, 4000), (False, 0, 0, 1)])
def test_key_weights_of_runs_match_the_cuda_core_kernel(causal, window, sink, observe):
    """Both kernels' errors are within the bound of the comparison with the
    oracle, so they differ by twice that at most."""
    dev = device()
    torch.manual_seed(observe)
    S, D = 12345, 128
    q = torch.randn(2, S, 4, D, device=dev).to(torch.bfloat16)
    k = torch.randn(2, S, 2, D, device=dev).to(torch.bfloat16)
    lse = torch.rand(2, 4, S, device=dev) + 10
    kw = dict(causal=causal, window=window, sink_tokens=sink, observe=observe)
    got, want = (usp.attn_key_weights(q, k, lse, flags=f, **kw) for f in (0, usp.FLAG_FORCE_SIMT))
    usp.usp_device_status()
    ds = D * U / np.sqrt(D) * float(q.abs().max() * k.abs().max()) * D
    bound = 2 * (2 * ds + 4 * U * 11 + 2 * observe * 4 * U + 2.0 ** -20)
    assert ((got - want).abs() <= bound * torch.maximum(got, want) + 1e-37).all()


def test_key_weights_captured_twice_with_their_own_workspaces():
    """Two graphs replayed at once on two streams, and with new inputs: cut
    into segments (a workspace), and with few queries."""
    dev = device()
    torch.manual_seed(5)
    q = torch.randn(1, 4096, 8, 128, device=dev).to(torch.bfloat16)
    k = torch.randn(1, 4096, 8, 128, device=dev).to(torch.bfloat16)
    _, lse = usp.attn_forward(q, k, k)
    for observe in (0, 64):
        graphs = []
        for _ in range(2):
            g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream(device=dev)
            with torch.cuda.graph(g, stream=s):
                w = usp.attn_key_weights(q, k, lse, observe=observe)
            graphs.append((g, s, w))
        for step in range(3):
            q.copy_(torch.randn_like(q))
            want = usp.attn_key_weights(q, k, lse, observe=observe)
            torch.cuda.synchronize()
            for g, s, w in graphs:
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            for _, _, w in graphs:
                assert torch.equal(w, want)
    usp.usp_device_status()


def test_key_weights_of_the_librarys_own_forward():
    """Every observed query spreads a weight of one per head of its group."""
    dev = device()
    g = gen(8)
    q = torch.randn(1, 2048, 8, 128, generator=g).to(torch.bfloat16).to(dev)
    k, v = (torch.randn(1, 2048, 2, 128, generator=g).to(torch.bfloat16).to(dev) for _ in "kv")
    kw = dict(causal=True, cp=4, layout="zigzag")
    _, lse = usp.attn_forward(q, k, v, **kw)
    w = usp.attn_key_weights(q, k, lse, **kw)
    assert torch.allclose(w.double().sum(-1), torch.full((1, 2), 4.0 * 2048, dtype=torch.float64, device=dev),
                          rtol=1e-5)
    w = usp.attn_key_weights(q, k, lse, observe=100, **kw)
    assert torch.allclose(w.double().sum(-1), torch.full((1, 2), 400.0, dtype=torch.float64, device=dev),
                          rtol=1e-5)


def test_key_weights_ignore_what_is_not_seen():
    """NaN and infinite rows that are not observed, or keys that no observed
    query sees, leave the other weights alone; LSE = -inf adds nothing."""
    dev = device()
    g = gen(11)
    q = torch.randn(1, 300, 2, 64, generator=g).to(torch.bfloat16).to(dev)
    k = torch.randn(1, 300, 1, 64, generator=g).to(torch.bfloat16).to(dev)
    _, lse = usp.attn_forward(q, k, k)
    want = usp.attn_key_weights(q, k, lse, observe=20)
    q2, lse2 = q.clone(), lse.clone()
    q2[:, 270:280] = float("nan")
    q2[:, :100] = float("inf")
    lse2[:, :, :280] = float("nan")
    assert torch.equal(usp.attn_key_weights(q2, k, lse2, observe=20), want)
    # causal: key 299 is seen by query 299 alone
    lse3 = lse.clone()
    lse3[:, :, 299] = -float("inf")
    w = usp.attn_key_weights(q, k, lse3, observe=20)
    assert (w[:, :, 299] == 0).all() and torch.isfinite(w).all()
    k2 = k.clone()
    k2[:, 299] = float("nan")
    w = usp.attn_key_weights(q, k2, lse3, observe=20)
    assert torch.isfinite(w[:, :, :299]).all()


@pytest.mark.parametrize("dtype,flags", [(torch.bfloat16, 0), (torch.bfloat16, 1),
                                         (torch.float32, 0)])
def test_key_weights_of_marked_queries_that_hold_nan(dtype, flags):
    """Queries whose LSE is -inf (padding) add nothing, whatever they hold, in
    tiles that the mask leaves whole as in others."""
    dev = device()
    g = gen(13)
    q = torch.randn(1, 1000, 2, 64, generator=g).to(dtype).to(dev)
    k = torch.randn(1, 1000, 1, 64, generator=g).to(dtype).to(dev)
    _, lse = usp.attn_forward(q, k, k)
    for a in (600, 990):
        lse[:, :, a:a + 10] = -float("inf")
    want = usp.attn_key_weights(q, k, lse, flags=flags)
    assert torch.isfinite(want).all()
    q[:, 600:605] = float("nan")
    q[:, 605:610] = float("inf")
    q[:, 990:1000] = float("nan")
    assert torch.equal(usp.attn_key_weights(q, k, lse, flags=flags), want)


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("cut", [None, [0, 300, 700]])
def test_key_weights_of_the_largest_window_and_sinks(cut, flags):
    dev = device()
    g = gen(14)
    shape = (700,) if cut else (1, 700)
    q = torch.randn(*shape, 2, 64, generator=g).to(torch.bfloat16).to(dev)
    k = torch.randn(*shape, 1, 64, generator=g).to(torch.bfloat16).to(dev)
    kw = dict(cu_seqlens=torch.tensor(cut, dtype=torch.int32, device=dev)) if cut else {}
    _, lse = usp.attn_forward(q, k, k, **kw)
    big = 2 ** 31 - 1
    want = usp.attn_key_weights(q, k, lse, flags=flags, **kw)
    for window, sink in ((big, 0), (big, big), (1, big)):
        got = usp.attn_key_weights(q, k, lse, flags=flags, window=window, sink_tokens=sink, **kw)
        # (a window makes tiles masked, whose sums are taken in another order)
        assert torch.allclose(got, want, rtol=700 * 2 * U)


@pytest.mark.parametrize("causal,window,observe", [(True, 0, 0), (False, 0, 0), (True, 90, 0),
                                                   (False, 0, 25)])
@pytest.mark.parametrize("path", ["bf16", "simt", "fp32"])
def test_key_weights_of_a_padded_batch(path, causal, window, observe):
    """Tokens before the first boundary and behind the last, whatever they hold, get
    0 and add nothing: the sequences' weights are those of the batch without them."""
    dev = device()
    dt = torch.float32 if path == "fp32" else torch.bfloat16
    cut, S, H = [30, 500, 500, 1101], 1400, 2
    g = gen(17)
    q = torch.randn(S, 4, 64, generator=g).to(dt).to(dev)
    k = torch.randn(S, H, 64, generator=g).to(dt).to(dev)
    kw = dict(causal=causal, window=window)
    flags = usp.FLAG_FORCE_SIMT if path == "simt" else 0
    mid = slice(cut[0], cut[-1])
    cu = torch.tensor(cut, dtype=torch.int32, device=dev)
    qm, km = q[mid].contiguous(), k[mid].contiguous()
    _, lm = usp.attn_forward(qm, km, km, cu_seqlens=cu - cut[0], **kw)
    want = usp.attn_key_weights(qm, km, lm, cu_seqlens=cu - cut[0], observe=observe, flags=flags, **kw)
    for junk in (0.5, float("nan")):
        lse = torch.full((4, S), junk, device=dev)
        lse[:, mid] = lm
        for t in (q, k):
            t[:cut[0]] = junk
            t[cut[-1]:] = junk
        got = usp.attn_key_weights(q, k, lse, cu_seqlens=cu, observe=observe, flags=flags, **kw)
        assert (got[:, :cut[0]] == 0).all() and (got[:, cut[-1]:] == 0).all()
        # the sums run over other tiles: n u in each, on up to 2 S positive terms
        assert torch.allclose(got[:, mid], want, rtol=2 * 2 * S * U, atol=0)
    usp.usp_device_status()


# ------------------------------------------------------------------------- evict

EVICT = [
    # B, C, H, D, lens, keep, recent, sink
    (1, 16, 1, 64, [16], 1, 0, 0),
    (1, 16, 1, 64, [16], 15, 3, 4),
    (3, 64, 2, 128, [0, 20, 64], 20, 5, 2),
    (2, 48, 3, 64, [47, 48], 48, 48, 0),       # nothing to evict
    (2, 128, 2, 128, [128, 100], 40, 36, 4),   # nothing to choose
    (2, 5008, 2, 128, [5001, 4000], 1000, 100, 4),
    (1, 70000, 2, 64, [69999], 3001, 0, 0),
    (2, 3008, 2, 128, [3000, 2999], 2998, 64, 4),
    (9, 96, 5, 64, [(11 * i) % 97 for i in range(9)], 33, 8, 1),
    (2, 600000, 1, 64, [600000, 500001], 2048, 512, 4),
]


@pytest.mark.parametrize("kind", ["random", "ties", "special"])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("B,C,H,D,lens,keep,recent,sink", EVICT)
def test_evict_matches_oracle(B, C, H, D, lens, keep, recent, sink, inplace, kind):
    dev = device()
    g = gen(C)
    c = usp.kv4_cache(B, C, H, D, device=dev, key_weight=True)
    for t in c[:4]:
        t.copy_(torch.randint(0, 255, t.shape, generator=g, dtype=torch.uint8))
    w = torch.rand(B, H, C, generator=g) ** 6
    if kind == "ties":
        w = (w * 3).round()
    if kind == "special":
        w = w - 0.3
        w[:, :, ::7] = -0.0
        w[:, :, 3::11] = 0.0
        w[:, :, 5::53] = float("inf")
        w[:, :, 6::53] = -float("inf")
        w[:, :, 7::61] = float("nan")
        w[:, :, 8::61] = -float("nan")
    for b, n in enumerate(lens):
        w[b, :, n:] = float("nan")  # behind the sequence: not looked at
    c.key_weight.copy_(w)
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    want = torch.from_numpy(kv4.kept_rows(w, lens, keep, recent, sink)).to(dev)
    before = snapshot(c)
    if inplace:
        dst, fill = c, before
        got, kept = usp.kv4_evict(c, keep, recent=recent, sink_tokens=sink)
        assert got is c
    else:
        dst = usp.kv4_cache(B, keep + 7, H, D, device=dev, key_weight=True)
        for t in dst[:4]:
            t.fill_(0x5A)
        dst.key_weight.fill_(-1)
        fill = snapshot(dst)
        got, kept = usp.kv4_evict(c, keep, recent=recent, sink_tokens=sink, out=dst)
        assert got is dst
        for x, y in zip(before, c[:6]):
            assert torch.equal(x, y) or (x.is_floating_point() and torch.equal(x.isnan(), y.isnan()))
    assert torch.equal(kept, want)
    assert dst.seq_lens.tolist() == [min(n, keep) for n in lens]
    for i, t in ((0, dst.k), (1, dst.k_scale), (2, dst.v), (3, dst.v_scale), (5, dst.key_weight)):
        expect = fill[i].clone()
        for b in range(B):
            n = min(lens[b], keep)
            if n:
                at = want[b, :, :n].long()
                src = before[i][b]
                if src.dim() == 3:
                    at = at[..., None].expand(-1, -1, src.shape[-1])
                expect[b, :, :n] = src.gather(1, at)
        if inplace:  # rows that held keys before are free now
            for b in range(B):
                n = min(lens[b], keep)
                if t.dtype == torch.float32:
                    assert torch.equal(t[b, :, :n].view(torch.int32), expect[b, :, :n].view(torch.int32))
                else:
                    assert torch.equal(t[b, :, :n], expect[b, :, :n])
        elif t.dtype == torch.float32:
            assert torch.equal(t.view(torch.int32), expect.view(torch.int32))
        else:
            assert torch.equal(t, expect)


def test_evict_into_a_cache_without_weights():
    dev = device()
    c = random_cache(dev, 1, 64, 2, 64, [64])
    dst = usp.kv4_cache(1, 32, 2, 64, device=dev)
    _, kept = usp.kv4_evict(c, 20, recent=3, out=dst)
    assert torch.equal(kept.cpu(), torch.from_numpy(kv4.kept_rows(c.key_weight.cpu(), [64], 20, 3, 0)))
    assert dst.seq_lens.tolist() == [20]


# --------------------------------------------------- a run of them, as it is used

def serve(dev, c, steps, q, k, v, workspace=None):
    outs = []
    for t in range(steps):
        usp.kv4_append(c, k[:, t:t + 1].contiguous(), v[:, t:t + 1].contiguous())
        outs.append(usp.attn_decode_kv4(q[:, t:t + 1].contiguous(), c, accumulate=True,
                                        workspace=workspace))
    return outs


def test_prompt_eviction_and_decoding_together():
    """A prompt through the ring forward, its keys' weights, the cache filled
    with them, brought down to its budget, then decoding steps that go on
    weighing and one more eviction; the cache's own contents through the
    oracle at each step."""
    dev = device()
    g = gen(21)
    B, S, Hq, H, D, steps = 2, 512, 8, 2, 128, 5
    q = torch.randn(B, S + steps, Hq, D, generator=g).to(torch.bfloat16).to(dev)
    k, v = (torch.randn(B, S + steps, H, D, generator=g).to(torch.bfloat16).to(dev) for _ in "kv")
    qs, ks, vs = (x[:, :S].contiguous() for x in (q, k, v))
    _, lse = usp.attn_forward(qs, ks, vs)
    w = usp.attn_key_weights(qs, ks, lse, observe=64)
    c = usp.kv4_cache(B, S + 64, H, D, device=dev, key_weight=True)
    usp.kv4_append(c, ks, vs, key_weight=w)
    assert torch.equal(c.key_weight[:, :, :S], w)
    kr, vr = usp.kv4_read(c, S)
    # half a step of a block is max / 14, and the scale's own rounding cuts at most 2^-4
    err = (kr.float() - ks.float()).abs().amax() / ks.float().abs().amax()
    assert float(err) < 1 / 14 + 2.0 ** -4
    small = usp.kv4_cache(B, 160, H, D, device=dev, key_weight=True)
    c, kept = usp.kv4_evict(c, 128, recent=32, sink_tokens=4, out=small)
    assert c.seq_lens.tolist() == [128, 128]
    for t in range(steps):
        n = 128 + t + 1
        old = c.key_weight.clone()
        usp.kv4_append(c, k[:, S + t:S + t + 1].contiguous(), v[:, S + t:S + t + 1].contiguous())
        old[:, :, n - 1] = 0
        qt = q[:, S + t:S + t + 1].contiguous()
        out, l = usp.attn_decode_kv4(qt, c, accumulate=True)
        check_decode(c, qt.cpu(), out, l, c.key_weight, old, [n, n], True, 0, 0)
    before = c.key_weight.clone()
    c, kept = usp.kv4_evict(c, 100, recent=16, sink_tokens=4)
    want = torch.from_numpy(kv4.kept_rows(before.cpu(), [133, 133], 100, 16, 4))
    assert torch.equal(kept.cpu(), want) and c.seq_lens.tolist() == [100, 100]
    usp.usp_device_status()


@pytest.mark.parametrize("layout,cp,packed", [("zigzag", 4, False), ("stripe", 2, False),
                                              ("zigzag", 2, True)])
def test_ring_prompt_into_the_cache_with_its_weights(layout, cp, packed):
    """The weights of a ring's prompt are restored to natural order like its keys,
    and are then those of the same prompt in natural order (sums over other tiles:
    n u in each); the cache's rows and weights belong together."""
    dev = device()
    g = gen(22)
    S, Hq, H, D = 776, 4, 2, 64
    lead = () if packed else (2,)
    q = torch.randn(*lead, S, Hq, D, generator=g).to(torch.bfloat16).to(dev)
    k, v = (torch.randn(*lead, S, H, D, generator=g).to(torch.bfloat16).to(dev) for _ in "kv")
    kw = dict(cu_seqlens=torch.tensor([0, 300, S], dtype=torch.int32, device=dev)) if packed else {}
    _, lse = usp.attn_forward(q, k, v, **kw)
    want = usp.attn_key_weights(q, k, lse, **kw)
    qp, kp, vp = (usp.permute(t, "extract", layout, cp) for t in (q, k, v))
    _, lp = usp.attn_forward(qp, kp, vp, cp=cp, layout=layout, **kw)
    w = usp.attn_key_weights(qp, kp, lp, cp=cp, layout=layout, **kw)
    nat = usp.permute(w.view(-1, S, 1, 1), "restore", layout, cp).view_as(w)
    back = usp.permute(nat.view(-1, S, 1, 1), "extract", layout, cp).view_as(w)
    assert torch.equal(back, w)
    index = layouts.restore(np.arange(S), layout, cp, axis=0)
    assert torch.equal(nat, w[..., torch.from_numpy(index).to(dev)])
    # the LSEs, rounded sums of up to S terms near 10, may differ too
    assert torch.allclose(nat, want, rtol=4 * S * U + 2 * 10 * U)
    c = usp.kv4_cache(2, S, H, D, device=dev, key_weight=True)
    usp.kv4_append(c, usp.permute(kp, "restore", layout, cp), usp.permute(vp, "restore", layout, cp),
                   key_weight=nat, **kw)
    for b, (at, n) in enumerate([(0, 300), (300, S - 300)] if packed else [(0, S)] * 2):
        one = nat[:, at:at + n] if packed else nat[b]
        assert torch.equal(c.key_weight[b, :, :n], one)
    usp.usp_device_status()


def test_evict_in_place_captured_and_twice():
    """An eviction in place, captured: each replay evicts what the cache holds
    then; a second one right behind it finds nothing to do."""
    dev = device()
    lens = [900, 500, 64]
    c = random_cache(dev, 3, 912, 2, 64, lens, seed=21)
    start = snapshot(c)
    eager = random_cache(dev, 3, 912, 2, 64, lens, seed=21)
    _, kept = usp.kv4_evict(eager, 200, recent=20, sink_tokens=3)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        _, k1 = usp.kv4_evict(c, 200, recent=20, sink_tokens=3)
        _, k2 = usp.kv4_evict(c, 200, recent=20, sink_tokens=3)
    for _ in range(2):
        for t, x in zip(c[:6], start):
            t.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(k1, kept) and c.seq_lens.tolist() == [200, 200, 64]
        for b, n in enumerate((200, 200, 64)):
            want = torch.arange(200, device=dev, dtype=torch.int32)
            want[n:] = -1
            assert (k2[b] == want).all()
        for x, y in zip(c[:6], eager[:6]):
            assert torch.equal(x, y)


def test_captured_step_grows_the_cache_on_replay():
    """An append and a decode captured once: every replay finds the longer
    sequence, and gives what the calls give one by one."""
    dev = device()
    g = gen(31)
    B, Hq, H, D, steps = 2, 8, 2, 128, 4
    k, v = (torch.randn(B, 60 + steps, H, D, generator=g).to(torch.bfloat16).to(dev) for _ in "kv")
    q = torch.randn(B, steps, Hq, D, generator=g).to(torch.bfloat16).to(dev)

    def fresh():
        c = usp.kv4_cache(B, 128, H, D, device=dev, key_weight=True)
        usp.kv4_append(c, k[:, :60].contiguous(), v[:, :60].contiguous())
        return c

    eager = fresh()
    want = serve(dev, eager, steps, q, k[:, 60:], v[:, 60:])
    c = fresh()
    static = [q[:, :1].clone(), k[:, 60:61].clone(), v[:, 60:61].clone()]
    ws = torch.empty(usp.usp_attn_decode_kv4_workspace_size(B, 1, 128, Hq, H, D, True),
                     dtype=torch.uint8, device=dev)
    s = torch.cuda.Stream(device=dev)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # warm-up on another cache
        d = fresh()
        usp.kv4_append(d, static[1], static[2])
        usp.attn_decode_kv4(static[0], d, accumulate=True, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        usp.kv4_append(c, static[1], static[2])
        out, lse = usp.attn_decode_kv4(static[0], c, accumulate=True, workspace=ws)
    for t in range(steps):
        for dst, src in zip(static, (q[:, t:t + 1], k[:, 60 + t:61 + t], v[:, 60 + t:61 + t])):
            dst.copy_(src)
        graph.replay()
        assert torch.equal(out, want[t][0]) and torch.equal(lse, want[t][1]), t
    for x, y in zip(c[:6], eager[:6]):
        assert torch.equal(x, y)
    usp.usp_device_status()


def test_explicit_stream_does_not_share_memory_with_the_current_one():
    """What a call allocates belongs to the stream it runs on: memory that work
    still queued on the current stream writes is not handed to it."""
    dev = device()
    c = random_cache(dev, 2, 512, 4, 128, [500, 300], seed=8)
    q = torch.randn(2, 1, 16, 128, generator=gen(8)).to(torch.bfloat16).to(dev)
    want, wl = usp.attn_decode_kv4(q, c)
    k, v = usp.kv4_read(c, 500)
    side = torch.cuda.Stream(device=dev)
    torch.cuda.synchronize()
    for _ in range(3):
        for stream in (side, side.cuda_stream):
            x = [torch.empty_like(t) for t in (want, wl, k, v)]
            torch.cuda._sleep(20_000_000)  # some 10 ms
            for t in x:
                t.fill_(7)
            del x, t
            out, lse = usp.attn_decode_kv4(q, c, stream=stream)
            k2, v2 = usp.kv4_read(c, 500, stream=stream)
            side.synchronize()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(lse, wl)
            assert torch.equal(k2, k) and torch.equal(v2, v)
            del out, lse, k2, v2


def test_two_streams_with_their_own_workspaces():
    dev = device()
    c = random_cache(dev, 2, 2048, 4, 128, [2000, 1500], seed=7)
    q = torch.randn(2, 1, 16, 128, generator=gen(7)).to(torch.bfloat16).to(dev)
    want = usp.attn_decode_kv4(q, c)
    streams = [torch.cuda.Stream(device=dev) for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(usp.attn_decode_kv4(q, c))
    explicit = usp.attn_decode_kv4(q, c, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    for o, l in got + [explicit]:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
