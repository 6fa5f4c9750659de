"""The attention to the paged 8-bit cache, every element of O within the tolerance of its own
row (tests/_kv8.py): the bound follows the values that the row sees, not those of pages
that no sequence has. And batches of more sequences than the tensor-core kernel's division
of the work takes at once (32)."""
import numpy as np
import pytest
import torch

import sequence_long_context_gb300 as usp
from oracle import fp8
from tests import _kv8
from tests._gpu import device
from tests.test_gpu_kv8 import ATTN, gen, host, i32, random_cache

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def queries(dev, lead, H, D, seed):
    return torch.randn(*lead, H, D, generator=gen(seed)).to(BF).to(dev)


def spread(B, top, step):
    return [(step * b) % (top + 1) for b in range(B)]


MANY = [
    # B, T, cap, H, G, D, page, lens, causal, window, sink: more than 64 rows per KV head
    (33, 20, 384, 2, 4, 64, 32, spread(33, 384, 37), True, 0, 0),
    (70, 33, 256, 1, 4, 128, 64, spread(70, 256, 91), True, 0, 0),
    (64, 17, 384, 3, 4, 128, 128, [0] * 63 + [384], True, 0, 0),      # the last one alone has keys
    (40, 150, 512, 1, 8, 64, 128, spread(40, 512, 201), False, 0, 0),  # five units each
    (36, 130, 640, 2, 10, 128, 32, spread(36, 640, 111), True, 100, 3),
]


@pytest.mark.parametrize("B,T,cap,H,G,D,page,lens,causal,window,sink", ATTN + MANY)
def test_every_element(B, T, cap, H, G, D, page, lens, causal, window, sink):
    dev = device()
    c = random_cache(dev, B, cap, H, D, page, lens, seed=T)
    q = queries(dev, (B, T), H * G, D, T + 1)
    out, lse = usp.attn_kv8(q, c, causal=causal, window=window, sink_tokens=sink)
    _kv8.check(q, c, out, lse, causal, window, sink)
    again = usp.attn_kv8(q, c, causal=causal, window=window, sink_tokens=sink)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    usp.usp_device_status()


def cuts(new, first=0):
    return np.concatenate([[first], first + np.cumsum(new)]).tolist()


PACKED = [
    # new tokens of the sequences, cached lengths, heads, capacity, what else
    ([1, 1, 3, 0, 25], [40, 1, 100, 64, 29], 2, 320, dict()),
    ([1, 1, 136, 1, 159], [70, 0, 250, 129, 300], 2, 320, dict()),
    ([40, 1, 0, 49, 1], [200, 33, 10, 49, 320], 2, 320, dict(window=40, sink_tokens=2)),
    ([1, 1, 1, 1, 1], [320, 1, 0, 63, 64], 2, 320, dict(causal=False)),
    ([1, 1, 1, 197, 300], [320, 1, 150, 197, 320], 12, 320, dict()),
    ([1, 1, 1, 197, 300], [8000, 5000, 3000, 2500, 1800], 8, 8192, dict()),
    # 33 to 70 sequences: none, single tokens, and more than 1024 rows behind the 32nd
    ([1] * 20 + [0] * 12 + [40, 1, 300, 0, 2], spread(37, 512, 73), 2, 512, dict()),
    ([0] * 33 + [70, 0, 1, 290], spread(33, 512, 73) + [70, 0, 500, 512], 1, 512, dict(window=60, sink_tokens=1)),
    ([b % 5 for b in range(69)] + [290], spread(69, 384, 91) + [384], 2, 384, dict(causal=False)),
    ([1] * 64, spread(64, 384, 91), 1, 384, dict()),
]


@pytest.mark.parametrize("new,lens,H,cap,kw", PACKED)
@pytest.mark.parametrize("hint", [False, True])
def test_every_element_of_a_packed_batch(new, lens, H, cap, kw, hint):
    dev = device()
    cut = cuts(new, 2)
    T = cut[-1] + 3
    c = random_cache(dev, len(new), cap, H, 128, 32, lens, seed=T)
    q = queries(dev, (T,), H * 4, 128, T)
    out, lse = usp.attn_kv8(q, c, cu_seqlens=i32(cut, dev), max_new=max(new) if hint else 0, **kw)
    _kv8.check(q, c, out, lse, kw.get("causal", True), kw.get("window", 0), kw.get("sink_tokens", 0), cut=cut)
    for s in (slice(0, cut[0]), slice(cut[-1], T)):  # padding
        assert not out[s].any() and torch.isneginf(lse[s]).all()
    usp.usp_device_status()


@pytest.mark.parametrize("T", [1, 40])
def test_every_element_where_rows_have_no_page(T):
    dev = device()
    c = random_cache(dev, 3, 512, 2, 128, 64, [500, 300, 64], seed=3)
    c.page_table[0, 0] = -1
    c.page_table[0, 3:5] = 1 << 30
    c.page_table[1, :] = -7
    q = queries(dev, (3, T), 4, 128, 8)
    out, lse = usp.attn_kv8(q, c)
    _kv8.check(q, c, out, lse)
    assert torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("exps", [(-34, 46), (-34, -33), (40, 46), (-3, 9)])
def test_every_element_beside_other_exponents(T, exps):
    dev = device()
    c = random_cache(dev, 1, 512, 1, 128, 64, [512], seed=3, exps=exps)
    c.k_exp.copy_(torch.randint(-9, -3, c.k_exp.shape, generator=gen(1)).to(torch.int8))
    q = queries(dev, (1, T), 2, 128, 8)
    out, lse = usp.attn_kv8(q, c)
    _kv8.check(q, c, out, lse)


@pytest.mark.parametrize("T", [1, 33, 130])
def test_every_element_of_small_keys_beside_a_sink(T):
    """A first key that takes nearly all the attention, with a value of 0, and 8191 keys of
    2^-24 of its weight."""
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
    _kv8.check(q, c, out, lse, causal=False)


@pytest.mark.parametrize("T", [1, 33])
@pytest.mark.parametrize("scale", [1e-30, 0.3, 4.0])
def test_every_element_at_other_scales(T, scale):
    dev = device()
    c = random_cache(dev, 2, 128, 1, 64, 64, [128, 50], seed=5)
    q = torch.randn(2, T, 4, 64, generator=gen(9))
    q[0, 0, 0] = 0
    q[0, 0, 1] *= 1e-30
    q[0, 0, 2] *= 1e20 if scale < 1e-9 else 1
    q = q.to(BF).to(dev)
    out, lse = usp.attn_kv8(q, c, softmax_scale=scale)
    _kv8.check(q, c, out, lse, scale=scale)
