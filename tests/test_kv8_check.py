"""What the comparison of the 8-bit cache's attention (tests/_kv8.py) lets through: the
oracle's own values rounded to the outputs' types, and no value that an error of the
kernel's parts would give."""
import numpy as np
import pytest
import torch

from oracle import attention, kv8
from tests import _kv8
from tests.test_gpu_kv8 import ATTN, gen, random_cache

BF = torch.bfloat16


def bf16(x):
    return torch.from_numpy(x).to(BF).double().numpy()


def outputs(q, k, v, there, causal, window, sink):
    O, L = kv8.attend(q, k, v, there, q.shape[-1] ** -0.5, causal, window, sink)
    return bf16(O), np.float32(L).astype(np.float64)


def heaviest(q, k, there, causal, window, sink):
    """The block of 32 rows with the most attention of all queries to KV head 0."""
    n, Hq, D = q.shape
    L, H = k.shape[:2]
    i = L - n + np.arange(n)
    vis = attention.visibility(i, np.arange(L), causal, window, sink) & (i >= 0)[:, None] & there
    s = np.where(vis, q[:, 0] @ k[:, 0].T * D ** -0.5, -np.inf)[vis.any(1)]
    p = np.exp(s - s.max(1, keepdims=True))
    p = (p / p.sum(1, keepdims=True)).sum(0)
    return int(np.argmax(np.add.reduceat(p, np.arange(0, L, 32)))) * 32


@pytest.mark.parametrize("B,T,cap,H,G,D,page,lens,causal,window,sink", ATTN)
def test_the_check_sees_what_it_should(B, T, cap, H, G, D, page, lens, causal, window, sink):
    c = random_cache("cpu", B, cap, H, D, page, lens, seed=T)
    h = _kv8.Host(c)
    q = torch.randn(B, T, H * G, D, generator=gen(T + 1)).to(BF).double().numpy()
    b = int(np.argmax(lens))
    k, v, there, _, _ = h.kv(b)
    kw = dict(causal=causal, window=window, sink=sink)
    wrong = lambda out, lse: _kv8.faults(h, b, q[b], out, lse, D ** -0.5, **kw)  # noqa: E731
    O, L = outputs(q[b], k, v, there, **kw)
    assert wrong(O, L) is None
    assert wrong(0 * O, L) and wrong(bf16(1.1 * O), L) and wrong(bf16(O * 0.97), L)
    assert wrong(np.roll(O, 1, -1), L)  # channels
    at = heaviest(q[b], k, there, **kw)
    for factor in (0.0, 2.0):  # a block of V left out, or of an exponent too many
        w = v.copy()
        w[at:at + 32] *= factor
        assert wrong(outputs(q[b], k, w, there, **kw)[0], L), factor
    w = k.copy()
    w[at:at + 32] *= 2.0
    assert wrong(*outputs(q[b], w, v, there, **kw))
    assert wrong(O, L + 0.01)
    if H * G > 1:
        assert wrong(np.roll(O, 1, 1), L)  # heads
    none = ~np.isfinite(L)
    if none.any():
        assert wrong(np.where(none[..., None], 1.0, O), L)
        assert wrong(O, np.where(none, 0.0, L))
