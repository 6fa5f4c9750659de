"""Pins of the 4-bit cache's oracle to something other than itself: closed
forms, torch's float8 conversion, the attention oracle's own decode step,
finite sums, sorting."""
import numpy as np
import pytest
import torch

from oracle import attention, decode, fp8, kv4


def test_codes_closed_forms():
    x = np.zeros((1, 64))
    x[0, :8] = [7, -7, 3.5, 2.5, 1.5, 0.5, -0.5, 0.49]  # max 7: scale exactly 1
    codes, sb = kv4.quantize(x, 1.0)
    assert sb[0, 0] == 0x38 and sb[0, 1] == 0  # e4m3(1) and 0
    v = kv4.values(codes, sb, 1.0)
    # halves go to the even integer
    assert v[0, :8].tolist() == [7, -7, 4, 2, 2, 0, 0, 0]
    assert (v[0, 8:] == 0).all()
    # the first channel is the low nibble of the first byte
    assert codes[0, 0] == (7 + 8) + 16 * (-7 + 8)
    assert (codes[0, 16:] == 0x88).all()


def test_special_values():
    x = np.ones((4, 32))
    x[0, 3] = np.nan
    x[1, 3] = np.inf
    x[2, 3] = -np.inf
    x[3] = 1e-9
    v = kv4.values(*kv4.quantize(x, 1.0), 1.0)
    assert v[0, 3] == 0 and np.allclose(v[0, 4], 1, rtol=1 / 16)
    assert v[1, 3] == 7 * 448 and v[1, 4] == 0
    assert v[2, 3] == -7 * 448
    assert (v[3] == 0).all()  # below the smallest scale


@pytest.mark.parametrize("descale", [1.0, 0.25, 0.37])
def test_matches_torch_arithmetic_and_error_bound(descale):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(257, 128, generator=g) * torch.logspace(-1, 1, 128)
    inv = torch.tensor(1.0, dtype=torch.float32) / torch.tensor(descale, dtype=torch.float32)
    y = (x * inv).unflatten(-1, (-1, 32))
    s = (y.abs().amax(-1) / torch.tensor(7.0)).clamp(max=448).to(torch.float8_e4m3fn)
    codes, sb = kv4.quantize(x, descale)
    assert np.array_equal(s.view(torch.uint8).numpy(), sb)
    c = (y / s.float()[..., None]).round().clamp(-7, 7)
    want = (c * s.float()[..., None]).flatten(-2).double() * float(np.float32(descale))
    got = kv4.values(codes, sb, descale)
    assert np.abs(got - want.numpy()).max() == 0
    # half a step, or what the clamp cuts off where s rounded down by 2^-4
    step = np.repeat(fp8.e4m3_decode(sb), 32, axis=-1) * descale
    assert (np.abs(got - x.double().numpy()) <= 0.5 * step * (1 + 1e-6)).mean() > 0.97
    assert (np.abs(got - x.double().numpy()) <= 1.0 * step).all()


@pytest.mark.parametrize("causal,window,sink", [(True, 0, 0), (False, 0, 0), (True, 5, 2)])
def test_decode_is_the_attention_oracle_on_each_prefix(causal, window, sink):
    rng = np.random.default_rng(1)
    B, Tq, Hq, H, C, D = 3, 2, 4, 2, 16, 64
    q = rng.normal(size=(B, Tq, Hq, D))
    k, v = rng.normal(size=(2, B, H, C, D))
    lens = [16, 9, 1]
    O, L, W = kv4.decode(q, k, v, lens, 0.125, causal, window, sink)
    for b, n in enumerate(lens):
        kk, vv = k[b:b + 1, :, :n].swapaxes(1, 2), v[b:b + 1, :, :n].swapaxes(1, 2)
        if n >= Tq and window == 0:
            o, l = decode.decode_fwd(q[b:b + 1], kk, vv, 0.125, causal)
            assert np.allclose(O[b], o[0]) and np.allclose(L[b], l[0])
        # every visible query spreads a weight of one per head
        assert np.isclose(W[b].sum(), np.isfinite(L[b]).sum())
        assert (W[b, :, n:] == 0).all()
    # one cached token, two queries: the first has no position
    assert np.isinf(L[2, 0]).all() and (O[2, 0] == 0).all()
    assert np.allclose(O[2, 1, 0], v[2, 0, 0])


@pytest.mark.parametrize("causal,window,sink,observe", [
    (True, 0, 0, 0), (False, 0, 0, 0), (True, 4, 1, 0), (True, 0, 0, 3)])
def test_key_weights_are_column_sums(causal, window, sink, observe):
    rng = np.random.default_rng(2)
    B, S, Hq, H, D = 2, 11, 4, 2, 64
    q, k = rng.normal(size=(B, S, Hq, D)), rng.normal(size=(B, S, H, D))
    _, lse = attention.attn_fwd(q, k, k, 0.2, causal, window, sink)
    w = kv4.key_weights(q, k, lse, 0.2, causal, window, sink, None, observe)
    n = observe or S
    assert np.allclose(w.sum(-1), n * Hq // H)
    # torch: softmax of the masked scores, summed over queries and the group
    s = torch.einsum("bihd,bjhd->bhij", torch.tensor(q), torch.tensor(k).repeat_interleave(Hq // H, 2)) * 0.2
    i, j = torch.arange(S)[:, None], torch.arange(S)[None]
    m = (j <= i) if causal else torch.ones(S, S, dtype=torch.bool)
    if window:
        m = m & ((i - j < window) | (j < sink))
    p = torch.softmax(s.masked_fill(~m, -torch.inf), -1)[:, :, S - n:]
    want = p.sum(2).unflatten(1, (H, Hq // H)).sum(2)
    assert np.allclose(w, want.numpy())


def test_key_weights_packed_is_each_sequence_alone():
    rng = np.random.default_rng(4)
    q, k = rng.normal(size=(12, 2, 64)), rng.normal(size=(12, 1, 64))
    cu = [0, 5, 5, 12]
    _, lse = attention.attn_fwd(q, k, k, 0.2, True, cu_seqlens=np.array(cu))
    w = kv4.key_weights(q, k, lse, 0.2, cu_seqlens=cu)
    assert np.isclose(w[0, :5].sum(), 10) and np.isclose(w[0, 5:].sum(), 14)


def test_kept_rows_by_sorting():
    rng = np.random.default_rng(5)
    w = rng.integers(0, 4, size=(2, 3, 40)).astype(float)
    got = kv4.kept_rows(w, [40, 7], 10, 3, 2)
    for h in range(3):
        order = np.argsort(-w[0, h, 2:37], kind="stable")[:5] + 2
        assert got[0, h].tolist() == sorted([0, 1, 37, 38, 39] + order.tolist())
        assert got[1, h].tolist() == list(range(7)) + [-1] * 3
    w[0, 0, 20] = np.nan
    w[0, 0, 21] = np.inf
    assert {20, 21} <= set(kv4.kept_rows(w, [40, 7], 10, 3, 2)[0, 0].tolist())
    assert 20 in kv4.kept_rows(w, [40, 7], 6, 3, 2)[0, 0] and 21 not in kv4.kept_rows(w, [40, 7], 6, 3, 2)[0, 0]
