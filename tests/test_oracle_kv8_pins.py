"""The oracle of the rotation and the paged 8-bit cache against something other than
itself: complex multiplication, torch's conversion, closed forms, fp64 SDPA."""
import math

import numpy as np
import pytest
import torch

from oracle import fp8, kv8


def table(n, R, base=100.0):
    a = np.arange(n)[:, None] * base ** (-2.0 * np.arange(R // 2) / R)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32), a


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("R", [16, 48, 64])
def test_rotation_is_complex_multiplication(R, inter):
    rng = np.random.default_rng(R)
    x = rng.standard_normal((7, 3, 64)).astype(np.float32)
    tab, ang = table(50, R)
    pos = np.array([0, 1, 2, 9, 30, 49, 49])
    y = kv8.rotate(x, pos, tab, inter).astype(np.float64)
    i = np.arange(R // 2)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
    z = (x[..., ia] + 1j * x[..., ib]) * np.exp(1j * ang[pos])[:, None]
    # each of three roundings and the table's: 4 half steps of |a| + |b|
    tol = 4 * 2.0 ** -24 * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    assert (np.abs(y[..., ia] - z.real) <= tol).all() and (np.abs(y[..., ib] - z.imag) <= tol).all()
    assert np.array_equal(y[..., R:], x[..., R:])
    back = kv8.rotate(y.astype(np.float32), pos, tab, inter, inverse=True)
    assert np.abs(back - x).max() < 1e-5


def test_rotation_depends_on_distance_alone():
    rng = np.random.default_rng(3)
    tab, _ = table(200, 64)
    q, k = rng.standard_normal((2, 1, 1, 64)).astype(np.float32)
    dots = [float((kv8.rotate(q, [p + 13], tab) * kv8.rotate(k, [p], tab)).sum()) for p in (0, 5, 150)]
    assert max(dots) - min(dots) < 1e-4


@pytest.mark.parametrize("amax,e", [(0.0, -40), (448.0, 0), (448.0001, 1), (447.0, 0), (224.0, -1),
                                    (224.5, 0), (3.5 * 2.0 ** -47, -40), (448 * 2.0 ** 40, 40),
                                    (math.inf, 40), (1e-30, -40)])
def test_exponents(amax, e):
    assert kv8.exponent(amax) == e


def test_codes_are_torchs():
    x = (np.random.default_rng(0).standard_normal(5000) * 100).astype(np.float32)
    want = torch.tensor(x / 8).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv8.encode(x, 3), want)
    assert kv8.encode([np.nan, np.inf, -np.inf], 0).tolist() == [0, 0x7E, 0xFE]


def empty(pages=4, H=2, ps=32, D=64):
    return np.zeros((pages, H, ps, D), np.uint8), np.zeros((pages, H, ps // 32), np.int8)


def test_append_reads_back_within_half_a_step():
    codes, exps = empty(ps=64)
    x = np.random.default_rng(1).standard_normal((100, 2, 64)) * np.logspace(-1, 1, 100)[:, None, None]
    kv8.append(codes, exps, [2, 0], 0, x)
    got, there = kv8.values(codes, exps, [2, 0], 100)
    top = np.abs(np.pad(x, ((0, 28), (0, 0), (0, 0))).reshape(4, 32, 2, 64)).max((1, 3))
    floor = np.repeat(2.0 ** np.ceil(np.log2(top / 448)) * 2.0 ** -10, 32, 0)[:100]
    assert there.all() and (np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), floor[..., None])).all()
    # an entry that names no page: nothing there
    assert not kv8.values(codes, exps, [2, 7], 100)[1][64:].any()


def test_append_in_parts_differs_by_subnormals_alone():
    x = np.random.default_rng(2).standard_normal((40, 2, 64))
    x[20:] *= 50
    one, two = empty(), empty()
    kv8.append(*one, [1, 3], 0, x)
    for t in range(40):
        kv8.append(*two, [1, 3], t, x[t:t + 1])
    assert np.array_equal(one[1], two[1])
    a, b = kv8.values(*one, [1, 3], 40)[0], kv8.values(*two, [1, 3], 40)[0]
    e = np.repeat(one[1][[1, 3], :, 0].astype(float), 32, 0)[:40, :, None]
    assert (np.abs(a - b) <= 2.0 ** (e - 9)).all()
    assert np.array_equal(np.where(np.abs(a) >= 2.0 ** (e - 6), a, 0)[20:], np.where(np.abs(b) >= 2.0 ** (e - 6), b, 0)[20:])


def test_append_drops_what_finds_no_room():
    codes, exps = empty(pages=2)
    codes[:] = 9
    kv8.append(codes, exps, [-1, 1], 20, np.ones((60, 2, 64)))
    assert (codes[0] == 9).all() and (codes[1] != 9).all()


@pytest.mark.parametrize("causal,n,L", [(True, 5, 70), (False, 3, 33), (True, 4, 4)])
def test_attend_is_sdpa(causal, n, L):
    g = torch.Generator().manual_seed(n)
    q = torch.randn(n, 4, 64, generator=g, dtype=torch.float64)
    k, v = (torch.randn(L, 2, 64, generator=g, dtype=torch.float64) for _ in "kv")
    mask = torch.ones(n, L, dtype=torch.bool).tril(L - n) if causal else torch.ones(n, L, dtype=torch.bool)
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.transpose(0, 1).repeat_interleave(2, 0),
        v.transpose(0, 1).repeat_interleave(2, 0), attn_mask=mask).transpose(0, 1)
    O, lse = kv8.attend(q.numpy(), k.numpy(), v.numpy(), np.ones(L, bool), 64 ** -0.5, causal)
    assert np.abs(O - want.numpy()).max() < 1e-12 and np.isfinite(lse).all()


def test_attend_hides_rows_without_a_page_and_early_tokens():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((6, 2, 64)), rng.standard_normal((4, 1, 64)), rng.standard_normal((4, 1, 64))
    there = np.array([True, False, True, True])
    O, lse = kv8.attend(q, k, v, there, 0.125)
    assert not O[:2].any() and np.isneginf(lse[:2]).all()       # i < 0
    assert np.allclose(O[2], v[0]) and np.allclose(lse[2], 0.125 * q[2] @ k[0, 0])
    sub = kv8.attend(q[3:4], k[:1], v[:1], there[:1], 0.125)
    assert np.allclose(O[3], sub[0][0])                          # key 1 has no page


def test_planted_mistakes_are_seen():
    tab, _ = table(20, 64)
    x = np.random.default_rng(7).standard_normal((2, 1, 64)).astype(np.float32)
    assert not np.allclose(kv8.rotate(x, [3, 4], tab), kv8.rotate(x, [4, 5], tab))
    assert not np.allclose(kv8.rotate(x, [3, 4], tab), kv8.rotate(x, [3, 4], tab, inverse=True))
    assert not np.array_equal(fp8.e4m3_decode(kv8.encode([3.3], 0)), fp8.e4m3_decode(kv8.encode([3.3], 9)))
