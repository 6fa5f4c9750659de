"""The attention to the paged 8-bit cache against the oracle, sequence by sequence.

Tolerances (u = 2^-24, n keys, codes c of the block's exponent e_v), for every element:
  |ds| <= D u max_ij sum_d |q_d k_d| scale   (fp32 accumulation of exact products)
          + 2^-22 (1 + max|s|)               (scaling, maximum, exp2's argument and result)
  LSE:    |ds| + n u + 4 u |LSE|
  O:      A (2^-11 + 2 |ds| + 2 n u) + 2^-32 2^E sum_j |c_j| + 2^-8 |O|
with A = sum_j P_j |v_j|, and j the keys that the row sees, E the largest exponent of V among
them. P is rounded to fp16, by 2^-11 of it or, where it is subnormal, by 2^-25. It stands
against a reference m, with p = 2^(s + e_v - m): some key k has s_k + e_k >= m + 7, so the
row's sum of 2^(s - m) is at least 2^(7 - e_k) >= 2^(7 - E), and an error of 2^-25 |c_j| in O's
numerator is at most 2^-32 2^E |c_j| in O. That holds for each partial with its own m and
keys, so for their sum. O is rounded to bf16."""
from __future__ import annotations

import numpy as np

from oracle import attention, fp8, kv8

U = 2.0 ** -24


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Host:
    """A cache's arrays on the host."""

    def __init__(self, c):
        self.kc, self.ke, self.vc, self.ve = (t.cpu().numpy().copy() for t in c[:4])
        self.table, self.lens = c.page_table.cpu().numpy(), c.seq_lens.cpu().numpy()
        self.page = c.k.shape[2]

    def rows(self, b):
        return min(max(int(self.lens[b]), 0), self.table.shape[1] * self.page)

    def kv(self, b):
        """(k, v [L, H, D], which rows have a page, |codes of v|, exponents of v [L, H])."""
        n, tab = self.rows(b), self.table[b]
        k, there = kv8.values(self.kc, self.ke, tab, n)
        v, _ = kv8.values(self.vc, self.ve, tab, n)
        one, _ = kv8.values(np.full_like(self.vc, fp8.e4m3_encode(np.ones(1))[0]), self.ve, tab, n)
        e = one[..., 0]  # 2^e, 0 without a page
        with np.errstate(divide="ignore", invalid="ignore"):
            codes = np.where(e[..., None] > 0, np.abs(v) / e[..., None], 0.0)
        return k, v, there, codes, e


def split(q, out, lse, cut):
    """[(q, out, lse)] of the sequences, in fp64."""
    Hq, D = q.shape[-2:]
    qf, of = (np64(t).reshape(-1, Hq, D) for t in (q, out))
    lf = np64(lse).reshape(-1, Hq)
    if cut is None:
        cut = [q.shape[1] * b for b in range(q.shape[0] + 1)]
    return [(qf[a:e], of[a:e], lf[a:e]) for a, e in zip(cut, cut[1:])]


def faults(h, b, q, out, lse, scale, causal=True, window=0, sink=0):
    """What is wrong with the outputs of sequence b, or None."""
    k, v, there, codes, e = h.kv(b)
    n, Hq, D = q.shape
    L, H = k.shape[:2]
    G = Hq // H
    O, lw = kv8.attend(q, k, v, there, scale, causal, window, sink)
    A, _ = kv8.attend(q, k, np.abs(v), there, scale, causal, window, sink)
    if not np.isfinite(out).all():
        return "O is not finite"
    if not np.array_equal(np.isneginf(lse), np.isneginf(lw)):
        return "rows without a key differ"
    fine = np.isfinite(lw)
    if out[~fine].any():
        return "O of a row without a key is not 0"
    if not fine.any():
        return None
    i = L - n + np.arange(n)
    vis = attention.visibility(i, np.arange(L), causal, window, sink) & (i >= 0)[:, None] & there
    dot = np.einsum("thd,jhd->thj", np.abs(q), np.abs(np.repeat(k, G, 1))).max()
    ds = D * U * dot * scale + 2.0 ** -22 * (1 + dot * scale)
    seen = vis.sum(1)[:, None]
    lw = np.where(fine, lw, 0.0)
    dl = np.abs(np.where(fine, lse, 0.0) - lw)
    if not (dl <= ds + seen * U + 4 * U * np.abs(lw)).all():
        return f"LSE is off by {dl.max()}, a score's error being {ds}"
    small = np.empty(O.shape)
    for g in range(H):
        top = np.where(vis, e[None, :, g], 0.0).max(1)  # 2^E of each row
        small[:, g * G:(g + 1) * G] = (2.0 ** -32 * top[:, None] * (vis @ codes[:, g]))[:, None]
    tol = A * (2.0 ** -11 + 2 * ds + 2 * seen[..., None] * U) + small + 2.0 ** -8 * np.abs(O)
    bad = np.abs(out - O) / np.maximum(tol, 1e-300)
    return None if (bad <= 1).all() else f"O is off by {bad.max()} of its tolerance"


def check(q, c, out, lse, causal=True, window=0, sink=0, cut=None, scale=None):
    h = Host(c)
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    for b, (qb, ob, lb) in enumerate(split(q, out, lse, cut)):
        wrong = faults(h, b, qb, ob, lb, scale, causal, window, sink)
        assert wrong is None, (b, wrong)
