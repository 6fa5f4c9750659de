"""The rotation of positions and the paged 8-bit KV cache: its numbers, an append,
reading back, and attention of the newest tokens (oracle; test infrastructure only).

Rotation. Pairs (a, b) of the first R channels, (i, i + R/2) or (2i, 2i + 1), become
(a c - b s, b c + a s) with c = table[p][i], s = table[p][R/2 + i], products and sums
rounded to fp32 one by one.

Numbers. A block of 32 rows of a head has the smallest e in [-40, 40] with
max|x| <= 448 * 2^e (40 if none), and the codes e4m3(x / 2^e), nearest, ties to the even
code, saturating, a NaN as 0. An append into a block with rows takes the larger of its
exponent and the new rows', and rounds the codes held once more.

Attention. Of a sequence's L cached tokens the newest n are the queries, token t at
i = L - n + t; it sees key j < L iff attention.visibility(i, j) and j's page is one
(nothing if i < 0).
"""
from __future__ import annotations

import math

import numpy as np

from oracle import attention, fp8

BLOCK = 32


def rotate(x, pos, table, interleaved: bool = False, inverse: bool = False) -> np.ndarray:
    """fp32 [n, heads, D] rotated at positions pos [n] (clipped to the table)."""
    x = np.asarray(x, dtype=np.float32).copy()
    table = np.asarray(table, dtype=np.float32)
    R = table.shape[1]
    row = table[np.clip(np.asarray(pos, dtype=np.int64), 0, table.shape[0] - 1)][:, None, :]
    c, s = row[..., : R // 2], row[..., R // 2:]
    if inverse:
        s = -s
    i = np.arange(R // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    a, b = x[..., ia], x[..., ib]
    with np.errstate(invalid="ignore", over="ignore"):
        x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def exponent(amax) -> int:
    """Smallest e in [-40, 40] with amax <= 448 * 2^e, 40 if there is none."""
    for e in range(-40, 40):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return 40


def encode(x, e: int) -> np.ndarray:
    x = attention._f64(x)
    x = np.where(np.isnan(x), 0.0, x)
    return fp8.e4m3_encode(np.clip(x, -1e300, 1e300) / 2.0 ** e)


def append(k_codes, k_exps, table, start: int, x) -> None:
    """Rows x [n, H, D] behind a sequence's `start` rows, in place, in codes
    [pages, H, page size, D] and exps [pages, H, page size / 32]; table: its pages."""
    n_pages, H, ps, _ = k_codes.shape
    cap = len(table) * ps
    x = attention._f64(x)
    n = x.shape[0]
    for base in range(start // BLOCK * BLOCK, min(start + n, cap), BLOCK):
        page, at = int(table[base // ps]), base % ps
        if not 0 <= page < n_pages:
            continue
        lo, hi = max(start, base) - base, min(start + n, base + BLOCK) - base
        for h in range(H):
            new = x[base + lo - start: base + hi - start, h]
            e = exponent(np.abs(np.where(np.isnan(new), 0.0, new)).max())
            if lo > 0:
                old = min(max(int(k_exps[page, h, at // BLOCK]), -40), 40)
                e = max(e, old)
                if e > old:
                    held = fp8.e4m3_decode(k_codes[page, h, at: at + lo])
                    k_codes[page, h, at: at + lo] = encode(held * 2.0 ** old, e)
            k_codes[page, h, at + lo: at + hi] = encode(new, e)
            k_exps[page, h, at // BLOCK] = e


def values(codes, exps, table, rows: int):
    """(values [rows, H, D], which rows have a page) of a sequence."""
    n_pages, H, ps, D = codes.shape
    out = np.zeros((rows, H, D))
    there = np.zeros(rows, dtype=bool)
    for r0 in range(0, rows, BLOCK):
        page, at = int(table[r0 // ps]), r0 % ps
        if not 0 <= page < n_pages:
            continue
        n = min(BLOCK, rows - r0)
        e = np.clip(exps[page, :, at // BLOCK].astype(np.float64), -40, 40)
        out[r0: r0 + n] = (fp8.e4m3_decode(codes[page, :, at: at + n]) *
                           2.0 ** e[:, None, None]).transpose(1, 0, 2)
        there[r0: r0 + n] = True
    return out, there


def attend(q, k, v, there, scale: float, causal=True, window=0, sink=0):
    """(O [n, Hq, D], LSE [n, Hq]) of the newest n tokens q against a sequence's
    values k, v [L, Hkv, D]."""
    q = attention._f64(q)
    n, Hq, _ = q.shape
    L, H = k.shape[:2]
    O, lse = np.zeros(q.shape), np.full((n, Hq), -math.inf)
    if L == 0:
        return O, lse
    i = L - n + np.arange(n)
    vis = attention.visibility(i, np.arange(L), causal, window, sink)
    vis = vis & (i >= 0)[:, None] & there[None, :]
    for h in range(Hq):
        O[:, h], lse[:, h] = attention.softmax_rows(q[:, h], k[:, h * H // Hq], v[:, h * H // Hq],
                                                    vis, scale)
    return O, lse
