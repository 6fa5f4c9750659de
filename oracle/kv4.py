"""The 4-bit KV cache: its numbers, a decoding step over it, the attention
weight of each key, and eviction (oracle; test infrastructure only).

Numbers. y = x * inv with inv = 1 / descale, both rounded to fp32 (a NaN is
0); per block of 32 channels s = e4m3(max |y| / 7), nearest, ties to the even
code, at most 448; c = clamp(round_half_even(y / s), -7, 7), 0 where s = 0.
The block stands for c * s * descale. Nibble c + 8; channel 2i is the low
nibble of byte i.

Decoding. A sequence has L cached tokens; token t of the Tq newest sits at
i = L - Tq + t and sees key j < L iff attention.visibility(i, j) (nothing if
i < 0).

Weights. weight_j = sum over observed queries that see key j, and over the
query heads that share its KV head, of the attention probability.

Eviction. Of L > keep keys the first `sink`, the last `recent`, and the
heaviest keep - sink - recent of the others; the first of equal ones, NaN
above every number; order kept.
"""
from __future__ import annotations

from typing import Tuple

import numpy as np

from oracle import attention, fp8

BLOCK = 32


def quantize(x, descale: float) -> Tuple[np.ndarray, np.ndarray]:
    """(packed codes uint8 [..., D/2], E4M3 scale bytes uint8 [..., D/32])."""
    x = attention._f64(x)
    inv = np.float32(1.0) / np.float32(descale)
    with np.errstate(over="ignore", invalid="ignore"):
        y = (x * np.float64(inv)).astype(np.float32).astype(np.float64)
    y = np.where(np.isnan(y), 0.0, y)
    y = y.reshape(x.shape[:-1] + (-1, BLOCK))
    sb = fp8.e4m3_encode(np.abs(y).max(-1) / 7.0)
    s = fp8.e4m3_decode(sb)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(s > 0, np.clip(np.rint(y / s), -7, 7), 0.0)
    u = (c + 8).astype(np.uint8).reshape(x.shape)
    return u[..., 0::2] + 16 * u[..., 1::2], sb


def values(codes, scales, descale: float) -> np.ndarray:
    """The fp64 values [..., D] of packed codes and scale bytes."""
    codes = np.asarray(codes, dtype=np.uint8)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,)).astype(np.float64)
    s = fp8.e4m3_decode(scales) * float(np.float32(descale))
    return (c - 8.0) * np.repeat(s, BLOCK, axis=-1)


def decode(q, k, v, lens, scale: float, causal: bool = True, window: int = 0,
           sink: int = 0) -> Tuple[np.ndarray, np.ndarray, np.ndarray]:
    """(O [B,Tq,Hq,D], LSE [B,Tq,Hq], weight [B,Hkv,C]) for q [B,Tq,Hq,D] and
    the cache's values k, v [B,Hkv,C,D]."""
    q, k, v = attention._f64(q), attention._f64(k), attention._f64(v)
    B, Tq, Hq, D = q.shape
    H, C = k.shape[1], k.shape[2]
    G = Hq // H
    O = np.zeros(q.shape)
    L = np.full((B, Tq, Hq), -np.inf)
    W = np.zeros((B, H, C))
    for b in range(B):
        n = int(min(max(int(lens[b]), 0), C))
        if n == 0:
            continue
        i = n - Tq + np.arange(Tq)
        vis = attention.visibility(i, np.arange(n), causal, window, sink) & (i >= 0)[:, None]
        for h in range(Hq):
            g = h // G
            o, lse = attention.softmax_rows(q[b, :, h], k[b, g, :n], v[b, g, :n], vis, scale)
            O[b, :, h], L[b, :, h] = o, lse
            s = scale * (q[b, :, h] @ k[b, g, :n].T)
            safe = np.where(np.isfinite(lse), lse, 0.0)
            W[b, g, :n] += np.where(vis, np.exp(np.where(vis, s, 0.0) - safe[:, None]), 0.0).sum(0)
    return O, L, W


def key_weights(q, k, lse, scale: float, causal: bool = True, window: int = 0, sink: int = 0,
                cu_seqlens=None, observe: int = 0) -> np.ndarray:
    """[B, Hkv, S] from natural-order q [B,S,Hq,D], k [B,S,Hkv,D] and
    lse [B,Hq,S] (packed: without B)."""
    q, k, lse = attention._f64(q), attention._f64(k), attention._f64(lse)
    if cu_seqlens is not None:
        cu = [int(x) for x in cu_seqlens]
        parts = [key_weights(q[None, a:e], k[None, a:e], lse[None, :, a:e], scale, causal, window,
                             sink, None, observe)[0] for a, e in zip(cu, cu[1:])]
        return np.concatenate(parts, axis=-1)
    B, S, Hq, D = q.shape
    H = k.shape[2]
    W = np.zeros((B, H, S))
    rows = np.arange(max(0, S - observe) if observe > 0 else 0, S)
    vis = attention.visibility(rows, np.arange(S), causal, window, sink)
    for b in range(B):
        for h in range(Hq):
            g = h // (Hq // H)
            l = lse[b, h, rows]
            ok = vis & np.isfinite(l)[:, None]
            s = scale * (q[b, rows, h] @ k[b, :, g].T)
            W[b, g] += np.where(ok, np.exp(np.where(ok, s, 0.0) - np.where(np.isfinite(l), l, 0.0)[:, None]),
                                0.0).sum(0)
    return W


def kept_rows(weight, lens, keep: int, recent: int, sink: int) -> np.ndarray:
    """[B, Hkv, keep] int32, -1 behind the last."""
    w = attention._f64(weight)
    B, H, C = w.shape
    out = np.full((B, H, keep), -1, dtype=np.int32)
    for b in range(B):
        n = int(min(max(int(lens[b]), 0), C))
        for h in range(H):
            if n <= keep:
                out[b, h, :n] = np.arange(n)
                continue
            mid = [(-(np.inf if np.isnan(x) else x), not np.isnan(x), j)
                   for j, x in enumerate(w[b, h, :n]) if sink <= j < n - recent]
            take = [j for _, _, j in sorted(mid)[: keep - sink - recent]]
            rows = sorted(list(range(sink)) + take + list(range(n - recent, n)))
            out[b, h] = rows
    return out
