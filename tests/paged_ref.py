"""Plain 64-bit forms of the paged-cache operators, sequence by sequence
(test infrastructure; numpy, no library code)."""
from __future__ import annotations

import math

import numpy as np

from oracle import ds4a_oracle as O

U16 = 2.0 ** -8  # half a step of bf16, relative


def cache_rows(pages, table_row, slots, page, D, R, fp8):
    """float64 rows of the given slots; pages: uint16 bits or uint8 rows [n_pages, page, row]."""
    slots = np.asarray(slots, dtype=np.int64)
    at = pages[np.asarray(table_row)[slots // page], slots % page]
    return O.dequantize_kv_fp8(at, D, R) if fp8 else O.widen(at)


def rotate(x, pos, R, base, sign):
    x = x.copy()
    if R:
        ang = sign * pos * base ** (-2.0 * np.arange(R // 2) / R)
        a, b = x[..., -R::2].copy(), x[..., x.shape[-1] - R + 1::2].copy()
        x[..., -R::2] = a * np.cos(ang) - b * np.sin(ang)
        x[..., x.shape[-1] - R + 1::2] = a * np.sin(ang) + b * np.cos(ang)
    return x


def attend(q, g, rows, n_sel, sink, pos, scale, R, base, eps, key_off=0.0):
    """q [H, D], rows [n, D] (the first n_sel of the cache) -> (out [H, D],
    weights [n_sel], bound of out, bound of weights).

    The bounds count the roundings to bf16 that the kernels make, u = 2^-8
    each, to first order: the prepared query (a logit moves by at most
    A = u scale sum |q^||k|, its probability by the factor A + sum p A), the
    probability before the second product (u) and the result (u); the
    denominator adds rounded probabilities (u).  The float32 arithmetic
    between them (512 terms, 2^-24 each, and 2 ulp of the exponential) is
    covered by taking 5 % more, and 1e-6 of the largest row value.  key_off: how
    far, relative, the rows in the cache may be from the given ones."""
    H, D = q.shape
    qh = q / np.sqrt((q * q).mean(-1, keepdims=True) + eps) * g
    qh = rotate(qh, pos, R, base, 1)
    n = rows.shape[0]
    if n == 0:
        return np.zeros((H, D)), np.zeros(0), np.zeros((H, D)), np.zeros(0)
    z = qh @ rows.T * scale
    top = np.maximum(z.max(-1), sink)[:, None]
    e = np.exp(z - top)
    p = e / (e.sum(-1, keepdims=True) + np.exp(sink[:, None] - top))
    A = (U16 + key_off) * scale * (np.abs(qh) @ np.abs(rows).T)
    rel = np.expm1(A + (p * A).sum(-1, keepdims=True))
    out = rotate(p @ rows, pos, R, base, -1)
    spread = (p * (rel + 2 * U16 + key_off)) @ np.abs(rows)
    if R:  # a rotation mixes a pair
        a, b = spread[:, -R::2].copy(), spread[:, D - R + 1::2].copy()
        spread[:, -R::2] = spread[:, D - R + 1::2] = a + b
    b_out = 1.05 * spread + U16 * (np.abs(out) + spread) + 1e-6 * np.abs(rows).max()
    w = p[:, :n_sel].sum(0)
    b_w = 1.05 * (p * (rel + 2 * U16))[:, :n_sel].sum(0)
    return out, w, b_out, b_w + U16 * (w + b_w) + 1e-7


def evict(w, acc, entry, drop, n, closed, budget, recent):
    """One sequence: acc (float32) [S], entry [S], drop, n slots in use ->
    (acc, entry, drop, moves) after; moves is a list of (from, to)."""
    acc, entry = acc.astype(np.float32).copy(), entry.copy()
    if w is not None:
        acc[:n] = acc[:n] + w[:n].astype(np.float32)
    if n <= budget:
        return acc, entry, drop, []
    num = np.where(entry[:n] < 0, np.arange(n) + drop, entry[:n])

    def order(s):
        a = acc[s]
        rank = math.inf if np.isnan(a) else float(a)
        return (0 if num[s] >= closed - recent else 1, 0 if np.isnan(a) else 1, -rank, s)

    keep = set(sorted(range(n), key=order)[:budget])
    holes = [s for s in range(budget) if s not in keep]
    movers = [s for s in range(budget, n) if s in keep]
    entry[:budget] = num[:budget]
    for to, fr in zip(holes, movers):
        acc[to], entry[to] = acc[fr], num[fr]
    acc[budget:], entry[budget:] = 0, -1
    return acc, entry, drop + n - budget, list(zip(movers, holes))


def untile_scales(t, rows, K):
    kb = K // 32
    r, b = np.arange(rows)[:, None], np.arange(kb)
    return t[((r // 128) * (K // 128) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]


def tile_scales(s):
    rows, kb = s.shape
    out = np.zeros(-(-rows // 128) * (kb // 4) * 512, np.uint8)
    r, b = np.arange(rows)[:, None], np.arange(kb)
    out[((r // 128) * (kb // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = s
    return out
