"""Attention by its definition, in float64 numpy, one sequence and one head at
a time; and how far a result that rounds the weights and the output to 16 bits
may be from it."""
from __future__ import annotations

import numpy as np

UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # half an ulp, relative


def chain(n: int, m: int) -> np.ndarray:
    """seen [n, m]: the n queries are the last of the m keys; each sees the keys up to its own."""
    return np.arange(m)[None, :] <= np.arange(n)[:, None] + m - n


def tree(bits: np.ndarray, m: int) -> np.ndarray:
    """seen [n, m] from the drafted tokens' bits [n, n]: everything before them, and what the bits say."""
    n = bits.shape[0]
    seen = np.zeros((n, m), dtype=bool)
    seen[:, :max(m - n, 0)] = True
    lo = max(n - m, 0)  # drafted tokens with no row of their own: there are fewer rows than queries
    seen[:, max(m - n, 0):] = bits[:, lo:]
    return seen


def ancestors(parents) -> np.ndarray:
    n = len(parents)
    bits = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            bits[i, j] = True
            j = parents[j]
    return bits


def attention(q, k, v, seen, scale):
    """q [n, H, D], k and v [m, Hkv, D], float64. Returns out [n, H, D], lse
    [n, H] and, per element, the weighted absolute values sum_j w_j |v_j| and
    the largest |score error| per unit of fp32 rounding (for tolerance())."""
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    out, lse = np.zeros((n, heads, dim)), np.full((n, heads), -np.inf)
    spread, product = np.zeros((n, heads, dim)), np.zeros((n, heads))
    for h in range(heads):
        for i in range(n):
            at = np.flatnonzero(seen[i])
            if not len(at):
                continue
            keys, values = k[at, h // group], v[at, h // group]
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (keys @ q[i, h])
                top = s.max()
                w = np.exp(s - top)
                lse[i, h] = top + np.log(w.sum())
                w = w / w.sum()
                # infinities among the values: what a sum of the seen ones gives
                out[i, h] = w @ values
                spread[i, h] = w @ np.abs(values)
                product[i, h] = scale * (np.abs(keys) @ np.abs(q[i, h])).max()
    return out, lse, spread, product


def tolerance(out, lse, spread, product, dim, keys, dtype, largest):
    """Bounds on |got - out| and |got - lse|.

    Scores: a dot product of `dim` exact 16-bit products added in fp32 is off
    by at most dim * 2^-22 of the sum of their absolute values (2^-23 a step
    where the addition truncates), and scaling, the exponent's argument and
    the exponential add a few 2^-22 of the same size. Weights: their relative
    error is twice that (the sum's too) plus half an ulp of the type they are
    held in; below fp16's smallest normal number half of 2^-24 each. Output:
    half an ulp more."""
    u = UNIT[dtype]
    score = (dim + 8) * 2.0 ** -22 * (product + 1.0) + 2.0 ** -20
    tiny = keys * 2.0 ** -25 * largest if dtype == "fp16" else 0.0
    small = 2.0 ** -25 if dtype == "fp16" else 0.0
    value = u * np.abs(out) + (u + 2.0 * score[..., None] + keys * 2.0 ** -23) * (1.0 + u) * spread + tiny + small
    return value, score + 2.0 ** -20 * (1.0 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
