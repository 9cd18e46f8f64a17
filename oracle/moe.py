"""The operators around the experts' products in float64. TEST INFRASTRUCTURE ONLY (see
oracle/__init__.py).

  route        the k largest logits of a token and their softmax weights, and the gradient
  expert_sort  rows of every expert: stable, by expert
  dispatch     rows of tokens to the rows of their assignments
  combine      weighted sums of the rows of a token's assignments, and the gradient
  fp8_rows     E4M3 with a power-of-two scale for each 128 columns of a row (the last group
               of a row holds what is left of it)

A position outside [0, rows) is an assignment without a row. Alongside a sum goes `mag`,
the sum of its terms' magnitudes, which error bounds are made of.
"""
from __future__ import annotations

import numpy as np

from .formats import e4m3_decode, e4m3_round_nearest_even
from .fp8 import fp8_group_exponent, fp8_scale_exponent


def choose(row: np.ndarray, k: int):
    """Experts of the k largest logits: NaN before all, equal values by expert, -Inf never (-1)."""
    rank = sorted(range(len(row)), key=lambda e: (0 if np.isnan(row[e]) else 1, 0 if np.isnan(row[e]) else -row[e], e))
    rank = [e for e in rank if np.isnan(row[e]) or row[e] > -np.inf][:k]
    return rank + [-1] * (k - len(rank))


def softmax(x: np.ndarray) -> np.ndarray:
    """Of one row; zeros where every value is -Inf, NaN where one is NaN or +Inf."""
    if len(x) == 0 or (x == -np.inf).all():
        return np.zeros(len(x))
    with np.errstate(invalid="ignore"):
        e = np.exp(x - x.max())
        return e / e.sum()


def route(logits: np.ndarray, k: int, renorm: bool):
    """(weights [T, k], experts int32 [T, k])."""
    T = logits.shape[0]
    weights, experts = np.zeros((T, k)), np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        experts[t] = choose(logits[t], k)
        on = experts[t] >= 0
        if renorm:
            weights[t, on] = softmax(logits[t, experts[t, on]])
        else:
            weights[t, on] = softmax(logits[t])[experts[t, on]]
    return weights, experts


def route_grad(dw, weights, experts, logits, renorm: bool):
    """(dlogits, mag) [T, E] for the weights that were given."""
    T, E = logits.shape
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = (experts[t] >= 0) & (experts[t] < E)
        x, w, at = (weights[t] * np.where(on, dw[t], 0.0))[on], weights[t][on], experts[t][on]
        share = np.zeros(E)
        if renorm:
            np.add.at(share, at, w)
        else:
            share = softmax(logits[t])
        np.add.at(d[t], at, x)
        np.add.at(mag[t], at, np.abs(x))
        d[t] -= x.sum() * share
        mag[t] += np.abs(x).sum() * share
    return d, mag


def expert_sort(experts: np.ndarray, n_experts: int):
    """(offsets int64 [E + 1], positions int32 like experts, order int32 [count])."""
    flat = np.asarray(experts).reshape(-1)
    lists = [[] for _ in range(n_experts)]
    for i, e in enumerate(flat):
        if 0 <= e < n_experts:
            lists[e].append(i)
    order = np.full(flat.size, -1, dtype=np.int32)
    positions = np.full(flat.size, -1, dtype=np.int32)
    offsets = np.zeros(n_experts + 1, dtype=np.int64)
    row = 0
    for e, mine in enumerate(lists):
        for i in mine:
            order[row], positions[i] = i, row
            row += 1
        offsets[e + 1] = row
    return offsets, positions.reshape(np.shape(experts)), order


def dispatch(x: np.ndarray, positions: np.ndarray, out: np.ndarray) -> np.ndarray:
    """`out` [rows, ...] with x[t] in the rows of t's assignments."""
    out = out.copy()
    for t, row in enumerate(positions):
        for r in row:
            if 0 <= r < len(out):
                out[r] = x[t]
    return out


def combine(y, positions, weights=None, residual=None):
    """(out, mag) [T, H]."""
    T, k = positions.shape
    out = np.zeros((T, y.shape[1])) if residual is None else residual.astype(np.float64).copy()
    mag = np.abs(out)
    for t in range(T):
        for j in range(k):
            r = positions[t, j]
            if 0 <= r < len(y):
                term = y[r] * (1.0 if weights is None else weights[t, j])
                out[t] += term
                mag[t] += np.abs(term)
    return out, mag


def combine_grad(grad, y, positions, weights=None):
    """(dy [R, H] with NaN in rows of no assignment, dw [T, k], mag of dw)."""
    dy = np.full(y.shape, np.nan)
    dw, mag = np.zeros(positions.shape), np.zeros(positions.shape)
    for t, row in enumerate(positions):
        for j, r in enumerate(row):
            if 0 <= r < len(y):
                dy[r] = grad[t] * (1.0 if weights is None else weights[t, j])
                dw[t, j] = (grad[t] * y[r]).sum()
                mag[t, j] = np.abs(grad[t] * y[r]).sum()
    return dy, dw, mag


def fp8_rows(x: np.ndarray):
    """(E4M3 uint8 [R, C], scale bits uint32 [R, ceil(C / 128)]): s = 2^i, i >= -126 the smallest
    with max|x| / s <= 448 (0 for zeros); a group with NaN or Inf has scale NaN, codes 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    q = np.zeros((R, C), dtype=np.uint8)
    s = np.zeros((R, (C + 127) // 128), dtype=np.uint32)
    for g in range(s.shape[1]):
        part = x[:, 128 * g:128 * g + 128]
        ok = np.isfinite(part).all(axis=1)
        v = np.where(ok[:, None], part, 0.0)
        i = np.maximum(fp8_group_exponent(np.abs(v).max(axis=1)), -126)
        codes = e4m3_round_nearest_even(v / np.ldexp(1.0, i)[:, None])
        q[:, 128 * g:128 * g + 128] = np.where(ok[:, None], codes, 0x7F)
        s[:, g] = np.where(ok, (i + 127).astype(np.uint32) << 23, 0x7FC00000)
    return q, s


def fp8_row_values(q: np.ndarray, s_bits: np.ndarray) -> np.ndarray:
    """float64 [R, C] of fp8_rows' layout; scales through their exponent field (255: NaN)."""
    ef = fp8_scale_exponent(s_bits)
    s = np.where(ef == 255, np.nan, np.ldexp(1.0, np.minimum(ef, 254) - 127))
    return e4m3_decode(q) * np.repeat(s, 128, axis=1)[:, :q.shape[1]]
