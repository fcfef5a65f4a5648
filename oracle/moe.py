"""Oracle of what a mixture-of-experts layer has around its grouped products,
in numpy fp64: the router's gate, pairs sorted by expert, rows there and back,
and their gradients.

TEST INFRASTRUCTURE.  Pair (t, j) is number t k + j; an expert outside 0 .. E-1
is nobody's, a row of -1 is no row.
"""
from __future__ import annotations

import numpy as np


def gate(logits: np.ndarray, k: int, renorm: bool):
    """logits [T, E] -> (weights [T, k], chosen [T, k]): the k largest, of equal ones the lowest, -inf never."""
    T, E = logits.shape
    weights, chosen = np.zeros((T, k)), np.full((T, k), -1, np.int32)
    for t in range(T):
        row = logits[t].astype(np.float64)
        rank = np.where(np.isnan(row), np.inf, row)
        order = sorted((e for e in range(E) if rank[e] > -np.inf), key=lambda e: (-rank[e], e))[:k]
        if not order:
            continue
        chosen[t, :len(order)] = order
        if not np.isfinite(rank.max()) or np.isnan(row).any():
            weights[t, :len(order)] = np.nan
            continue
        p = np.exp(row - row.max())
        weights[t, :len(order)] = p[order] / (p[order].sum() if renorm else p.sum())
    return weights, chosen


def gate_bwd(grad: np.ndarray, logits: np.ndarray, chosen: np.ndarray, renorm: bool):
    """The gradient of the logits: the derivative of gate's weights, one expert after another."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        row = logits[t].astype(np.float64)
        js = [j for j, e in enumerate(chosen[t]) if 0 <= e < E]
        if not js:
            continue
        p = np.exp(row - row.max())
        inside = np.zeros(E, bool)
        inside[[chosen[t, j] for j in js]] = True
        q = p * inside / (p * inside).sum() if renorm else p / p.sum()
        for j in js:
            e = chosen[t, j]
            out[t] += grad[t, j] * q[e] * ((np.arange(E) == e) - q)
    return out


def sort(experts: np.ndarray, groups: int):
    """(offsets [groups], rows like experts, order [rows of anybody's])."""
    flat = experts.reshape(-1)
    rows, order, offsets = np.full(flat.size, -1, np.int32), [], []
    for g in range(groups):
        mine = np.flatnonzero(flat == g)
        rows[mine] = np.arange(len(order), len(order) + mine.size)
        order += mine.tolist()
        offsets.append(len(order))
    return np.array(offsets, np.int32), rows.reshape(experts.shape), np.array(order, np.int32)


def gather(x: np.ndarray, rows: np.ndarray):
    """[T k, H] of x's dtype; rows of no pair are 0."""
    out = np.zeros((rows.size, x.shape[1]), x.dtype)
    for t in range(rows.shape[0]):
        for r in rows[t]:
            if 0 <= r < rows.size:
                out[r] = x[t]
    return out


def combine(y: np.ndarray, rows: np.ndarray, weights=None):
    """(out [T, H], the sum of the terms' magnitudes)."""
    T, k = rows.shape
    out, size = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j, r in enumerate(rows[t]):
            if 0 <= r < rows.size:
                term = (1.0 if weights is None else float(weights[t, j])) * y[r]
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def combine_dots(grad: np.ndarray, y: np.ndarray, rows: np.ndarray):
    """(grad_weights [T, k], the sum of the terms' magnitudes)."""
    out, size = np.zeros(rows.shape), np.zeros(rows.shape)
    for t in range(rows.shape[0]):
        for j, r in enumerate(rows[t]):
            if 0 <= r < rows.size:
                out[t, j], size[t, j] = grad[t] @ y[r], np.abs(grad[t]) @ np.abs(y[r])
    return out, size
