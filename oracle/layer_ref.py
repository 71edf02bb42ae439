"""CPU oracle for 4-bit weights with group scales, the way of tokens' rows into the experts'
order and back, and SwiGLU, with their gradients (float64; test infrastructure only)."""
from __future__ import annotations

import numpy as np

__all__ = ["g4_weights", "g4_product", "moe_dispatch", "moe_combine", "moe_combine_grad", "swiglu", "swiglu_grad"]


def g4_weights(codes, scales, zeros, group: int) -> np.ndarray:
    """``w = s (q - z)``: codes ``[n, k / 2]`` uint8 (the first of a byte in its low half), scales
    (and zero points, or None: 8) one per ``group`` weights of a row, the last group may be short."""
    c = np.asarray(codes, dtype=np.uint8)
    q = np.empty((c.shape[0], 2 * c.shape[1]))
    q[:, 0::2], q[:, 1::2] = c % 16, c // 16
    k = q.shape[1]
    wide = lambda v: np.repeat(np.asarray(v, dtype=np.float64), group, axis=1)[:, :k]  # noqa: E731
    return wide(scales) * (q - (8.0 if zeros is None else wide(zeros)))


def g4_product(w, x) -> np.ndarray:
    return np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T


def _slots(slot_row, n_rows):
    s = np.asarray(slot_row)
    return s, (s >= 0) & (s < n_rows)


def moe_dispatch(x, slot_row, w, rows):
    """``rows`` (a copy) with ``rows[slot_row[t, j]] = w[t, j] x[t]`` for the pairs that have a row."""
    out = np.array(rows, dtype=np.float64)
    s, has = _slots(slot_row, len(out))
    for t in range(s.shape[0]):
        for j in range(s.shape[1]):
            if has[t, j]:
                out[s[t, j]] = np.asarray(x[t], dtype=np.float64) * (1.0 if w is None else float(w[t, j]))
    return out


def moe_combine(rows, slot_row, w, add=None):
    """``out[t] = sum_j w[t, j] rows[slot_row[t, j]] (+ add[t])``."""
    s, has = _slots(slot_row, len(rows))
    out = np.zeros((s.shape[0], rows.shape[1]))
    for t in range(s.shape[0]):
        for j in range(s.shape[1]):
            if has[t, j]:
                out[t] += np.asarray(rows[s[t, j]], dtype=np.float64) * (1.0 if w is None else float(w[t, j]))
    return out if add is None else out + np.asarray(add, dtype=np.float64)


def moe_combine_grad(dout, rows, slot_row, w):
    """``(drows, dw)``; rows that no pair has get NaN."""
    s, has = _slots(slot_row, len(rows))
    drows = np.full(rows.shape, np.nan)
    dw = np.zeros(s.shape)
    for t in range(s.shape[0]):
        for j in range(s.shape[1]):
            if has[t, j]:
                d = np.asarray(dout[t], dtype=np.float64)
                drows[s[t, j]] = d * (1.0 if w is None else float(w[t, j]))
                dw[t, j] = d @ np.asarray(rows[s[t, j]], dtype=np.float64)
    return drows, dw


def _sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(g, u):
    g, u = np.asarray(g, dtype=np.float64), np.asarray(u, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        return g * _sigmoid(g) * u


def swiglu_grad(dh, g, u):
    """``(dg, du)``."""
    dh, g, u = (np.asarray(v, dtype=np.float64) for v in (dh, g, u))
    s, r = _sigmoid(g), _sigmoid(-g)
    with np.errstate(invalid="ignore"):
        return dh * u * (s + g * s * r), dh * g * s
