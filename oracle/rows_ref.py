"""CPU oracle for rows of activations in 8 or 4 bits, the RMS norm that makes them and the
products on microscaled rows (float64; test infrastructure only).

Formats.  A block is 32 consecutive elements of a row.  MX (OCP microscaling): scale byte
``s`` stands for 2^(s - 127), 255 for NaN; an element is an E4M3 byte (``"mxfp8"``) or an
E2M1 nibble (``"mxfp4"``, element 2i in the low nibble of byte i).  ``"q8_1"``: int8 codes
and a binary16 scale.  Rows here carry no padding: codes ``[m, k / 2]`` or ``[m, k]`` uint8
(int8 for q8_1), scales ``[m, k / 32]`` uint8 (float16 for q8_1).
"""
from __future__ import annotations

import numpy as np

from .iq4_ref import quantize_q8_1

__all__ = ["mx_levels", "quantize_rows", "dequant_rows", "rmsnorm", "mx_product"]

BLOCK = 32
_LARGEST = {"mxfp4": 6.0, "mxfp8": 448.0}
_EMAX = {"mxfp4": 2, "mxfp8": 8}


def mx_levels(fmt: str) -> np.ndarray:
    """The value of every code (16 or 256 of them; E4M3's two NaN codes are NaN)."""
    if fmt == "mxfp4":
        mag = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    else:
        mag = [(f / 8) * 2.0**-6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7) for e in range(16) for f in range(8)]
        mag[-1] = float("nan")
    return np.array(mag + [-v for v in mag])


def quantize_rows(x, fmt: str):
    """Float32 rows ``[m, k]`` -> (codes, scales).  A block that holds an infinity or a NaN
    has zero codes and a NaN scale."""
    x = np.asarray(x, dtype=np.float32)
    m, k = x.shape
    b = x.reshape(m, k // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(axis=2)
    b = np.where(bad[:, :, None], np.float32(0), b)
    if fmt == "q8_1":
        q, d = quantize_q8_1(b.reshape(m, k))
        d = d.copy()
        d[bad] = np.nan
        return q, d
    amax = np.abs(b).max(axis=2).astype(np.float64)
    # the largest power of two in the block, 2^floor(log2 amax), from frexp (exact)
    power = np.frexp(amax)[1] - 1
    s = np.where(amax > 0, np.clip(power - _EMAX[fmt] + 127, 0, 254), 0).astype(np.int64)
    v = b.astype(np.float64) * np.exp2(127.0 - s)[:, :, None]
    levels = mx_levels(fmt)
    mags = levels[: len(levels) // 2]
    mags = mags[np.isfinite(mags)]
    mid = (mags[1:] + mags[:-1]) / 2
    a = np.abs(v)
    code = np.searchsorted(mid, a, side="left")  # midpoints below a
    # a tie goes to the even code: at a midpoint `code` is the lower neighbour
    tie = (code < len(mid)) & (a == mid[np.minimum(code, len(mid) - 1)])
    code = np.where(tie & (code % 2 == 1), code + 1, code)
    code = np.where(np.signbit(v), code + len(levels) // 2, code)
    code = np.where(bad[:, :, None], 0, code).reshape(m, k).astype(np.uint8)
    s = np.where(bad, 255, s).astype(np.uint8)
    if fmt == "mxfp4":
        code = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    return code, s


def dequant_rows(codes, scales, fmt: str) -> np.ndarray:
    """The float64 values ``[m, k]`` that codes and scales stand for (exact)."""
    if fmt == "q8_1":
        return np.asarray(codes, dtype=np.float64) * np.repeat(np.asarray(scales, dtype=np.float64), BLOCK, axis=1)
    c = np.asarray(codes, dtype=np.uint8)
    if fmt == "mxfp4":
        c = np.stack([c & 15, c >> 4], axis=2).reshape(c.shape[0], -1)
    s = np.asarray(scales).astype(np.float64)
    power = np.where(s == 255, np.nan, np.exp2(s - 127))
    return mx_levels(fmt)[c] * np.repeat(power, BLOCK, axis=1)


def rmsnorm(x, res, gain, eps: float, round_to):
    """``(h, y)``: ``h = x + res`` rounded by ``round_to`` (a function float64 -> float64 of
    the rows' type), ``y = f32(f32(h * u) * gain)`` with ``u = f32(1 / sqrt(mean(h^2) +
    eps))``; ``eps`` is the binary32 value."""
    h = np.asarray(x, dtype=np.float64)
    if res is not None:
        h = round_to(h + np.asarray(res, dtype=np.float64))
    with np.errstate(all="ignore"):
        total = (h * h).sum(axis=1, keepdims=True)
        u = (1.0 / np.sqrt(total / h.shape[1] + np.float64(np.float32(eps)))).astype(np.float32)
        u = np.where(np.isfinite(total), u, np.float32("nan"))
        y = h.astype(np.float32) * u
        if gain is not None:
            y = y * np.asarray(gain, dtype=np.float32)
    return h, y


def mx_product(w, x) -> np.ndarray:
    """``Y = X W^T`` of decoded float64 rows (``w`` [n, k], ``x`` [m, k]), not rounded."""
    with np.errstate(all="ignore"):
        return np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
