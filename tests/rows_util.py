"""Helpers for the tests of rows in 8 or 4 bits: types, strided buffers with sentinels."""
from __future__ import annotations

import numpy as np
import torch

import dequant_matmul_iq4_amd as iq4
import oracle
from gpu_util import dev, host

FMT = {"mxfp4": iq4.IQ4_ROWS_MXFP4, "mxfp8": iq4.IQ4_ROWS_MXFP8, "q8_1": iq4.IQ4_ROWS_Q8_1}
TYPES = {"f32": (iq4.IQ4_F32, torch.float32), "f16": (iq4.IQ4_F16, torch.float16), "bf16": (iq4.IQ4_BF16, torch.bfloat16)}
# half a step of the type, relative: one rounding to nearest
HALF_STEP = {t: torch.finfo(d).eps / 2 for t, (_, d) in TYPES.items()}


def rounder(t: str):
    """float64 -> float64 values of the type (through torch on the CPU: one rounding)."""
    return lambda v: torch.from_numpy(np.ascontiguousarray(v)).to(TYPES[t][1]).double().numpy()


def floats(x: np.ndarray, t: str, ld: int | None = None) -> torch.Tensor:
    """Rows of `t` on the device, `ld` elements apart, NaN between them."""
    m, k = x.shape
    b = torch.full((m, ld or k), float("nan"), dtype=TYPES[t][1], device="cuda")
    b[:, :k] = dev(np.asarray(x, dtype=np.float32)).to(TYPES[t][1])
    return b


def row_buffers(fmt: str, m: int, k: int, ldq: int | None = None, lds: int | None = None, fill: int = 0xEE):
    """Code and scale buffers of m rows, filled with a sentinel, and their strides."""
    c, s = iq4.iq4_rows_bytes(FMT[fmt], k)
    ldq, lds = ldq or c, lds or s
    return (torch.full((m, ldq), fill, dtype=torch.uint8, device="cuda"),
            torch.full((m, lds), fill, dtype=torch.uint8, device="cuda"), ldq, lds)


def split_rows(fmt: str, k: int, q: torch.Tensor, d: torch.Tensor):
    """Device buffers -> the oracle's arrays (codes, scales), with the padding checked to be zero."""
    c, s = iq4.iq4_rows_bytes(FMT[fmt], k)
    q, d = host(q), host(d)
    if fmt == "q8_1":
        return q[:, :k].copy().view(np.int8), d[:, : k // 16].copy().view(np.float16)
    n = k // 2 if fmt == "mxfp4" else k
    assert not q[:, n:c].any() and not d[:, k // 32:s].any(), "padding is not zero"
    return q[:, :n], d[:, : k // 32]


def stored(fmt: str, codes: np.ndarray, scales: np.ndarray, k: int, ldq: int | None = None, lds: int | None = None):
    """The oracle's MX rows as the library reads them: zero padding, 0xFF between the rows."""
    q, d, ldq, lds = row_buffers(fmt, len(codes), k, ldq, lds, 0xFF)
    c, s = iq4.iq4_rows_bytes(FMT[fmt], k)
    q[:, :c] = 0
    d[:, :s] = 0
    q[:, : codes.shape[1]] = dev(codes)
    d[:, : scales.shape[1]] = dev(scales)
    return q, d, ldq, lds


def packed(codes: np.ndarray, scales: np.ndarray, n: int, k: int) -> torch.Tensor:
    nbytes = iq4.iq4_mx_packed_bytes(n, k)
    out = torch.full((nbytes,), 0xEE, dtype=torch.uint8, device="cuda")
    iq4.iq4_mx_pack_weights(dev(codes), codes.shape[1], dev(scales), scales.shape[1], n, k, out)
    return out


def value(fmt: str, codes, scales) -> np.ndarray:
    return oracle.dequant_rows(codes, scales, fmt)
