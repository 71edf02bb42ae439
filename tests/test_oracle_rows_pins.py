"""Pins of the row-format oracle: the formats' own numbers, and rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest

import oracle
from exact import f16, f32, round_to_format


def test_levels():
    four = oracle.mx_levels("mxfp4")
    assert four.tolist()[:8] == [0, 0.5, 1, 1.5, 2, 3, 4, 6] and np.all(four[8:] == -four[:8])
    eight = oracle.mx_levels("mxfp8")
    assert eight[0x38] == 1.0 and eight[0x7E] == 448.0 and eight[1] == 2.0**-9 and eight[0x08] == 2.0**-6
    assert np.isnan(eight[0x7F]) and np.isnan(eight[0xFF]) and eight[0xB8] == -1.0
    assert np.isnan(eight).sum() == 2


def _by_hand(x, fmt):
    """One block, element by element, with rationals: (values, scale byte)."""
    amax = max(abs(Fraction(float(v))) for v in x)
    e = 0
    if amax:
        e = -200
        while Fraction(2) ** (e + 1) <= amax:
            e += 1
    s = max(0, e - (2 if fmt == "mxfp4" else 8) + 127) if amax else 0
    scale = Fraction(2) ** (s - 127)
    out = []
    for v in x:
        f = Fraction(float(v)) / scale
        bits, emin, top = (2, 0, 6) if fmt == "mxfp4" else (4, -6, 448)
        r = Fraction(round_to_format(f, bits, emin, 40))
        out.append(max(-top, min(top, r)) * scale)
    return out, s


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_quantisation_is_round_to_nearest_even(fmt):
    rng = np.random.default_rng(5)
    blocks = [rng.standard_normal(32) * s for s in (1e-3, 1.0, 300.0, 1e30, 1e-40)]
    blocks.append(np.arange(-16, 16) / 4.0)                       # halves and quarters: ties
    blocks.append(np.concatenate([[7.9, -7.9, 6.0, 5.0, 4.99], np.zeros(27)]))  # above the largest code
    blocks.append(np.zeros(32))
    blocks.append(np.full(32, -0.0))
    blocks.append(np.concatenate([[3.4e38, 1.2e-38], np.full(30, 2.0**-149)]))
    blocks.append(np.concatenate([[480.0, 449.0, -464.0, 2.0**-10], np.full(28, 2.0**-10 * 1.5)]))
    x = np.stack(blocks).astype(np.float32)
    codes, scales = oracle.quantize_rows(x, fmt)
    got = oracle.dequant_rows(codes, scales, fmt)
    for i in range(len(x)):
        want, s = _by_hand(x[i], fmt)
        assert scales[i, 0] == s, (i, scales[i, 0], s)
        assert [Fraction(float(v)) for v in got[i]] == want, i
    assert np.array_equal(np.signbit(got), np.signbit(x))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8", "q8_1"])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_blocks_with_infinities_and_nans(fmt, bad):
    x = np.ones((2, 96), dtype=np.float32)
    x[0, 40] = bad
    codes, scales = oracle.quantize_rows(x, fmt)
    v = oracle.dequant_rows(codes, scales, fmt)
    assert np.isnan(v[0, 32:64]).all() and np.isfinite(v[1]).all() and np.isfinite(v[0, :32]).all()
    assert not np.any(np.asarray(codes).reshape(2, 3, -1)[0, 1])


def test_norm_steps():
    x = np.array([[3.0, -4.0] + [0.0] * 30], dtype=np.float64)
    gain = np.linspace(0.5, 2, 32).astype(np.float32)
    h, y = oracle.rmsnorm(x, None, gain, 1e-6, None)
    mean = Fraction(25, 32) + Fraction(float(np.float32(1e-6)))
    u = f32(Fraction(1 / float(mean) ** 0.5))  # 1 / sqrt to 2^-52, far from a binary32 midpoint here
    for i, v in enumerate((3, -4)):
        assert y[0, i] == f32(Fraction(f32(Fraction(v) * Fraction(u))) * Fraction(float(gain[i])))
    h, _ = oracle.rmsnorm(x, x * 1e-4, gain, 1e-6, lambda v: v.astype(np.float16).astype(np.float64))
    assert h[0, 0] == f16(Fraction(3) + Fraction(3 * 1e-4))


def test_product_is_plain():
    w = np.array([[1.0, 2.0], [0.5, -3.0], [0.0, 1.0]])
    x = np.array([[2.0, 1.0]])
    assert oracle.mx_product(w, x).tolist() == [[4.0, -2.0, 1.0]]
