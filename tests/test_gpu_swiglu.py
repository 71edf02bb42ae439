"""SwiGLU and its gradient on the GPU against the oracle.

h: the power's argument carries its product's rounding along; then the power (one step, 2^-23),
its correction and the sum (half a step each), the reciprocal (one step), the products with g
and u (half a step each), and what the steps' own errors add up to: under 2^-20 of h.  The gradient
of g has the term 1 + g (1 - s), off by under 2^-20 of 1 + |g| s (1 - s is off by half a step of
one, and s by its own error), and two more products.  Where the sigmoid is below the smallest normal
number it counts as zero or as itself: 2^-125 |g u|.  Then half a step of the output's type.
"""
import numpy as np
import pytest
import torch

import dequant_matmul_iq4_amd as iq4
import oracle
from gpu_util import dev, host, note
from rows_util import FMT, HALF_STEP, TYPES, floats, row_buffers, rounder, same_rows, split_rows

pytestmark = pytest.mark.gpu
SHAPES = [(1, 1), (1, 32), (3, 7), (2, 96), (5, 130), (4, 768), (33, 544), (2, 14336), (300, 33)]


def inputs(seed, m, k, t):
    rng = np.random.default_rng(seed)
    g, u = rounder(t)(3 * rng.standard_normal((m, k))), rounder(t)(rng.standard_normal((m, k)))
    some = np.array([0.0, -0.0, 100.0, -100.0, -88.0, -87.0, 88.0, 30.0, -30.0, -1.2784645, 60000.0, -60000.0, 2.0**-14])
    at = rng.integers(0, m * k, min(m * k, 4 * len(some)))
    g.reshape(-1)[at] = rounder(t)(np.resize(some, len(at)))
    return g, u


def _small(t):
    """Half a step below the smallest normal number."""
    return float(torch.finfo(TYPES[t][1]).smallest_normal) * HALF_STEP[t] * 2


@pytest.mark.parametrize("t,y_t", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("m,k", SHAPES)
def test_forward(m, k, t, y_t):
    note(f"swiglu: {m} x {k} {t} -> {y_t}")
    g, u = inputs(m * k, m, k, t)
    y = torch.full((m, k + 3), -7.0, dtype=TYPES[y_t][1], device="cuda")
    gd, ud = floats(g, t, k + 1), floats(u, t, k + 2)
    iq4.iq4_swiglu(gd, k + 1, ud, k + 2, TYPES[t][0], m, k, y, TYPES[y_t][0], k + 3)
    got, want = host(y.double()), oracle.swiglu(g, u)
    assert np.all(got[:, k:] == -7.0)
    top = float(torch.finfo(TYPES[y_t][1]).max)
    fine = abs(want) < top
    bound = (2.0**-20 + HALF_STEP[y_t]) * abs(want) + 2.0**-125 * abs(g * u) + _small(y_t)
    assert np.all(abs(got[:, :k] - want)[fine] <= bound[fine]) and np.all(abs(got[:, :k])[~fine] >= top)
    # side by side in one buffer, as a product of gate and up weights leaves them
    both = floats(np.concatenate([g, u], 1), t)
    y2 = torch.zeros(m, k, dtype=TYPES[y_t][1], device="cuda")
    iq4.iq4_swiglu(both, 2 * k, both[:, k:], 2 * k, TYPES[t][0], m, k, y2, TYPES[y_t][0], k)
    assert np.array_equal(host(y2.double()), got[:, :k])


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("m,k", [(1, 32), (3, 96), (5, 544), (2, 4096), (70, 160)])
def test_quantised_rows(m, k, t, fmt):
    """The codes are those of the float32 values, bit for bit; the plain rows may come with them."""
    note(f"swiglu: {m} x {k} {t} -> {fmt}")
    g, u = inputs(m * k, m, k, t)
    g, u = np.clip(g, -200, 200), np.clip(u, -200, 200)
    if m > 2:
        u[2, 40] = np.inf if k > 40 else 1.0
    gd, ud = floats(g, t, k + 5), floats(u, t, k + 1)
    for with_y in (True, False):
        q, d, ldq, lds = row_buffers(fmt, m, k)
        y = torch.zeros(m, k, device="cuda") if with_y else None
        iq4.iq4_swiglu(gd, k + 5, ud, k + 1, TYPES[t][0], m, k, y, iq4.IQ4_F32, k, FMT[fmt], q, ldq, d, lds)
        if with_y:
            want = oracle.quantize_rows(host(y), fmt)
        same_rows(fmt, k, q, d, want)


@pytest.mark.parametrize("dt,t", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f16"), ("bf16", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("m,k", SHAPES)
def test_gradient(m, k, dt, t):
    note(f"swiglu: gradient {m} x {k} {dt}, {t}")
    g, u = inputs(m * k, m, k, t)
    dh = rounder(dt)(np.random.default_rng(4).standard_normal((m, k)))
    dg, du = (torch.full((m, k + 3), -7.0, dtype=TYPES[t][1], device="cuda") for _ in range(2))
    iq4.iq4_swiglu_grad(floats(dh, dt, k + 4), TYPES[dt][0], k + 4, floats(g, t, k + 1), k + 1, floats(u, t, k + 2), k + 2, TYPES[t][0], m, k, dg,
                        k + 3, du, k + 3)
    wg, wu = oracle.swiglu_grad(dh, g, u)
    a, b = host(dg.double()), host(du.double())
    assert np.all(a[:, k:] == -7.0) and np.all(b[:, k:] == -7.0)
    s = 1 / (1 + np.exp(-np.clip(g, -700, 700)))
    top = float(torch.finfo(TYPES[t][1]).max)
    fine = abs(wu) < top
    bu = (2.0**-20 + HALF_STEP[t]) * abs(wu) + 2.0**-125 * abs(g * dh) + _small(t)
    assert np.all(abs(b[:, :k] - wu)[fine] <= bu[fine]) and np.all(abs(b[:, :k])[~fine] >= top)
    bg = abs(dh * u) * s * 2.0**-20 * (2 + abs(g)) + HALF_STEP[t] * abs(wg) + 2.0**-125 * abs(dh * u) * (1 + abs(g)) + _small(t)
    assert np.all(abs(a[:, :k] - wg) <= bg)


def test_gradient_against_differences():
    note("swiglu: gradient against differences")
    rng = np.random.default_rng(5)
    m, k, step = 6, 40, 1e-5
    g, u, dh = (rng.standard_normal((m, k)).astype(np.float32).astype(np.float64) * 2 for _ in range(3))
    dg, du = torch.zeros(m, k, device="cuda"), torch.zeros(m, k, device="cuda")
    iq4.iq4_swiglu_grad(floats(dh, "f32"), 0, k, floats(g, "f32"), k, floats(u, "f32"), k, 0, m, k, dg, k, du, k)
    # element by element; the difference is off by step^2 / 6 of the third derivative and 2^-53 over the step
    wg = dh * (oracle.swiglu(g + step, u) - oracle.swiglu(g - step, u)) / (2 * step)
    wu = dh * (oracle.swiglu(g, u + step) - oracle.swiglu(g, u - step)) / (2 * step)
    assert np.abs(host(dg) - wg).max() <= 2e-6 * np.abs(wg).max() and np.abs(host(du) - wu).max() <= 2e-6 * np.abs(wu).max()


@pytest.mark.parametrize("t", list(TYPES))
def test_infinities_and_nan(t):
    note(f"swiglu: infinities and NaN, {t}")
    inf, nan = np.inf, np.nan
    g = np.array([[inf, -inf, nan, 1.0, 1.0, 0.0, inf, 1.0]])
    u = np.array([[2.0, 2.0, 2.0, inf, nan, inf, -1.0, 1.0]])
    y = torch.zeros(1, 8, device="cuda")
    iq4.iq4_swiglu(floats(g, t), 8, floats(u, t), 8, TYPES[t][0], 1, 8, y, iq4.IQ4_F32, 8)
    got = host(y)[0]
    # g = -inf: -inf * 0
    assert got[0] == inf and np.isnan(got[1]) and np.isnan(got[2]) and got[3] == inf and np.isnan(got[4]) and np.isnan(got[5]) and got[6] == -inf
    assert np.isfinite(got[7])
