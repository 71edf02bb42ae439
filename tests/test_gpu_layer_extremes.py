"""The group-scaled products, the experts' rows and SwiGLU where values lie at the ends of their types, or
past them."""
import numpy as np
import pytest
import torch

import dequant_matmul_iq4_amd as iq4
import oracle
from gpu_util import dev, host, note
from rows_util import FMT, HALF_STEP, TYPES, floats, row_buffers, rounder, same_rows
from test_gpu_g4 import bank, pack, weights

pytestmark = pytest.mark.gpu
F = np.float32


# ---- SwiGLU -------------------------------------------------------------------------------


def deep(seed, m, k, t):
    """Gates from -75 to -180 (and some beyond), and values and gradients of any size the type has."""
    rng = np.random.default_rng(seed)
    top = 14 if t == "f16" else 126
    g = rounder(t)(-rng.uniform(75, 180, (m, k)))
    g.reshape(-1)[:: 7] = rounder(t)(rng.choice([-80.0, -88.0, -88.72, -91.8, -1000.0, -60000.0, 3.0], g.reshape(-1)[:: 7].shape))
    wide = lambda: rounder(t)(rng.choice([1, -1], (m, k)) * 2.0 ** rng.uniform(-14, top, (m, k)))  # noqa: E731
    return g, wide(), wide()


def _step(t):
    """Half a step of the type's subnormal numbers."""
    f = torch.finfo(TYPES[t][1])
    return float(f.smallest_normal) * float(f.eps) / 2


@pytest.mark.parametrize("t,y_t", [("f32", "f32"), ("bf16", "f32"), ("f16", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16")])
def test_swiglu_of_deeply_closed_gates(t, y_t):
    """silu(g) falls to 2^-126 at -91.8 and is a part of h below: 2^-20 of h, as everywhere, and a rounding (2^-150 more
    for the binary32 value behind one of 16 bits)."""
    note(f"extremes: SwiGLU of closed gates, {t} -> {y_t}")
    m, k = 9, 133
    g, u, _ = deep(1, m, k, t)
    y = torch.full((m, k), -7.0, dtype=TYPES[y_t][1], device="cuda")
    iq4.iq4_swiglu(floats(g, t), k, floats(u, t), k, TYPES[t][0], m, k, y, TYPES[y_t][0], k)
    got, want = host(y.double()), oracle.swiglu(g, u)
    assert y_t == "f16" or (np.abs(want[g < -88]) > float(torch.finfo(TYPES[y_t][1]).smallest_normal)).sum() > 50
    assert np.all(abs(want) < float(torch.finfo(TYPES[y_t][1]).max))
    assert np.all(abs(got - want) <= (2.0**-20 + HALF_STEP[y_t]) * abs(want) + _step(y_t) + 2.0**-150)


@pytest.mark.parametrize("dt,t", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("bf16", "f32")])
def test_swiglu_gradient_of_deeply_closed_gates(dt, t):
    """The same of the gradients, where 1 + g (1 - s) is 1 + g (or, at three, off by 2^-20 of 1 + |g|)."""
    note(f"extremes: SwiGLU's gradient of closed gates, {dt}, {t}")
    m, k = 9, 133
    g, u, _ = deep(2, m, k, t)
    dh = deep(3, m, k, dt)[2]
    dh *= np.where(abs(dh * u) > 2.0**120, 2.0**-126, 1)  # (dh u is a binary32 number)
    dh = rounder(dt)(dh)
    dg, du = (torch.full((m, k), -7.0, dtype=TYPES[t][1], device="cuda") for _ in range(2))
    iq4.iq4_swiglu_grad(floats(dh, dt), TYPES[dt][0], k, floats(g, t), k, floats(u, t), k, TYPES[t][0], m, k, dg, k, du, k)
    wg, wu = oracle.swiglu_grad(dh, g, u)
    small = _step(t) + 2.0**-149  # (and of one product on the way where the gate is open)
    assert np.all(abs(host(du.double()) - wu) <= (2.0**-20 + HALF_STEP[t]) * abs(wu) + small)
    assert np.all(abs(host(dg.double()) - wg) <= (2.0**-18 + HALF_STEP[t]) * abs(wg) + small)
    assert ((g < -88) & (abs(wg) > 2.0**-126)).sum() > 50 and ((g < -88) & (abs(wu) > 2.0**-126)).sum() > 50


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_quantised_rows_of_deeply_closed_gates(fmt):
    note(f"extremes: SwiGLU of closed gates -> {fmt}")
    m, k = 5, 160
    g, u, _ = deep(4, m, k, "bf16")
    q, d, ldq, lds = row_buffers(fmt, m, k)
    y = torch.zeros(m, k, device="cuda")
    iq4.iq4_swiglu(floats(g, "bf16"), k, floats(u, "bf16"), k, iq4.IQ4_BF16, m, k, y, iq4.IQ4_F32, k, FMT[fmt], q, ldq, d, lds)
    same_rows(fmt, k, q, d, oracle.quantize_rows(host(y), fmt))
    want = oracle.swiglu(g, u)
    assert np.all(abs(host(y) - want) <= 2.0**-19 * abs(want) + 2.0**-149)


# ---- experts' rows ------------------------------------------------------------------------


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("top", [1, 9])
@pytest.mark.parametrize("hidden", [3, 9, 37, 70, 131, 261, 1093])
def test_an_infinity_at_every_place_of_a_row(hidden, top, t):
    """dw of a row (or of a gradient) with an infinity anywhere is that infinity, where the kernel reads a place twice too."""
    note(f"extremes: gradient of combine, an infinity in rows of {hidden}, top {top}, {t}")
    rng = np.random.default_rng(hidden)
    tokens = -(-hidden // top)
    n = tokens * top
    slot = rng.permutation(n).astype(np.int32).reshape(tokens, top)
    x, do = (rounder(t)(rng.choice([1, -1], s) * rng.uniform(0.5, 2, s)) for s in ((n, hidden), (tokens, hidden)))
    at = np.arange(n) % hidden
    rows = x.copy()
    rows[slot.reshape(-1), at] = np.inf

    def dw_of(d, r):
        dw = torch.full((tokens, top), -7.0, device="cuda")
        iq4.iq4_moe_combine_grad(floats(d, t), TYPES[t][0], hidden, floats(r, t), TYPES[t][0], hidden, n, dev(slot), None, tokens, top, hidden, None,
                                 0, dw)
        return host(dw)

    assert np.array_equal(dw_of(do, rows), (np.repeat(do, top, 0)[np.arange(n), at] * np.inf).reshape(tokens, top))
    for i in range(0, hidden, 1 + hidden // 40):
        d = do.copy()
        d[:, i] = -np.inf
        assert np.array_equal(dw_of(d, x), -np.inf * x[slot][:, :, i])
        r = x.copy()
        r[:, i] = np.nan
        assert np.isnan(dw_of(do, r)).all()


# ---- group-scaled products ----------------------------------------------------------------


def _product(p, n, k, group, z, x, t, y_t="f32"):
    y = torch.full((len(x), n), -7.0, dtype=TYPES[y_t][1], device="cuda")
    iq4.iq4_g4_qmv(p, n, k, group, iq4.IQ4_F16, z is not None, floats(x, t), TYPES[t][0], k, len(x), y, TYPES[y_t][0], n)
    return host(y.double())


# one operand of rows and two; short rows, long ones, ones in slices; a last group, row tile and code tile that are not full
ODD = [(33, 544, 32, 3), (33, 544, 32, 20), (2100, 4096, 64, 33), (4100, 160, 128, 21), (600, 8768, 32, 17), (70, 6240, 128, 5), (2105, 2048, 32, 70)]


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n,k,group,m", ODD)
def test_infinities_and_nan_in_every_form_of_the_product(n, k, group, m, t):
    """Rows with an infinity, with two of either sign, with a NaN, with the largest numbers: each result what the formula says, the
    other rows' whole numbers exact."""
    note(f"extremes: infinities and NaN, {m} x {n} x {k} by {group}, {t}")
    codes, s, z = weights(n + k, n, k, group, True, "f16", True)
    p, w = pack(codes, s, z, group, "f16"), oracle.g4_weights(codes, s, z, group)
    rng = np.random.default_rng(m)
    x = rng.integers(-4, 5, (m, k)).astype(np.float64)
    for y_t in ("f32", t):
        inf, both, nan = rng.permutation(m)[:3]
        v = x.copy()
        i, j, l = rng.integers(0, k, 3)
        v[inf, i], v[both, j], v[both, (j + k // 2) % k], v[nan, l] = -np.inf, np.inf, -np.inf, np.nan
        got = _product(p, n, k, group, z, v, t, y_t)
        rest = np.delete(np.arange(m), [inf, both, nan])
        assert np.array_equal(got[rest], rounder(y_t)(oracle.g4_product(w, v[rest])))
        assert np.isnan(got[nan]).all()
        with np.errstate(invalid="ignore"):
            assert np.array_equal(got[inf], -np.inf * w[:, i], equal_nan=True)
            assert np.array_equal(got[both], np.inf * w[:, j] - np.inf * w[:, (j + k // 2) % k], equal_nan=True)


def test_large_bfloat16_sums_that_cancel():
    """The terms that 16 + q makes pass binary32's largest number where those of q - z do not."""
    note("extremes: bfloat16 values near the largest")
    n, k, group, m = 50, 1024, 64, 18
    codes, s, z = weights(3, n, k, group, True, "f16", True)
    p, w = pack(codes, s, z, group, "f16"), oracle.g4_weights(codes, s, z, group)
    x = np.random.default_rng(4).integers(-4, 5, (m, k)).astype(np.float64)
    x[::3] *= 2.0**113  # |y| <= 1024 * 30 * 4 * 2^113 < 2^128
    assert np.array_equal(_product(p, n, k, group, z, x, "bf16"), rounder("f32")(oracle.g4_product(w, x)))
    x[1::3] *= 2.0**124
    got, want = _product(p, n, k, group, z, x, "bf16"), oracle.g4_product(w, x)
    with np.errstate(over="ignore"):
        assert np.array_equal(got, want.astype(F))
    assert np.isinf(got[1::3]).any() and np.isfinite(got[1::3]).any()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("n,k,group,m", ODD)
def test_scales_near_the_largest_number(n, k, group, m, t):
    """Scales of some 2^105 by values of some 2^-100, results of ordinary size: every product and sum is a binary32 number,
    whatever power of two the values are held with on the way.  (The bfloat16 kernel holds them as they are.)"""
    note(f"extremes: scales of 2^105, {m} x {n} x {k} by {group}, {t}")
    codes, s, z = weights(n * k, n, k, group, True, "bf16", True)
    p, w = pack(codes, s * 2.0**105, z, group, "bf16"), oracle.g4_weights(codes, s * 2.0**105, z, group)
    x = np.random.default_rng(m).integers(-4, 5, (m, k)) * 2.0**-100
    x[1::3] *= 2.0**90   # |y| < 2^(105 + 23 - 10)
    x[2::3] *= 2.0**-27  # (2^-127 .. 2^-125: subnormal)
    y = torch.full((m, n), -7.0, device="cuda")
    iq4.iq4_g4_qmv(p, n, k, group, iq4.IQ4_BF16, 1, floats(x, t), TYPES[t][0], k, m, y, iq4.IQ4_F32, n)
    assert np.array_equal(host(y), oracle.g4_product(w, x))


@pytest.mark.parametrize("n,k,group,m", ODD)
def test_a_large_activation_without_a_weight(n, k, group, m):
    """A column of X 2^26 times the others, whose weights are all zero: the others keep their bits (2^-23 of each, or 2^-50 of
    the largest, 2^-24 here).  The errors are of either sign, so their norm shows what a sum of bounds would hide."""
    note(f"extremes: a large activation without a weight, {m} x {n} x {k} by {group}")
    codes, s, z = weights(n + m, n, k, group, False, "f16", False)
    rng = np.random.default_rng(k)
    at = rng.permutation(k // 2)[: 1 + k // 500]  # bytes of two weights each
    codes[:, at] = 0x88
    x = rng.standard_normal((m, k)).astype(F).astype(np.float64)
    x[:, 2 * at] = rng.choice([1, -1], (m, len(at))) * 2.0**26
    y = torch.full((m, n), -7.0, device="cuda")
    iq4.iq4_g4_qmv(pack(codes, s, None, group, "f16"), n, k, group, iq4.IQ4_F16, 0, floats(x, "f32"), iq4.IQ4_F32, k, m, y, iq4.IQ4_F32, n)
    want = oracle.g4_product(oracle.g4_weights(codes, s, None, group), x)
    assert np.linalg.norm(host(y) - want) <= 1e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("what", [np.nan, np.inf])
@pytest.mark.parametrize("t", list(TYPES))
def test_rows_that_are_not_finite_cost_no_more_than_many_rows(t, what):
    """A batch whose padding holds NaN: a few times the call without (each such result once took a lane through all of k)."""
    note(f"extremes: time of rows that are {what}, {t}")
    n, k, group, m = 4096, 4096, 64, 16
    codes, s, z = weights(5, n, k, group, True, "f16", True)
    p = pack(codes, s, z, group, "f16")
    x = floats(np.ones((m, k)), t)
    bad = x.clone()
    bad[1:9, 77] = what
    y = torch.zeros(m, n, dtype=TYPES[t][1], device="cuda")
    times = []
    for v in (x, bad, x, bad):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        for i in range(6):
            if i == 1:
                a.record()
            iq4.iq4_g4_qmv(p, n, k, group, iq4.IQ4_F16, 1, v, TYPES[t][0], k, m, y, TYPES[t][0], n)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) / 5 * 1e3)
    note(f"  {times[2]:.1f} us, {times[3]:.1f} with them")
    assert times[3] <= (20 if np.isnan(what) else 100) * times[2]


def _offset_lists(e, m):
    rng = np.random.default_rng(e)
    yield np.linspace(0, m, e + 1).astype(int)
    yield np.concatenate([[-5], np.linspace(0, m, e).astype(int)])  # below the rows, and past them
    yield np.linspace(3, m + 90, e + 1).astype(int)
    yield np.sort(rng.choice([-(2**31), -1, 0, 9, m, m + 1, 2**31 - 1], e + 1))
    for v in (2**31 - 1, -(2**31), m):
        yield np.full(e + 1, v)
    yield np.linspace(m, 0, e + 1).astype(int)  # from here on they fall, somewhere at least
    for _ in range(3):
        yield rng.integers(-m, 2 * m, e + 1)
    yield rng.choice([2**31 - 1, -(2**31), 0, m], e + 1)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("e", [1, 4, 64, 130, 300])
def test_offsets_and_pairs_of_any_kind(e, t):
    """Offsets that ascend count within the rows, pair ids name a row of x whatever they are; rows without an expert are left
    alone, and what lies around the rows always."""
    n, k, group, m, top, around = 16, 32, 32, 61, 2, 40
    p, ws = bank(7, e, n, k, group, True, "f16")
    rng = np.random.default_rng(e)
    x = rng.integers(-4, 5, (-(-m // top), k)).astype(np.float64)
    for i, offsets in enumerate(_offset_lists(e, m)):
        note(f"extremes: {e} experts, offsets of kind {i}, {t}")
        pairs = rng.integers(0, m, m) if i % 2 else rng.choice([-1, 1000, 2**31 - 1, -(2**31), 7, -7], m)
        big = torch.full((m + 2 * around, n + 3), -7.0, device="cuda")
        y = big[around:]
        iq4.iq4_g4_grouped_qmv(p, e, n, k, group, iq4.IQ4_F16, 1, floats(x, t), TYPES[t][0], k, len(x), dev(offsets.astype(np.int32)),
                               dev(pairs.astype(np.int32)), top, m, y, iq4.IQ4_F32, n + 3)
        got = host(big)
        assert np.all(got[:around] == -7.0) and np.all(got[around + m:] == -7.0) and np.all(got[:, n:] == -7.0)
        if np.all(offsets[1:] >= offsets[:-1]):
            want = np.full((m, n), -7.0)
            at = offsets.clip(0, m)
            src = x[np.trunc(pairs / top).clip(0, len(x) - 1).astype(int)]
            for j in range(e):
                want[at[j]: at[j + 1]] = oracle.g4_product(ws[j], src[at[j]: at[j + 1]])
            assert np.array_equal(got[around: around + m, :n], want), i
