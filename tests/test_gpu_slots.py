"""Tokens' rows into the experts' order and back on the GPU against the oracle.

A dispatched row is one binary32 product rounded once more to its type, and a combined one a
binary32 sum of such products in a fixed order: both are held to the same steps in numpy, bit for
bit.  A weight's gradient is a sum of `hidden` products in binary32, each addition (and its
product) off by at most half a step of the magnitudes' sum: hidden 2^-24 of it.
"""
import numpy as np
import pytest
import torch

import dequant_matmul_iq4_amd as iq4
import oracle
from gpu_util import dev, host, note
from rows_util import TYPES, floats, rounder

pytestmark = pytest.mark.gpu
F = np.float32


def slots(seed, tokens, top, n_rows, dropped):
    """slot_row [tokens, top]: every row at most once, some pairs without one (in several wordings)."""
    rng = np.random.default_rng(seed)
    s = rng.permutation(max(tokens * top, n_rows))[: tokens * top].reshape(tokens, top).astype(np.int32)
    s[s >= n_rows] = -1
    drop = rng.random(s.shape) < dropped
    s[drop] = rng.choice([-1, n_rows, n_rows + 7, 2**31 - 1, -(2**31)], int(drop.sum()))
    return s


def acts(seed, m, k, t):
    rng = np.random.default_rng(seed)
    return rounder(t)(rng.standard_normal((m, k)) * np.exp(rng.standard_normal((m, 1)))).astype(F)


CASES = [  # tokens, top, rows, hidden, share dropped
    (1, 1, 1, 1, 0.0), (3, 2, 9, 7, 0.3), (5, 8, 40, 64, 0.0), (4, 8, 32, 2048, 0.1), (33, 3, 90, 333, 0.2), (2, 16, 40, 4100, 0.0), (130, 5, 650, 40, 0.5),
    (7, 6, 30, 1000, 1.0), (300, 4, 1200, 8, 0.0), (1, 9, 12, 9001, 0.2)]
PAIRS = [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "bf16"), ("bf16", "f16"), ("f32", "f16"), ("bf16", "f32"), ("f16", "bf16")]


def _has(s, n_rows):
    return (s >= 0) & (s < n_rows)


@pytest.mark.parametrize("types", PAIRS, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("tokens,top,n_rows,hidden,dropped", CASES)
def test_dispatch(tokens, top, n_rows, hidden, dropped, types):
    tx, tr = types
    note(f"slots: dispatch {tokens} x {top} -> {n_rows} rows of {hidden}, {tx} -> {tr}")
    s = slots(tokens + hidden, tokens, top, n_rows, dropped)
    x = acts(hidden, tokens, hidden, tx)
    w = np.random.default_rng(1).random((tokens, top)).astype(F)
    for weights, ldx, ldr in ((None, hidden, hidden), (w, hidden + 3, hidden + 5)):
        xd = floats(x, tx, ldx)
        rows = torch.full((n_rows, ldr), -7.0, dtype=TYPES[tr][1], device="cuda")
        iq4.iq4_moe_dispatch(xd, TYPES[tx][0], ldx, tokens, hidden, dev(s), None if weights is None else dev(weights), top, n_rows, rows,
                             TYPES[tr][0], ldr)
        want = np.full((n_rows, ldr), -7.0)
        has = _has(s, n_rows)
        for t in range(tokens):
            for j in range(top):
                if has[t, j]:
                    want[s[t, j], :hidden] = rounder(tr)((x[t] if weights is None else w[t, j] * x[t]).astype(np.float64))
        assert np.array_equal(host(rows.double()), want)


def combined(x, s, w, add, n_rows):
    """The binary32 steps in the order of j."""
    has = _has(s, n_rows)
    out = np.zeros((s.shape[0], x.shape[1]), dtype=F)
    for j in range(s.shape[1]):
        v = x[np.where(has[:, j], s[:, j], 0)]
        v = v if w is None else w[:, j:j + 1] * v
        out = np.where(has[:, j:j + 1], out + v, out)
    return out if add is None else out + add


@pytest.mark.parametrize("types", PAIRS, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("tokens,top,n_rows,hidden,dropped", CASES)
def test_combine(tokens, top, n_rows, hidden, dropped, types):
    tr, to = types
    note(f"slots: combine {n_rows} rows of {hidden} -> {tokens} x {top}, {tr} -> {to}")
    s = slots(tokens + hidden, tokens, top, n_rows, dropped)
    x = acts(hidden, n_rows, hidden, tr)
    x[~np.isin(np.arange(n_rows), s)] = np.nan  # rows of no pair are not looked at
    add = acts(7, tokens, hidden, to)
    w = np.random.default_rng(1).random((tokens, top)).astype(F)
    for weights, addend, over in ((None, None, False), (w, None, False), (w, add, False), (None, add, True)):
        ld = hidden + 3
        rows = floats(x, tr, ld)
        ad = None if addend is None else floats(addend, to, ld)
        out = ad if over else torch.full((tokens, ld), -7.0, dtype=TYPES[to][1], device="cuda")
        iq4.iq4_moe_combine(rows, TYPES[tr][0], ld, n_rows, dev(s), None if weights is None else dev(weights), tokens, top, hidden, ad, ld, out,
                            TYPES[to][0], ld)
        got = host(out.double())
        want = combined(x, s, weights, addend, n_rows)
        assert np.array_equal(got[:, :hidden], rounder(to)(want.astype(np.float64)))
        assert np.isnan(got[:, hidden:]).all() if over else np.all(got[:, hidden:] == -7.0)
        exact = oracle.moe_combine(np.nan_to_num(x), s, weights, addend)
        mags = oracle.moe_combine(abs(np.nan_to_num(x)), s, weights, None if addend is None else abs(addend))
        assert np.all(abs(want - exact) <= (2 * top + 1) * 2.0**-24 * mags)


@pytest.mark.parametrize("types", PAIRS, ids=lambda p: "-".join(p))
@pytest.mark.parametrize("tokens,top,n_rows,hidden,dropped", CASES)
def test_combine_grad(tokens, top, n_rows, hidden, dropped, types):
    td, tr = types
    note(f"slots: gradient of combine, {n_rows} rows of {hidden}, {tokens} x {top}, {td}, {tr}")
    s = slots(tokens + hidden, tokens, top, n_rows, dropped)
    x, do = acts(hidden, n_rows, hidden, tr), acts(hidden + 1, tokens, hidden, td)
    w = np.random.default_rng(1).random((tokens, top)).astype(F)
    has = _has(s, n_rows)
    for weights, want_rows, want_dw in ((w, True, True), (None, True, True), (w, True, False), (w, False, True)):
        ld = hidden + 5
        drows = torch.full((n_rows, ld), -7.0, dtype=TYPES[tr][1], device="cuda")
        dw = torch.full((tokens, top), -7.0, device="cuda")
        dod = floats(do, td, ld)
        iq4.iq4_moe_combine_grad(dod, TYPES[td][0], ld, floats(x, tr, ld) if want_dw else None, TYPES[tr][0], ld, n_rows, dev(s),
                                 None if weights is None else dev(weights), tokens, top, hidden, drows if want_rows else None, ld,
                                 dw if want_dw else None)
        want = np.full((n_rows, ld), -7.0)
        if want_rows:
            for t in range(tokens):
                for j in range(top):
                    if has[t, j]:
                        want[s[t, j], :hidden] = rounder(tr)((do[t] if weights is None else w[t, j] * do[t]).astype(np.float64))
        assert np.array_equal(host(drows.double()), want)
        if want_dw:
            exact = oracle.moe_combine_grad(do, x, s, weights)[1]
            mags = oracle.moe_combine_grad(abs(do), abs(x), s, weights)[1]
            assert np.all(abs(host(dw) - exact) <= (hidden + 1) * 2.0**-24 * mags)
        else:
            assert np.all(host(dw) == -7.0)


def test_gradients_against_differences():
    """The kernels' gradients against central differences of the oracle's combine."""
    note("slots: gradients against differences")
    tokens, top, n_rows, hidden, step = 4, 3, 11, 6, 1e-5
    s = slots(5, tokens, top, n_rows, 0.2)
    x, do = acts(1, n_rows, hidden, "f32").astype(np.float64), acts(2, tokens, hidden, "f32").astype(np.float64)
    w = np.random.default_rng(3).random((tokens, top)).astype(F).astype(np.float64)
    drows, dw = torch.zeros(n_rows, hidden, device="cuda"), torch.zeros(tokens, top, device="cuda")
    iq4.iq4_moe_combine_grad(floats(do, "f32"), 0, hidden, floats(x, "f32"), 0, hidden, n_rows, dev(s), dev(w.astype(F)), tokens, top, hidden,
                             drows, hidden, dw)

    def slope(f, v):
        out = np.zeros(v.shape)
        for i in np.ndindex(v.shape):
            a, b = v.copy(), v.copy()
            a[i], b[i] = a[i] + step, b[i] - step
            out[i] = (f(a) - f(b)) / (2 * step)
        return out

    # linear in each argument: the difference is off by its own roundings, 2^-53 of the values over the step
    want = slope(lambda v: (oracle.moe_combine(v, s, w) * do).sum(), x)
    assert np.abs(host(drows) - want).max() <= 1e-6 * np.abs(want).max()
    want = slope(lambda v: (oracle.moe_combine(x, s, v) * do).sum(), w)
    assert np.abs(host(dw) - want).max() <= 1e-6 * np.abs(want).max()
    dx = torch.zeros(tokens, hidden, device="cuda")
    iq4.iq4_moe_combine(floats(x, "f32"), 0, hidden, n_rows, dev(s), None, tokens, top, hidden, None, 0, dx, 0, hidden)
    want = slope(lambda v: (oracle.moe_dispatch(v, s, None, np.zeros((n_rows, hidden))) * x).sum(), np.zeros((tokens, hidden)))
    assert np.abs(host(dx) - want).max() <= 1e-6 * np.abs(want).max()


@pytest.mark.parametrize("t", list(TYPES))
def test_infinities_and_nan_stay_where_they_are(t):
    note(f"slots: infinities and NaN, {t}")
    s = np.array([[0, 1], [2, -1], [3, 4]], dtype=np.int32)
    x = np.ones((5, 9), dtype=F)
    x[1, 2], x[2, 3] = np.inf, np.nan
    out = torch.zeros(3, 9, dtype=TYPES[t][1], device="cuda")
    w = np.array([[0.0, 1.0], [1.0, 5.0], [2.0, np.inf]], dtype=F)
    iq4.iq4_moe_combine(floats(x, t), TYPES[t][0], 9, 5, dev(s), dev(w), 3, 2, 9, None, 0, out, TYPES[t][0], 9)
    want = np.ones((3, 9))
    want[0, 2], want[1, 3], want[2] = np.inf, np.nan, np.inf
    assert np.array_equal(host(out.double()), want, equal_nan=True)


def test_no_rows_at_all():
    note("slots: every pair dropped, no rows")
    s = np.full((3, 2), -1, dtype=np.int32)
    w = np.ones((3, 2), dtype=F)
    out = torch.full((3, 5), 7.0, device="cuda")
    iq4.iq4_moe_combine(None, 0, 0, 0, dev(s), dev(w), 3, 2, 5, None, 0, out, 0, 5)
    dw = torch.full((3, 2), 7.0, device="cuda")
    iq4.iq4_moe_combine_grad(out, 0, 5, None, 0, 0, 0, dev(s), dev(w), 3, 2, 5, None, 0, dw)
    assert not host(out).any() and not host(dw).any()
