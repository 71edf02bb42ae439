"""The oracle of the expert layer's further operators against small cases worked out by hand
and against central differences in 64 bits."""
import numpy as np

import oracle


def test_g4_weights_by_hand():
    codes = np.array([[0x21, 0xF0] + [0x88] * 14 + [0x10] * 16], dtype=np.uint8)  # 1 2 0 15 8 8 .. | 0 1 0 1 ..
    w = oracle.g4_weights(codes, np.array([[0.5, 2.0]]), None, 32)
    assert w.shape == (1, 64)
    assert w[0, :6].tolist() == [-3.5, -3.0, -4.0, 3.5, 0.0, 0.0] and w[0, 32:36].tolist() == [-16.0, -14.0, -16.0, -14.0]
    w = oracle.g4_weights(codes, np.array([[0.5]]), np.array([[15]], dtype=np.uint8), 128)  # a short last group
    assert w[0, :4].tolist() == [-7.0, -6.5, -7.5, 0.0] and w[0, 63] == -7.0


def test_slots_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    slot = np.array([[2, 0], [-1, 1]])
    w = np.array([[0.5, 2.0], [7.0, 3.0]])
    rows = oracle.moe_dispatch(x, slot, w, np.full((4, 2), 9.0))
    assert rows.tolist() == [[2, 4], [9, 12], [0.5, 1], [9, 9]]
    assert oracle.moe_combine(rows, slot, w).tolist() == [[4.25, 8.5], [27, 36]]
    assert oracle.moe_combine(rows, slot, None, x).tolist() == [[3.5, 7], [12, 16]]
    assert oracle.moe_combine(rows, np.full((1, 3), -1), None).tolist() == [[0, 0]]


def _difference(f, x, h=1e-6):
    out = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        out[i] = (f(a) - f(b)) / (2 * h)
    return out


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(1)
    rows, w, do = rng.standard_normal((5, 3)), rng.random((3, 2)), rng.standard_normal((3, 3))
    slot = np.array([[4, 0], [-1, 2], [3, 9]])  # 9: no such row
    drows, dw = oracle.moe_combine_grad(do, rows, slot, w)
    want = _difference(lambda r: (oracle.moe_combine(r, slot, w) * do).sum(), rows)
    assert np.allclose(np.nan_to_num(drows), want, atol=1e-8) and np.isnan(drows[1]).all()
    assert np.allclose(dw, _difference(lambda v: (oracle.moe_combine(rows, slot, v) * do).sum(), w), atol=1e-8)
    # a dispatch's gradient is the combine without weights
    x = rng.standard_normal((3, 3))
    dr = rng.standard_normal((5, 3))
    want = _difference(lambda v: (oracle.moe_dispatch(v, slot, None, np.zeros((5, 3))) * dr).sum(), x)
    assert np.allclose(oracle.moe_combine(dr, slot, None), want, atol=1e-8)


def test_swiglu_and_gradient_against_differences():
    assert oracle.swiglu([0.0, 1.0], [5.0, 2.0]).tolist() == [0.0, 2.0 / (1.0 + np.exp(-1.0))]
    rng = np.random.default_rng(2)
    g, u, dh = (2 * rng.standard_normal((4, 5)) for _ in range(3))
    dg, du = oracle.swiglu_grad(dh, g, u)
    assert np.allclose(dg, _difference(lambda v: (oracle.swiglu(v, u) * dh).sum(), g), atol=1e-7)
    assert np.allclose(du, _difference(lambda v: (oracle.swiglu(g, v) * dh).sum(), u), atol=1e-7)
