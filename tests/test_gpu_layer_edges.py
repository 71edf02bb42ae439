"""Where the group-scaled products, the experts' rows and SwiGLU could go wrong by their sizes: places past
2^31 elements and 2^32 bytes, grids with more than one column, buffers off their natural address, values
of very different magnitude."""
import numpy as np
import pytest
import torch

import dequant_matmul_iq4_amd as iq4
import oracle
from gpu_util import dev, host, note
from rows_util import TYPES, floats, rounder
from test_gpu_g4 import pack, weights

pytestmark = pytest.mark.gpu
F = np.float32
FAR = (1 << 31) + 24  # elements between two rows
HALF = iq4.IQ4_F16


def far_rows(m, k, seed=0):
    """Rows of small whole numbers FAR elements apart (binary16)."""
    b = torch.empty(FAR * (m - 1) + k, dtype=torch.float16, device="cuda")
    v = np.random.default_rng(seed).integers(-4, 5, (m, k)).astype(F)
    for i in range(m):
        b[i * FAR: i * FAR + k] = dev(v[i]).half()
    return b, v.astype(np.float64)


def near(b, m, k):
    torch.cuda.synchronize()
    return np.stack([host(b[i * FAR: i * FAR + k].double()) for i in range(m)])


def test_products_of_rows_far_apart():
    note("edges: rows of the products 2^31 elements apart")
    n, k, m = 48, 256, 3
    codes, s, z = weights(1, n, k, 32, True, "f16", True)
    p, w = pack(codes, s, z, 32, "f16"), oracle.g4_weights(codes, s, z, 32)
    x, xs = far_rows(m, k)
    y, _ = far_rows(m, n)
    iq4.iq4_g4_qmv(p, n, k, 32, HALF, 1, x, HALF, FAR, m, y, HALF, FAR)
    want = rounder("f16")(oracle.g4_product(w, xs))
    assert np.array_equal(near(y, m, n), want)
    y.zero_()
    iq4.iq4_g4_grouped_qmv(p, 1, n, k, 32, HALF, 1, x, HALF, FAR, m, dev(np.array([0, m], dtype=np.int32)), None, 1, m, y, HALF, FAR)
    assert np.array_equal(near(y, m, n), want)


def test_experts_far_into_a_bank():
    """1024 experts of over 4 MB: the last ones lie past 2^32 bytes."""
    note("edges: a bank of more than 4 GiB")
    n, k, e = 4096, 2048, 1024
    each = iq4.iq4_g4_packed_bytes(n, k, 128, 1)
    assert each * (e - 1) > 1 << 32
    p = torch.zeros(e * each, dtype=torch.uint8, device="cuda")
    ws = {}
    for i in (0, 511, 1022, 1023):
        codes, s, z = weights(i, n, k, 128, True, "bf16", True)
        pack(codes, s, z, 128, "bf16", p[i * each:(i + 1) * each])
        ws[i] = oracle.g4_weights(codes, s, z, 128)
    x = np.random.default_rng(3).integers(-4, 5, (4, k)).astype(np.float64)
    offsets = np.zeros(e + 1, dtype=np.int32)
    for j, i in enumerate(ws):
        offsets[i + 1:] = j + 1
    y = torch.zeros(4, n, device="cuda")
    iq4.iq4_g4_grouped_qmv(p, e, n, k, 128, iq4.IQ4_BF16, 1, floats(x, "bf16"), iq4.IQ4_BF16, k, 4, dev(offsets), None, 1, 4, y, iq4.IQ4_F32, n)
    assert np.array_equal(host(y), np.stack([oracle.g4_product(w, v[None])[0] for w, v in zip(ws.values(), x)]))


@pytest.mark.parametrize("t", list(TYPES))
def test_a_million_rows(t):
    """More tiles of rows than a grid has in one dimension."""
    note(f"edges: a product of 1.1 million rows, {t}")
    n, k, m = 3, 32, 1_100_003
    codes, s, z = weights(2, n, k, 32, True, "f16", True)
    w = oracle.g4_weights(codes, s, z, 32)
    x = torch.randint(-4, 5, (m, k), device="cuda").to(TYPES[t][1])
    y = torch.full((m, n), -7.0, device="cuda")
    iq4.iq4_g4_qmv(pack(codes, s, z, 32, "f16"), n, k, 32, HALF, 1, x, TYPES[t][0], k, m, y, iq4.IQ4_F32, n)
    assert np.array_equal(host(y), oracle.g4_product(w, host(x.double())))


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("m", [1, 9, 40])
def test_activations_off_their_natural_address(m, t):
    note(f"edges: activations one element off, {m} rows, {t}")
    n, k = 35, 1568
    codes, s, z = weights(4, n, k, 32, False, "f16", True)
    x = np.random.default_rng(5).integers(-4, 5, (m, k)).astype(np.float64)
    ld = k + 1
    b = torch.full((m * ld + 1,), float("nan"), dtype=TYPES[t][1], device="cuda")
    b[1:].view(m, ld)[:, :k] = dev(x).to(TYPES[t][1])
    y = torch.full((m * (n + 2) + 1,), -7.0, dtype=TYPES[t][1], device="cuda")
    iq4.iq4_g4_qmv(pack(codes, s, z, 32, "f16"), n, k, 32, HALF, 0, b[1:], TYPES[t][0], ld, m, y[1:], TYPES[t][0], n + 2)
    got = host(y.double())
    assert got[0] == -7.0 and np.all(got[1:].reshape(m, n + 2)[:, n:] == -7.0)
    assert np.array_equal(got[1:].reshape(m, n + 2)[:, :n], rounder(t)(oracle.g4_product(oracle.g4_weights(codes, s, z, 32), x)))


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("m", [2, 20])
def test_one_large_activation_among_small_ones(m, t):
    """What is said of an activation's precision: of binary32, 2^-23 of itself or 2^-39 of the largest of its slice,
    and sums of terms of |w x|; of bfloat16, sums of terms of |s (16 + q) x| and |s (16 + z) x|."""
    note(f"edges: one large activation, {m} rows, {t}")
    n, k, group = 64, 2048, 64
    codes, s, z = weights(6, n, k, group, True, "bf16", False)
    rng = np.random.default_rng(7)
    x = rng.standard_normal((m, k))
    x[np.arange(m), rng.integers(0, k, m)] = rng.choice([1e4, -1e6], m)
    x = rounder(t)(x.astype(F))
    w = oracle.g4_weights(codes, s, z, group)
    got = np.zeros((m, n))
    y = torch.zeros(m, n, device="cuda")
    iq4.iq4_g4_qmv(pack(codes, s, z, group, "bf16"), n, k, group, iq4.IQ4_BF16, 1, floats(x, t), TYPES[t][0], k, m, y, iq4.IQ4_F32, n)
    got, want = host(y), oracle.g4_product(w, x)
    if t == "f32":
        mags = oracle.g4_product(abs(w), abs(x))
        own = 2.0**-23 * mags + 2.0**-39 * abs(x).max(1, keepdims=True) * abs(w).sum(1)
    else:
        q = np.stack((codes & 15, codes >> 4), 2).reshape(n, k)
        wide = lambda v: np.repeat(v, group, axis=1)  # noqa: E731
        mags = oracle.g4_product(abs(wide(s)) * (32 + q + wide(z)), abs(x))
        own = 0
    assert np.all(abs(got - want) <= (1.001 * (k + 2 * k / 32) + 64) * 2.0**-23 * mags + own)


@pytest.mark.parametrize("H", [40, 700, 2060])
def test_rows_to_experts_and_back_far_apart(H):
    note(f"edges: experts' rows of {H}, 2^31 elements apart")
    T, top, n = 2, 2, 3
    slot = np.array([[2, 0], [1, 2]], dtype=np.int32)  # row 2 has two pairs: combine reads it for both
    w = np.array([[1.0, 2.0], [0.5, 4.0]], dtype=F)
    x, xs = far_rows(T, H, 1)
    rows, rs = far_rows(n, H, 2)
    out = torch.zeros(T, H, device="cuda")
    iq4.iq4_moe_combine(rows, HALF, FAR, n, dev(slot), dev(w), T, top, H, None, 0, out, iq4.IQ4_F32, H)
    assert np.array_equal(host(out), oracle.moe_combine(rs, slot, w))
    far = torch.empty(FAR + H, dtype=torch.float16, device="cuda")
    iq4.iq4_moe_combine(rows, HALF, FAR, n, dev(slot), dev(w), T, top, H, x, FAR, far, HALF, FAR)
    assert np.array_equal(near(far, T, H), oracle.moe_combine(rs, slot, w, xs))
    dw = torch.zeros(T, top, device="cuda")
    iq4.iq4_moe_combine_grad(x, HALF, FAR, rows, HALF, FAR, n, dev(slot), dev(w), T, top, H, None, 0, dw)
    assert np.array_equal(host(dw), oracle.moe_combine_grad(xs, rs, slot, w)[1])
    slot[1, 1] = -1
    for weights_ in (None, w):
        rows.zero_()
        iq4.iq4_moe_dispatch(x, HALF, FAR, T, H, dev(slot), None if weights_ is None else dev(weights_), top, n, rows, HALF, FAR)
        assert np.array_equal(near(rows, n, H), oracle.moe_dispatch(xs, slot, weights_, np.zeros((n, H))))


def test_swiglu_of_rows_far_apart():
    note("edges: SwiGLU of rows 2^31 elements apart")
    m, k = 2, 40
    g, gs = far_rows(m, k, 1)
    u, us = far_rows(m, k, 2)
    y, dg, du = (torch.empty(FAR + k, dtype=torch.float16, device="cuda") for _ in range(3))
    iq4.iq4_swiglu(g, FAR, u, FAR, HALF, m, k, y, HALF, FAR)
    near_y = torch.zeros(m, k, dtype=torch.float16, device="cuda")
    a, b = floats(gs, "f16"), floats(us, "f16")
    iq4.iq4_swiglu(a, k, b, k, HALF, m, k, near_y, HALF, k)
    assert np.array_equal(near(y, m, k), host(near_y.double()))
    iq4.iq4_swiglu_grad(y, HALF, FAR, g, FAR, u, FAR, HALF, m, k, dg, FAR, du, FAR)
    ng, nu = torch.zeros_like(near_y), torch.zeros_like(near_y)
    iq4.iq4_swiglu_grad(near_y, HALF, k, a, k, b, k, HALF, m, k, ng, k, nu, k)
    assert np.array_equal(near(dg, m, k), host(ng.double())) and np.array_equal(near(du, m, k), host(nu.double()))


def test_many_elements():
    """More than 2^31 elements of a call, and of its pairs."""
    note("edges: SwiGLU of 2^31 elements and more, a million tokens of eight pairs")
    m, k = 270_001, 8193
    g = torch.randn(m, k, device="cuda", dtype=torch.bfloat16)
    y = torch.zeros(m, k, device="cuda", dtype=torch.bfloat16)
    iq4.iq4_swiglu(g, k, g, k, iq4.IQ4_BF16, m, k, y, iq4.IQ4_BF16, k)
    some = [0, 1, m // 2, m - 2, m - 1]
    got, want = host(y[some].double()), oracle.swiglu(host(g[some].double()), host(g[some].double()))
    assert np.all(abs(got - want) <= (2.0**-20 + 2.0**-8) * abs(want) + 2.0**-120)
    del g, y
    T, top, H = 1_000_003, 8, 48
    x = torch.randint(-4, 5, (T, H), device="cuda").half()
    slot = torch.randperm(T * top, device="cuda", dtype=torch.int32)
    rows = torch.zeros(T * top, H, device="cuda", dtype=torch.float16)
    iq4.iq4_moe_dispatch(x, HALF, H, T, H, slot, None, top, T * top, rows, HALF, H)
    assert torch.equal(rows[slot.long()].view(T, top, H), x[:, None].expand(T, top, H))
    out = torch.zeros(T, H, device="cuda")
    iq4.iq4_moe_combine(rows, HALF, H, T * top, slot, None, T, top, H, None, 0, out, iq4.IQ4_F32, H)
    assert torch.equal(out, 8.0 * x.float())
    dw = torch.zeros(T, top, device="cuda")
    iq4.iq4_moe_combine_grad(x, HALF, H, rows, HALF, H, T * top, slot, None, T, top, H, None, 0, dw)
    assert torch.equal(dw, (x.float() ** 2).sum(1, keepdim=True).expand(T, top))


def test_more_rows_than_a_launch_takes():
    """2^24 tokens of 129 pieces of 16 bytes are more than 2^31 lanes: the calls go in parts."""
    note("edges: 2^24 tokens of 1032")
    T, H = 1 << 24, 1032
    value = (torch.arange(T, device="cuda") % 31).half()
    x = torch.empty(T, H, dtype=torch.float16, device="cuda")
    x.copy_(value[:, None].expand(T, H))
    x[-1] = torch.arange(H, device="cuda") % 29
    slot = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    rows = torch.zeros(T, H, dtype=torch.float16, device="cuda")
    iq4.iq4_moe_dispatch(x, HALF, H, T, H, slot, None, 1, T, rows, HALF, H)
    last = x[-1].clone()
    dw = torch.zeros(T, 1, device="cuda")
    iq4.iq4_moe_combine_grad(x, HALF, H, rows, HALF, H, T, slot, None, T, 1, H, None, 0, dw)
    want = H * value.float() ** 2
    want[-1] = (last.float() ** 2).sum()
    assert torch.equal(dw[:, 0], want)
    x.zero_()
    iq4.iq4_moe_combine(rows, HALF, H, T, slot, None, T, 1, H, None, 0, x, HALF, H)
    assert torch.equal(x[-1], last) and torch.equal(rows[0], last)
    for at in (0, 1, H // 2, H - 1):
        assert torch.equal(x[:-1, at], value[:-1]) and torch.equal(rows[1:, at].flip(0), value[:-1])
    rows.zero_()
    iq4.iq4_moe_combine_grad(x, HALF, H, None, HALF, H, T, slot, None, T, 1, H, rows, H, None)
    assert torch.equal(rows[0], last) and torch.equal(rows[1:, H - 1].flip(0), value[:-1])
    del x, rows
    torch.cuda.empty_cache()


def test_the_largest_swiglu():
    """2^34 elements, 2^31 lanes: in two parts, the second of one row."""
    note("edges: SwiGLU of 16384 x 2^20")
    m, k, bf = 1 << 14, 1 << 20, iq4.IQ4_BF16
    row = torch.randn(k, device="cuda").bfloat16()
    g = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    g.copy_(row.expand(m, k))
    g[-1].neg_()
    one = torch.zeros(2, k, dtype=torch.bfloat16, device="cuda")
    two = torch.zeros_like(one)
    y, z = torch.zeros_like(g), torch.zeros_like(g)
    iq4.iq4_swiglu(g, k, g, k, bf, m, k, y, bf, k)
    iq4.iq4_swiglu(g[-2:], k, g[-2:], k, bf, 2, k, one, bf, k)
    assert torch.equal(y[-2:], one) and torch.equal(y[0], one[0]) and torch.equal(y[:, -1], one[0, -1:].expand(m).where(torch.arange(m, device="cuda") < m - 1, one[1, -1]))
    iq4.iq4_swiglu_grad(g, bf, k, g, k, g, k, bf, m, k, y, k, z, k)
    iq4.iq4_swiglu_grad(g[-2:], bf, k, g[-2:], k, g[-2:], k, bf, 2, k, one, k, two, k)
    for big, small in ((y, one), (z, two)):
        assert torch.equal(big[-2:], small) and torch.equal(big[0], small[0]) and torch.equal(big[m // 2], small[0])
    del g, y, z
    torch.cuda.empty_cache()
