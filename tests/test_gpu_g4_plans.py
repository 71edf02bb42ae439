"""The group-scaled products in every shape of a launch: one operand of rows of X and two, each number of code tiles a wave
(1, 2, 3, 4, 6), k in slices, sums joined once and several times; dense and by expert, all groups and types.

Whole numbers and powers of two make every product, and every partial sum in any order, a binary32 number: the result has to be
the exact one.  Each row of X, and each stretch of it that a wave may take, has its own power of two, so that what belongs to one
row, operand, wave or slice (the power that binary32's values are held with, bfloat16's group sums) shows if it goes to another.
"""
import numpy as np
import pytest
import torch

import dequant_matmul_iq4_amd as iq4
import oracle
from gpu_util import note
from rows_util import TYPES, floats, rounder
from test_gpu_g4 import grouped, pack, product, weights

pytestmark = pytest.mark.gpu


def _codes(seed, n, k, group, zeros):
    """Weights of whole numbers: scales of one, of either sign."""
    codes, s, z = weights(seed, n, k, group, zeros, "f16", True)
    return codes, np.sign(s), z


def _rows(seed, m, k):
    """|x| <= 2 in each stretch's power (1/2, 1 or 2) by its row's: |sum| <= 2 * 2 * 15 k below 2^20 for k <= 9696, in
    steps of 1/2 of the row's power: 21 bits of a binary32 number."""
    rng = np.random.default_rng(seed)
    stretch = 128 if k <= 1024 else 512 if k <= 4096 else 768
    parts = 2.0 ** rng.integers(-1, 2, (m, -(-k // stretch)))
    return rng.integers(-2, 3, (m, k)) * np.repeat(parts, stretch, 1)[:, :k] * 2.0 ** rng.integers(-8, 9, (m, 1))


# n, k, rows
DENSE = [(17, 32, 5), (130, 1184, 1), (100, 2912, 3), (33, 4256, 3), (2100, 2976, 12), (4096, 4096, 1), (4100, 1600, 16), (40, 8768, 5), (3850, 7424, 40),
         (9000, 224, 100), (1500, 800, 300), (157, 992, 6390), (157, 992, 3190), (163, 1120, 760), (2100, 4000, 300), (1200, 2016, 700),
         (100, 2112, 1500), (3850, 5984, 300), (3850, 6400, 300), (500, 9696, 1400)]


@pytest.mark.parametrize("n,k,m", DENSE)
def test_dense(n, k, m):
    for i, t in enumerate(TYPES):
        group = (32, 64, 128)[(i + n) % 3]
        note(f"g4 plans: {m} x {n} x {k} by {group}, {t}")
        codes, s, z = _codes(n + k, n, k, group, i != 1)
        p, w = pack(codes, s, z, group, "f16"), oracle.g4_weights(codes, s, z, group)
        x = _rows(m, m, k)
        got = product(p, n, k, group, z, "f16", x, t, "f32", ldx=k + i, ldy=n + 1)
        assert np.array_equal(got, oracle.g4_product(w, x))


# n, k, pairs, experts
GROUPED = [(40, 2976, 4, 1), (40, 4384, 3, 2), (24, 9312, 8, 3), (512, 768, 488, 128), (1528, 2016, 32, 40), (512, 736, 2400, 64), (200, 160, 700, 100),
           (700, 480, 700, 100), (40, 992, 3000, 64), (2500, 32, 1500, 42), (5000, 32, 2044, 83), (3464, 160, 2040, 39), (8131, 160, 585, 33),
           (2041, 992, 520, 8), (333, 4096, 70, 5), (500, 4064, 300, 9), (1100, 2592, 300, 5), (1200, 3968, 300, 4), (1300, 2336, 2400, 3),
           (300, 5984, 300, 30), (545, 4864, 507, 2), (700, 6368, 40, 4), (633, 6560, 2000, 1), (900, 8768, 2000, 1)]


@pytest.mark.parametrize("n,k,m,e", GROUPED)
def test_by_expert(n, k, m, e):
    """Counts from a few loads that differ, a tenth of the experts without rows; the rows gathered by pairs, or in their order."""
    top = 3
    for i, t in enumerate(TYPES):
        group, zeros, gather = (32, 64, 128)[(i + e) % 3], i != 2, i != 1
        note(f"g4 plans: {m} pairs of {e} experts, {n} x {k} by {group}, {t}")
        rng = np.random.default_rng(n + i)
        each = iq4.iq4_g4_packed_bytes(n, k, group, zeros)
        p = torch.full((e * each,), 0xEE, dtype=torch.uint8, device="cuda")
        some = [_codes(n + j, n, k, group, zeros) for j in range(min(e, 5))]  # (matrices repeat from the sixth on)
        ws = [oracle.g4_weights(*v, group) for v in some]
        for j in range(e):
            pack(*some[j % 5], group, "f16", p[j * each:(j + 1) * each])
        load = rng.exponential(1, e) * (rng.random(e) > 0.1) + 1e-9
        counts = rng.multinomial(m, load / load.sum())
        at = np.concatenate([[0], np.cumsum(counts)])
        rows = -(-m // top) if gather else m
        x = _rows(m, rows, k)
        pairs = rng.permutation(rows * top)[:m] if gather else None
        got = grouped(p, e, n, k, group, zeros, "f16", x, t, "f32", at, pairs, top, m, ldx=k + i, ldy=n + 1)
        src = x[pairs // top] if gather else x
        for j in range(e):
            assert np.array_equal(got[at[j]: at[j + 1]], oracle.g4_product(ws[j % 5], src[at[j]: at[j + 1]])), j


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n,k,group,m", [(2100, 4000, 64, 40), (600, 8768, 32, 17), (500, 6528, 128, 300), (1200, 2016, 32, 700)])
def test_real_inputs(n, k, group, m, t):
    """Sums of k products and of the groups' scalings, each off by at most a step of the magnitudes' sum (of |s| (16 + q) and
    |s| (16 + z) for bfloat16); a binary32 value by 2^-23 of itself or 2^-50 of its slice's largest."""
    note(f"g4 plans: real {m} x {n} x {k} by {group}, {t}")
    codes, s, z = weights(k, n, k, group, True, "bf16", False)
    rng = np.random.default_rng(m)
    x = rounder(t)(rng.standard_normal((m, k)) * np.exp(rng.standard_normal((m, 1)) + 0.5 * rng.standard_normal((m, k))))
    w = oracle.g4_weights(codes, s, z, group)
    want, mags = oracle.g4_product(w, x), oracle.g4_product(abs(w), abs(x))
    got = product(pack(codes, s, z, group, "bf16"), n, k, group, z, "bf16", x, t, "f32")
    own = 2.0**-23 * mags + 2.0**-50 * abs(x).max(1, keepdims=True) * abs(w).sum(1) if t == "f32" else 0
    if t == "bf16":
        q = np.stack((codes & 15, codes >> 4), 2).reshape(n, k)
        wide = lambda v: np.repeat(v, group, axis=1)[:, :k]  # noqa: E731
        mags = oracle.g4_product(abs(wide(s)) * (32 + q + wide(z)), abs(x))
    assert np.all(abs(got - want) <= (1.001 * (k + 2 * k / 32) + 64) * 2.0**-23 * mags + own)
    assert np.linalg.norm(got - want) <= 2e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("t", list(TYPES))
def test_infinities_and_nan_by_expert(t):
    note(f"g4 plans: infinities and NaN by expert, {t}")
    n, k, group, m, e, top = 700, 2016, 64, 130, 6, 2
    rng = np.random.default_rng(3)
    each = iq4.iq4_g4_packed_bytes(n, k, group, True)
    p = torch.empty(e * each, dtype=torch.uint8, device="cuda")
    ws = []
    for j in range(e):
        codes, s, z = _codes(j, n, k, group, True)
        pack(codes, s, z, group, "f16", p[j * each:(j + 1) * each])
        ws.append(oracle.g4_weights(codes, s, z, group))
    x = _rows(4, m // top, k)
    odd = {5: (40, np.inf), 17: (k - 1, -np.inf), 30: (1000, np.nan), 64: (0, np.inf)}
    for r, (at, v) in odd.items():
        x[r, at] = v
    at = np.concatenate([[0], np.cumsum(rng.multinomial(m, np.ones(e) / e))])
    pairs = rng.permutation(m)
    got = grouped(p, e, n, k, group, True, "f16", x, t, "f32", at, pairs, top, m)
    for j in range(e):
        for i in range(at[j], at[j + 1]):
            r = pairs[i] // top
            if r in odd:
                with np.errstate(invalid="ignore"):
                    want = ws[j][:, odd[r][0]] * odd[r][1]
            else:
                want = oracle.g4_product(ws[j], x[r][None])[0]
            assert np.array_equal(got[i], want, equal_nan=True), (j, i)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n,k,group", [(40, 96, 32), (520, 1024, 64), (70000, 512, 128), (4096, 4096, 128), (100, 5024, 64), (300, 7200, 32), (2560, 6144, 32)])
def test_a_row_alone_is_the_row_among_few(n, k, group, t):
    """Up to eight rows of binary32, or 16 of 16 bits, against one matrix: bit for bit what each is by itself."""
    note(f"g4 plans: rows alone and together, {n} x {k} by {group}, {t}")
    most = 8 if t == "f32" else 16
    codes, s, z = weights(n, n, k, group, True, "f16", False)
    p = pack(codes, s, z, group, "f16")
    x = rounder(t)(np.random.default_rng(k).standard_normal((most, k)))
    together = [product(p, n, k, group, z, "f16", x[:m], t, "f32") for m in (2, 4, 7, most)]
    for r in range(0, most, 3 if n > 9999 else 1):
        alone = product(p, n, k, group, z, "f16", x[r:r + 1], t, "f32")[0]
        assert all(np.array_equal(y[r], alone) for y in together if r < len(y)), r


@pytest.mark.parametrize("n,fewer,k,m", [(14336, 13978, 6144, 47), (9566, 9216, 6144, 66)])
def test_no_second_round_of_workgroups(n, fewer, k, m):
    """Sizes whose workgroups just fit the device take little longer than a few row tiles less (1.7 times as long, were some
    XCDs given more of them than they hold)."""
    note(f"g4 plans: time of {m} x {n} x {k}")
    group = 64
    codes, s, z = weights(1, n, k, group, True, "f16", True)
    x = floats(np.ones((m, k)), "bf16")
    y = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    p = [(r, pack(codes[:r], s[:r], z[:r], group, "f16")) for r in (n, fewer)]
    times = [[], []]
    for _ in range(7):
        for (rows, w), out in zip(p, times):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(10):
                iq4.iq4_g4_qmv(w, rows, k, group, iq4.IQ4_F16, 1, x, iq4.IQ4_BF16, k, m, y, iq4.IQ4_BF16, rows)
            b.record()
            torch.cuda.synchronize()
            out.append(a.elapsed_time(b) * 100)
    note("  {:.1f} us, {:.1f} with fewer row tiles".format(*map(min, times)))
    assert min(times[0]) <= 1.35 * min(times[1])
