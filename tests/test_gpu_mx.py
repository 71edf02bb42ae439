"""Products of microscaled rows on the GPU against the oracle.

Exact cases: with scale bytes 126..128 on both sides and codes whose values are multiples
of 1/2 up to 6 (E2M1) or multiples of 1/8 up to 15 (E4M3 codes 0x38..0x57, both signs),
every product is a multiple of 2^-6 and at most 6 * 15 * 4 = 360 (of 2^-4 and at most
6 * 6 * 4 = 144 for E2M1), so every partial sum of up to 512 of them (1024) is an integer
multiple of 2^-6 (2^-4) below 2^24 of those units: any order of binary32 additions gives the
exact sum, and the result must equal the oracle's, rounded once to the output's type.

Other cases: k products summed in binary32 in some order, each addition rounded to
nearest, are within (k - 1) * 2^-24 * sum |w x| of the exact sum (to first order; the
products themselves are exact), and the rounding to the output's type adds half a step of
the result.
"""
import numpy as np
import pytest
import torch

import dequant_matmul_iq4_amd as iq4
import oracle
from gpu_util import bits_equal, dev, host, note
from rows_util import FMT, HALF_STEP, TYPES, packed, rounder, stored, value

pytestmark = pytest.mark.gpu

E4M3_EXACT = np.array([c | s for c in range(0x38, 0x58) for s in (0, 0x80)], dtype=np.uint8)


def exact_weights(seed, n, k):
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 256, (n, k // 2)).astype(np.uint8), rng.integers(126, 129, (n, k // 32)).astype(np.uint8))


def exact_rows(seed, fmt, m, k):
    rng = np.random.default_rng(seed + 1000)
    s = rng.integers(126, 129, (m, k // 32)).astype(np.uint8)
    if fmt == "mxfp4":
        return rng.integers(0, 256, (m, k // 2)).astype(np.uint8), s
    return rng.choice(E4M3_EXACT, (m, k)), s


def real_weights(seed, n, k):
    return oracle.quantize_rows((np.random.default_rng(seed).standard_normal((n, k)) * 0.02).astype(np.float32), "mxfp4")


def real_rows(seed, fmt, m, k):
    rng = np.random.default_rng(seed + 1000)
    x = rng.standard_normal((m, k)) * np.exp(rng.standard_normal((m, 1)))
    x[:, rng.random(k) < 1 / 32] *= 20
    return oracle.quantize_rows(x.astype(np.float32), fmt)


def product(w, x, fmt, n, k, m, out, ldy=None, ldq=None, lds=None, shift=0, extra=2):
    """iq4_mx_gemm into a buffer with sentinel columns and rows; y as float64."""
    ldy = ldy or n
    q, d, ldq, lds = stored(fmt, *x, k, ldq, lds)
    flat = torch.full(((m + extra) * ldy + shift,), -7.0, dtype=TYPES[out][1], device="cuda")
    y = flat[shift:]
    iq4.iq4_mx_gemm(w, n, k, FMT[fmt], q, ldq, d, lds, m, y, TYPES[out][0], ldy)
    got = host(y.double()).reshape(m + extra, ldy)
    assert np.all(got[m:] == -7.0) and np.all(got[:m, n:] == -7.0), "wrote outside the result"
    return got[:m, :n]


def bound(w, x, k, out):
    """(exact result, allowed absolute error) of decoded rows."""
    r = oracle.mx_product(w, x)
    return r, (k - 1) * 2.0**-24 * oracle.mx_product(np.abs(w), np.abs(x)) + HALF_STEP[out] * np.abs(r)


SHAPES = [(1, 16, 32), (1, 1, 128), (2, 15, 96), (3, 17, 512), (15, 33, 160), (16, 64, 544), (17, 100, 256), (33, 48, 1024),
          (63, 129, 96), (64, 256, 512), (65, 300, 640), (100, 255, 992), (129, 130, 128), (257, 272, 384), (300, 520, 1024)]


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_exact_sums(fmt, m, n, k):
    note(f"mx gemm exact: {m} x {n} x {k} {fmt}")
    k = min(k, 512) if fmt == "mxfp8" else k
    cw, sw = exact_weights(m + n, n, k)
    x = exact_rows(m + k, fmt, m, k)
    r = oracle.mx_product(value("mxfp4", cw, sw), value(fmt, *x))
    w = packed(cw, sw, n, k)
    for out in TYPES:
        assert np.array_equal(product(w, x, fmt, n, k, m, out), rounder(out)(r)), out


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("k", [32, 160, 416, 512])
@pytest.mark.parametrize("m,n", [(325, 4099), (641, 4100), (1003, 7201), (40, 10300)])
def test_exact_sums_of_larger_tiles(fmt, m, n, k):
    """Sizes that fill the device with 128 x 64, 128 x 128, 256 x 128 and 64 x 64 tiles, one to four
    128-element steps, the last row and column tiles partial."""
    note(f"mx gemm exact, large: {m} x {n} x {k} {fmt}")
    cw, sw = exact_weights(m + n, n, k)
    x = exact_rows(m + k, fmt, m, k)
    r = oracle.mx_product(value("mxfp4", cw, sw), value(fmt, *x))
    w = packed(cw, sw, n, k)
    assert np.array_equal(product(w, x, fmt, n, k, m, "f32"), r)
    assert np.array_equal(product(w, x, fmt, n, k, m, "bf16", ldy=n + 5), rounder("bf16")(r))
    if n % 4 == 0:
        assert np.array_equal(product(w, x, fmt, n, k, m, "f16", ldy=n + 4), rounder("f16")(r))


@pytest.mark.parametrize("m", [1, 20, 70])
def test_very_wide_matrix(m):
    note(f"mx gemm: 200003 weight rows, {m} rows")
    n, k = 200003, 96
    cw, sw = exact_weights(4, n, k)
    x = exact_rows(5, "mxfp4", m, k)
    y = product(packed(cw, sw, n, k), x, "mxfp4", n, k, m, "f32", extra=1)
    assert np.array_equal(y, oracle.mx_product(value("mxfp4", cw, sw), value("mxfp4", *x)))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_large_tiles_over_many_steps(fmt):
    note(f"mx gemm: 900 x 6144 x 2336 {fmt} (19 steps)")
    m, n, k = 900, 6144, 2336
    cw, sw = real_weights(n, n, k)
    x = real_rows(m, fmt, m, k)
    dw, dx = value("mxfp4", cw, sw), value(fmt, *x)
    r, tol = bound(dw, dx, k, "f32")
    y = product(packed(cw, sw, n, k), x, fmt, n, k, m, "f32")
    assert np.all(np.abs(y - r) <= tol), float(np.max(np.abs(y - r) / tol))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_rows_more_than_32_bits_apart(fmt):
    note(f"mx gemm: rows of X some 17 and 67 MB apart, {fmt}")
    n, k = 96, 160
    cw, sw = exact_weights(1, n, k)
    w = packed(cw, sw, n, k)
    for m, ldq in ((40, (1 << 24) + 64), (70, 1 << 26)):
        x = exact_rows(3, fmt, m, k)
        r = oracle.mx_product(value("mxfp4", cw, sw), value(fmt, *x))
        c, s = iq4.iq4_rows_bytes(FMT[fmt], k)
        q = torch.empty(m * ldq, dtype=torch.uint8, device="cuda")
        rows = q.view(m, ldq)
        rows[:, :c] = 0
        rows[:, : x[0].shape[1]] = dev(x[0])
        d = torch.zeros(m, s, dtype=torch.uint8, device="cuda")
        d[:, : k // 32] = dev(x[1])
        y = torch.full((m, n), -7.0, device="cuda")
        iq4.iq4_mx_gemm(w, n, k, FMT[fmt], q, ldq, d, s, m, y, iq4.IQ4_F32, n)
        assert np.array_equal(host(y), r)
        y.fill_(-7.0)
        off = dev(np.array([0, m], np.int32))
        iq4.iq4_mx_grouped_gemm(w, 1, n, k, FMT[fmt], q, ldq, d, s, m, off, None, 0, m, y, iq4.IQ4_F32, n)
        assert np.array_equal(host(y), r)
        del q, rows


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m,n,k", [(1, 4096, 4096), (4, 2560, 6144), (16, 1024, 14336), (20, 1000, 2592), (200, 333, 2048), (700, 1300, 2592)])
def test_real_values(fmt, m, n, k):
    note(f"mx gemm: {m} x {n} x {k} {fmt}")
    cw, sw = real_weights(n, n, k)
    x = real_rows(m, fmt, m, k)
    w = packed(cw, sw, n, k)
    dw, dx = value("mxfp4", cw, sw), value(fmt, *x)
    for out in TYPES:
        r, tol = bound(dw, dx, k, out)
        y = product(w, x, fmt, n, k, m, out)
        assert np.all(np.abs(y - r) <= tol), (out, float(np.max(np.abs(y - r) / tol)))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m", [3, 40, 300])
def test_strides_and_alignment(fmt, m):
    note(f"mx gemm: strides, {m} rows {fmt}")
    n, k = 77, 544
    cw, sw = exact_weights(7, n, k)
    if fmt == "mxfp8":
        sw[:] = 127  # keeps 544 sums of E4M3 products exact
    x = exact_rows(8, fmt, m, k)
    r = oracle.mx_product(value("mxfp4", cw, sw), value(fmt, *x))
    w = packed(cw, sw, n, k)
    c, s = iq4.iq4_rows_bytes(FMT[fmt], k)
    for out in TYPES:
        for ldy, shift in ((77, 0), (80, 0), (80, 1), (83, 3), (96, 4)):
            y = product(w, x, fmt, n, k, m, out, ldy=ldy, ldq=c + 48, lds=s + 16, shift=shift)
            assert np.array_equal(y, rounder(out)(r)), (out, ldy, shift)


def test_weights_packed_from_padded_rows():
    note("mx pack: rows with strides and padding give the same bytes")
    n, k = 37, 544
    cw, sw = real_weights(5, n, k)
    a = packed(cw, sw, n, k)
    q, d, ldq, lds = stored("mxfp4", cw, sw, k, 400, 48)
    b = torch.full_like(a, 0x11)
    iq4.iq4_mx_pack_weights(q, ldq, d, lds, n, k, b)
    assert bits_equal(host(a), host(b))
    # against the layout as it is documented
    kt, kq, rt = 5, 2, 3
    want = np.zeros(rt * kt * 1024 + rt * kq * 256, dtype=np.uint8)
    for row in range(n):
        for blk in range(k // 32):
            t, g = divmod(blk, 4)
            at = ((row // 16) * kt + t) * 1024 + (16 * g + row % 16) * 16
            want[at:at + 16] = cw[row, 16 * blk:16 * blk + 16]
            want[rt * kt * 1024 + ((row // 16) * kq + t // 4) * 256 + (16 * g + row % 16) * 4 + t % 4] = sw[row, blk]
    assert np.array_equal(host(a), want)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m", [5, 130])
def test_nan_scales_and_codes(fmt, m):
    note(f"mx gemm: NaN scales, {m} rows {fmt}")
    n, k = 40, 256
    cw, sw = exact_weights(1, n, k)
    x = exact_rows(2, fmt, m, k)
    sw[7, 3] = 255
    x[1][m - 2, 5] = 255
    if fmt == "mxfp8":
        x[0][1, 100] = 0x7F
    r = oracle.mx_product(value("mxfp4", cw, sw), value(fmt, *x))
    y = product(packed(cw, sw, n, k), x, fmt, n, k, m, "f32")
    assert np.array_equal(y, r, equal_nan=True)
    assert np.isnan(y[:, 7]).all() and np.isnan(y[m - 2]).all() and np.isfinite(y[0, :7]).all()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m", [5, 30, 130])
def test_nan_blocks_as_the_quantiser_makes_them(fmt, m):
    """A block with an infinity or a NaN is held as zero codes with a NaN scale: its row's results are NaN all the
    same, and no other row's are.  Rows, scales and codes of both operands in one buffer, side by side."""
    note(f"mx gemm: rows with infinities and NaN, quantised and multiplied, {m} rows {fmt}")
    n, k = 72, 160
    rng = np.random.default_rng(m)
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[1, 3], x[m - 1, 159], x[2, 64:96] = np.nan, np.inf, 0
    wf = rng.standard_normal((n, k)).astype(np.float32)
    wf[7, 130], wf[70, 0] = -np.inf, np.nan

    def held(v, f):
        c, s = iq4.iq4_rows_bytes(FMT[f], k)
        both = torch.full((len(v), c + s + 16), 0xEE, dtype=torch.uint8, device="cuda")
        iq4.iq4_quantize_rows(dev(v), iq4.IQ4_F32, len(v), k, k, FMT[f], both, c + s + 16, both[:, c:], c + s + 16)
        assert bool((both[:, c + s:] == 0xEE).all())
        return both, c, c + s + 16

    wb, wc, wld = held(wf, "mxfp4")
    xb, xc, xld = held(x, fmt)
    w = torch.empty(iq4.iq4_mx_packed_bytes(n, k), dtype=torch.uint8, device="cuda")
    iq4.iq4_mx_pack_weights(wb, wld, wb[:, wc:], wld, n, k, w)
    dw, dx = value("mxfp4", *oracle.quantize_rows(wf, "mxfp4")), value(fmt, *oracle.quantize_rows(x, fmt))
    r, tol = bound(dw, dx, k, "f32")
    off = dev(np.array([0, m], np.int32))
    for by_expert in (False, True):
        y = torch.full((m, n), -7.0, device="cuda")
        if by_expert:
            iq4.iq4_mx_grouped_gemm(w, 1, n, k, FMT[fmt], xb, xld, xb[:, xc:], xld, m, off, None, 0, m, y, iq4.IQ4_F32, n)
        else:
            iq4.iq4_mx_gemm(w, n, k, FMT[fmt], xb, xld, xb[:, xc:], xld, m, y, iq4.IQ4_F32, n)
        got = host(y).astype(np.float64)
        bad = np.isnan(r)
        assert bad[[1, m - 1]].all() and bad[:, [7, 70]].all() and not bad[[0, 2]][:, :7].any()
        assert np.array_equal(np.isnan(got), bad)
        assert np.all(np.abs(got - r)[~bad] <= tol[~bad])


def test_whole_range_of_8_bit_codes():
    """Every E4M3 code next to the largest ones: the largest product of a row is some 2^21
    times its smallest, and the small ones must not be lost."""
    note("mx gemm: E4M3 codes of all magnitudes")
    n, m, k = 64, 200, 128
    rng = np.random.default_rng(9)
    cw, _ = exact_weights(3, n, k)
    sw, sx = np.full((n, 4), 127, np.uint8), np.full((m, 4), 127, np.uint8)
    c = rng.integers(0, 256, (m, k)).astype(np.uint8)
    c[rng.random((m, k)) < 0.2] = 0x7E
    c[:, 1::8] = rng.integers(1, 0x48, (m, k // 8))
    c[(c & 0x7F) == 0x7F] = 0x80
    w = packed(cw, sw, n, k)
    for rows in (m, 7):
        r, tol = bound(value("mxfp4", cw, sw), value("mxfp8", c[:rows], sx[:rows]), k, "f32")
        y = product(w, (c[:rows], sx[:rows]), "mxfp8", n, k, rows, "f32")
        assert np.all(np.abs(y - r) <= tol), float(np.max(np.abs(y - r) / tol))


def test_far_scales():
    note("mx gemm: scales far apart, results that overflow or vanish")
    n, k, m = 32, 128, 4
    cw, _ = exact_weights(3, n, k)
    x0, _ = exact_rows(4, "mxfp4", m, k)
    for a, b in ((0, 127), (127, 0), (254, 100), (1, 20), (60, 60), (250, 254)):
        sw, sx = np.full((n, 4), a, np.uint8), np.full((m, 4), b, np.uint8)
        r = oracle.mx_product(value("mxfp4", cw, sw), value("mxfp4", x0, sx))
        y = product(packed(cw, sw, n, k), (x0, sx), "mxfp4", n, k, m, "f32")
        with np.errstate(over="ignore"):
            want = r.astype(np.float32).astype(np.float64)
        if a + b < 504:
            # all products share one power of two: the sum is exact, also as a subnormal multiple of 2^-149
            assert np.max(np.abs(y - want)) <= 2.0**-149 * (1 if a + b < 110 else 0), (a, b)
        else:
            assert not np.isfinite(y[np.abs(r) > 3.5e38]).any()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("n,k", [(4096, 4096), (100, 2592), (2560, 14336)])
def test_few_rows_equal_single_rows_bitwise(fmt, n, k):
    note(f"mx gemm: up to 16 rows bitwise the single row's, {n} x {k} {fmt}")
    w = packed(*real_weights(11, n, k), n, k)
    x = real_rows(12, fmt, 16, k)
    ones = [product(w, (x[0][i:i + 1], x[1][i:i + 1]), fmt, n, k, 1, "f32") for i in range(16)]
    for m in (2, 3, 4, 8, 15, 16):
        y = product(w, (x[0][:m], x[1][:m]), fmt, n, k, m, "f32")
        for i in range(m):
            assert bits_equal(y[i:i + 1], ones[i]), (m, i)


@pytest.mark.parametrize("m", [7, 30, 200])
def test_8_bit_sums_of_one_scale_are_exact(m):
    """With one scale for all blocks, sums of 128 products that binary32 can hold are the exact ones: of all
    E4M3 codes of magnitude 2 and above (products with E2M1 are multiples of 2^-3, the sums below
    128 * 448 * 6 < 2^19: 22 bits), of all below 2 (multiples of 2^-10, below 128 * 1.875 * 6 < 2^11: 21
    bits), and of all up to 15 (multiples of 2^-10, below 128 * 15 * 6 < 2^14: 24 bits)."""
    note(f"mx gemm: E4M3 codes with one scale, {m} rows")
    n, k = 96, 128
    rng = np.random.default_rng(m)
    cw = rng.integers(0, 256, (n, k // 2)).astype(np.uint8)
    cw[::3] = rng.choice(np.array([0x77, 0x71, 0x17, 0x9F, 0xF1, 0x79, 0x11], np.uint8), (n // 3, k // 2))  # +-6 and +-1/2
    sw, sx = np.full((n, 4), 127, np.uint8), np.full((m, 4), 127, np.uint8)
    w, dw = packed(cw, sw, n, k), value("mxfp4", cw, sw)
    ends = np.array([0x7E, 0xFE, 0x41, 0xC1, 0x40, 0x43], np.uint8)  # 448, 2.25, 2, 2.75
    for name, mags in {"high": np.arange(0x40, 0x7F), "low": np.arange(0x40), "both": np.arange(0x58)}.items():
        c = (rng.choice(mags, (m, k)) | rng.choice([0, 0x80], (m, k))).astype(np.uint8)
        if name == "high":
            c[::2] = rng.choice(ends, c[::2].shape)
        r = oracle.mx_product(dw, value("mxfp8", c, sx))
        assert np.array_equal(r, r.astype(np.float32))
        y = product(w, (c, sx), "mxfp8", n, k, m, "f32")
        assert np.array_equal(y, r), (name, float(np.max(np.abs(y - r))))


@pytest.mark.parametrize("m", [7, 30, 200])
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_scales_that_differ_inside_a_row(fmt, m):
    """Any order of binary32 additions gives the exact sum here.  First, blocks up to 2^9 (MXFP8 2^6) apart: the
    products are multiples of 2^-2 * 2^-9 (2^-4 * 2^-6), the sums below 128 * 6 * 6 < 2^13 (128 * 15 * 6 <
    2^14), 24 bits.  Then a single product of 1 beside three blocks 2^-20 (2^-18) below it: multiples of
    2^-22, sums below 1 + 96 * 36 * 2^-20 < 2 (1 + 96 * 90 * 2^-18 < 2), 23 bits."""
    note(f"mx gemm: scales that differ inside a row, {m} rows {fmt}")
    n, k = 96, 128
    rng = np.random.default_rng(m)
    low = 5 if fmt == "mxfp4" else 3
    cw, _ = exact_weights(5, n, k)
    c, _ = exact_rows(6, fmt, m, k)
    sw = (127 - rng.integers(0, low + 1, (n, 4))).astype(np.uint8)
    sx = (127 - rng.integers(0, (4 if fmt == "mxfp4" else 3) + 1, (m, 4))).astype(np.uint8)
    r = oracle.mx_product(value("mxfp4", cw, sw), value(fmt, c, sx))
    assert np.array_equal(product(packed(cw, sw, n, k), (c, sx), fmt, n, k, m, "f32"), r)
    for block in range(4):
        bw, bx = cw.copy(), c.copy()
        sw, sx = np.full((n, 4), 117, np.uint8), np.full((m, 4), 117 if fmt == "mxfp4" else 119, np.uint8)
        sw[:, block], sx[:, block] = 127, 127
        bw[:, 16 * block:16 * block + 16] = 0
        bw[:, 16 * block + 3] = 0x02  # 1
        each = 16 if fmt == "mxfp4" else 32
        bx[:, each * block:each * block + each] = 0
        bx[:, each * block + 3 * each // 16] = 0x02 if fmt == "mxfp4" else 0x38
        r = oracle.mx_product(value("mxfp4", bw, sw), value(fmt, bx, sx))
        assert np.all(np.abs(r - 1) < 0.5)
        assert np.array_equal(product(packed(bw, sw, n, k), (bx, sx), fmt, n, k, m, "f32"), r), block


def tiles(n, m, bn, bm):
    return -(-n // bn) * -(-m // bm)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m,n", [(1100, 6392), (900, 6144), (300, 5000), (100, 1000), (20, 1000), (9, 1000)])
def test_exact_sums_over_many_steps(fmt, m, n):
    """19 steps of 128 elements, five quads of scales, results stored 16 bytes at a time: 256 x 128 tiles (from 224 of
    them), 128 x 128 (MXFP4) and 128 x 64 (from 160), 64 x 64, and the kernel for few rows.  All sums are
    exact: E2M1 products are multiples of 2^-4 and at most 144, and 2336 * 144 < 2^24 * 2^-4; E4M3 ones, with
    weight scales 127 and 128 and row scales 126 and 127, multiples of 2^-5 and at most 180, and
    2336 * 180 < 2^24 * 2^-5."""
    note(f"mx gemm exact: {m} x {n} x 2336 {fmt}")
    k = 2336
    assert (tiles(n, m, 256, 128) >= 224) == (m == 1100)
    assert (tiles(n, m, 128, 128) >= 160) == (m >= 900) and (tiles(n, m, 128, 64) >= 160) == (m >= 300)
    cw, sw = exact_weights(m, n, k)
    c, sx = exact_rows(m, fmt, m, k)
    if fmt == "mxfp8":
        sw, sx = np.maximum(sw, 127), np.minimum(sx, 127)
    r = oracle.mx_product(value("mxfp4", cw, sw), value(fmt, c, sx))
    w = packed(cw, sw, n, k)
    for out in TYPES:
        with np.errstate(over="ignore"):
            want = rounder(out)(r)
        assert np.array_equal(product(w, (c, sx), fmt, n, k, m, out), want), out


# ---- by expert ------------------------------------------------------------------------------


def bank(seed, e, n, k):
    ws = [exact_weights(seed + i, n, k) for i in range(e)]
    each = iq4.iq4_mx_packed_bytes(n, k)
    out = torch.empty(e * each, dtype=torch.uint8, device="cuda")
    for i, (c, s) in enumerate(ws):
        iq4.iq4_mx_pack_weights(dev(c), k // 2, dev(s), k // 32, n, k, out[i * each:])
    return out, [value("mxfp4", c, s) for c, s in ws]


def grouped(w, e, n, k, fmt, x, offsets, pairs, top, cap, out="f32", ldy=None, extra=3):
    ldy = ldy or n
    q, d, ldq, lds = stored(fmt, *x, k)
    y = torch.full((cap + extra, ldy), -7.0, dtype=TYPES[out][1], device="cuda")
    iq4.iq4_mx_grouped_gemm(w, e, n, k, FMT[fmt], q, ldq, d, lds, len(x[0]), dev(np.asarray(offsets, np.int32)),
                            None if pairs is None else dev(np.asarray(pairs, np.int32)), top, cap, y, TYPES[out][0], ldy)
    got = host(y.double())
    assert np.all(got[:, n:] == -7.0) and np.all(got[cap:] == -7.0)
    return got[:cap, :n]


COUNTS = {
    "even": [5] * 7,
    "empty": [0, 0, 3, 0, 1, 0, 0],
    "one": [0, 0, 0, 70],
    "first": [300, 1, 0],
    "ragged": [1, 16, 17, 0, 63, 64, 65, 128, 129, 2, 33],
    "single": [41],
    "many": [i % 3 for i in range(150)],
    "long": [260, 0, 515, 31],
    "crowd": [i % 5 for i in range(300)],
    "crowded": [i % 8 for i in range(301)],
    "most": [(i * 7) % 4 for i in range(1024)],
}


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("n,k", [(40, 160), (272, 512)])
def test_grouped(fmt, name, n, k):
    note(f"mx grouped: {name} {n} x {k} {fmt}")
    counts = COUNTS[name]
    e, total = len(counts), sum(counts)
    w, dense = bank(100, e, n, k)
    off = np.concatenate([[0], np.cumsum(counts)])
    expert = np.repeat(np.arange(e), counts)
    # rows in the experts' order; two rows of the buffer unused at its end
    x = exact_rows(5, fmt, total + 2, k)
    dx = value(fmt, *x)
    r = np.stack([dense[expert[i]] @ dx[i] for i in range(total)])
    for out in TYPES:
        y = grouped(w, e, n, k, fmt, x, off, None, 0, total, out)
        assert np.array_equal(y, rounder(out)(r)), out
    # rows behind the last expert's stay as they were
    y = grouped(w, e, n, k, fmt, x, off, None, 0, total + 2)
    assert np.array_equal(y[:total], r) and np.all(y[total:] == -7.0)
    # rows gathered: pair p of token p // top
    top = 3
    tokens = (total + top - 1) // top
    pairs = np.random.default_rng(6).permutation(total)
    x = exact_rows(7, fmt, tokens, k)
    dx = value(fmt, *x)
    r = np.stack([dense[expert[i]] @ dx[pairs[i] // top] for i in range(total)])
    y = grouped(w, e, n, k, fmt, x, off, pairs, top, total, ldy=n + 3)
    assert np.array_equal(y, r)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("k", [160, 512])
def test_grouped_large_tiles(fmt, k):
    note(f"mx grouped: 256 x 128 tiles, k = {k} {fmt}")
    counts, n = [130, 0, 1, 300, 64, 65, 128, 33], 7201
    e, total = len(counts), sum(counts)
    w, dense = bank(300, e, n, k)
    off = np.concatenate([[0], np.cumsum(counts)])
    expert = np.repeat(np.arange(e), counts)
    top = 2
    tokens = (total + 1) // 2 + 2
    pairs = np.concatenate([np.random.default_rng(8).permutation(total), [0, 0, 0]])  # three pairs more than rows
    x = exact_rows(9, fmt, tokens, k)
    dx = value(fmt, *x)
    r = np.concatenate([dx[pairs[off[i]:off[i + 1]] // top] @ dense[i].T for i in range(e)])
    assert np.array_equal(expert, np.sort(expert)) and r.shape == (total, n)
    for out, ldy in (("f32", n), ("f16", n + 7)):
        y = grouped(w, e, n, k, fmt, x, off, pairs, top, total + 3, out, ldy)
        assert np.array_equal(y[:total], rounder(out)(r)) and np.all(y[total:] == -7.0)


def test_grouped_offsets_and_pairs_out_of_range():
    """Device values that break the rules are clamped: the result means nothing, and no byte
    outside it is written."""
    note("mx grouped: offsets and pairs out of range")
    e, n, k, cap = 5, 40, 160, 60
    w, _ = bank(100, e, n, k)
    x = exact_rows(5, "mxfp4", 30, k)
    for off in ([-5, 10, 7, 90, 20, 1 << 30], [0, 60, 60, 60, 60, 60], [1 << 30] * 6, [60, 50, 40, 30, 20, 10]):
        for pairs in (None, [-(1 << 31), (1 << 31) - 1, 59, -1] * 15):
            rows = exact_rows(5, "mxfp4", 60, k) if pairs is None else x
            grouped(w, e, n, k, "mxfp4", rows, off, pairs, 2, cap)  # checks the sentinels around y


def test_grouped_no_rows_at_all():
    note("mx grouped: every expert empty")
    w, _ = bank(100, 3, 40, 160)
    y = grouped(w, 3, 40, 160, "mxfp4", exact_rows(5, "mxfp4", 9, 160), [0, 0, 0, 0], None, 0, 9)
    assert np.all(y == -7.0)


def spread_rows(x, k, fmt, ldq):
    """Compact rows of X on the device (codes, scales) with `ldq` bytes between the codes' rows."""
    c, s = iq4.iq4_rows_bytes(FMT[fmt], k)
    q = torch.empty(len(x[0]) * ldq, dtype=torch.uint8, device="cuda")
    rows = q.view(len(x[0]), ldq)
    rows[:, :c] = 0
    rows[:, : x[0].shape[1]] = dev(x[0])
    d = torch.zeros(len(x[1]), s, dtype=torch.uint8, device="cuda")
    d[:, : k // 32] = dev(x[1])
    return q, d, ldq, s


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_many_rows_past_4_gib(fmt, gather):
    """X of 4.6 GB and some 70,000 rows: such a call is an ordinary one of the documented sizes.
    The rows are 64 KB apart; the same rows side by side must give the same bits (all sums are exact)."""
    note(f"mx grouped: 70001 rows of X in 4.6 GB, pairs {gather}, {fmt}")
    counts, n, k, top = [40000, 1, 0, 30000], 16384, 160, 2
    e, m = len(counts), sum(counts)
    w, dense = bank(400, e, n, k)
    off = np.concatenate([[0], np.cumsum(counts)])
    x = exact_rows(11, fmt, m, k)
    q, d, ldq, lds = spread_rows(x, k, fmt, 1 << 16)
    pairs = np.random.default_rng(12).permutation(m * top)[:m] if gather else None
    row = pairs // top if gather else np.arange(m)
    assert q.numel() >= 1 << 32 and row.max() > m - 10
    doff = dev(off.astype(np.int32))
    y = torch.full((m + 1, n), -7.0, dtype=torch.float16, device="cuda")
    iq4.iq4_mx_grouped_gemm(w, e, n, k, FMT[fmt], q, ldq, d, lds, m, doff, dev(pairs.astype(np.int32)) if gather else None,
                            top, m, y, iq4.IQ4_F16, n)
    assert bool((y[m] == -7.0).all())
    del q
    near, dn, ldn, lsn = stored(fmt, x[0][row], x[1][row], k)
    z = torch.full((m, n), -7.0, dtype=torch.float16, device="cuda")
    iq4.iq4_mx_grouped_gemm(w, e, n, k, FMT[fmt], near, ldn, dn, lsn, m, doff, None, 0, m, z, iq4.IQ4_F16, n)
    assert torch.equal(y[:m].view(torch.int16), z.view(torch.int16))
    for i in (0, 1, 63, 64, 39999, 40000, 40001, 40002, m - 65, m - 1):
        r = dense[int(np.searchsorted(off, i, side="right")) - 1] @ value(fmt, x[0][row[i]][None], x[1][row[i]][None])[0]
        assert np.array_equal(host(y[i].double()), rounder("f16")(r)), i


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("ldq", [(1 << 25) - 64, 1 << 25])
def test_grouped_rows_of_a_tile_2_to_4_gib_apart(fmt, ldq):
    """The last rows of a tile begin past 2^31 bytes from its first one (and, of X, short of 2^32 and past it)."""
    note(f"mx grouped: 127 rows {ldq} bytes apart {fmt}")
    counts, n, k = [3, 121, 0, 3], 200, 160
    e, m = len(counts), sum(counts)
    w, dense = bank(500, e, n, k)
    off = np.concatenate([[0], np.cumsum(counts)])
    expert = np.repeat(np.arange(e), counts)
    x = exact_rows(13, fmt, m, k)
    dx = value(fmt, *x)
    q, d, ldq, lds = spread_rows(x, k, fmt, ldq)
    assert (m - 1) * ldq > 1 << 31
    pairs = np.random.default_rng(14).permutation(m)
    for p in (None, pairs):
        row = np.arange(m) if p is None else p
        r = np.stack([dense[expert[i]] @ dx[row[i]] for i in range(m)])
        y = torch.full((m, n), -7.0, device="cuda")
        iq4.iq4_mx_grouped_gemm(w, e, n, k, FMT[fmt], q, ldq, d, lds, m, dev(off.astype(np.int32)),
                                None if p is None else dev(p.astype(np.int32)), 1, m, y, iq4.IQ4_F32, n)
        assert np.array_equal(host(y), r)


def test_grouped_garbage_offsets_and_pairs_with_rows_far_apart():
    """As test_grouped_offsets_and_pairs_out_of_range, rows of X so far apart that lanes hold addresses."""
    note("mx grouped: offsets and pairs out of range, rows 64 MB apart")
    e, n, k, cap, fmt = 5, 40, 160, 66, "mxfp4"
    w, _ = bank(100, e, n, k)
    q, d, ldq, lds = spread_rows(exact_rows(5, fmt, cap, k), k, fmt, 1 << 26)
    for off in ([-5, 10, 7, 90, 20, 1 << 30], [0, 60, 60, 60, 60, 60], [1 << 30] * 6, [60, 50, 40, 30, 20, 10]):
        for pairs in (None, [-(1 << 31), (1 << 31) - 1, 59, -1, 0, 65] * 11):
            y = torch.full((cap + 3, n + 1), -7.0, device="cuda")
            iq4.iq4_mx_grouped_gemm(w, e, n, k, FMT[fmt], q, ldq, d, lds, cap, dev(np.asarray(off, np.int32)),
                                    None if pairs is None else dev(np.asarray(pairs, np.int32)), 2, cap, y, iq4.IQ4_F32, n + 1)
            got = host(y)
            assert np.all(got[cap:] == -7.0) and np.all(got[:, n:] == -7.0)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("counts,n", [([300, 0, 129, 340], 7168), ([30, 0, 129, 2, 65], 200), ([1, 0, 2, 1, 3], 1000)])
def test_grouped_over_many_steps(fmt, counts, n):
    """10 steps, three quads of scales: 256 x 128 tiles (28 of them side by side, some 6 + 4 / 2 high: at least
    192, and 64 rows an expert), 128 x 64, and few rows; in each, rows of X side by side, gathered, and gathered from 4 GiB
    and more.  E2M1 products are multiples of 2^-4, at most 144: 1184 * 144 < 2^20.  E4M3 ones, with row
    scales 126 and 127, multiples of 2^-6, at most 180: 1184 * 180 < 2^18."""
    note(f"mx grouped: {counts} {n} x 1184 {fmt}")
    e, total, k, top = len(counts), sum(counts), 1184, 2
    assert (-(-n // 256) * (total // 128 + e // 2) >= 192) == (n == 7168) and (total <= 2 * e) == (n == 1000)
    w, dense = bank(600, e, n, k)
    off = np.concatenate([[0], np.cumsum(counts)])
    rows = {"side by side": (total, None), "gathered": ((total + 1) // 2, np.random.default_rng(15).permutation(total))}
    for name, (count, pairs) in rows.items():
        c, sx = exact_rows(16, fmt, count, k)
        if fmt == "mxfp8":
            sx = np.minimum(sx, 127)
        dx = value(fmt, c, sx)
        dx = dx if pairs is None else dx[pairs // top]
        r = np.concatenate([dx[off[i]:off[i + 1]] @ dense[i].T for i in range(e)])
        for out in TYPES:
            y = grouped(w, e, n, k, fmt, (c, sx), off, pairs, top, total, out)
            assert np.array_equal(y, rounder(out)(r)), (name, out)
        if pairs is None:
            continue
        q, d, ldq, lds = spread_rows((c, sx), k, fmt, ((1 << 32) // count + 64) // 64 * 64)
        assert count * ldq >= 1 << 32
        y = torch.full((total, n), -7.0, device="cuda")
        iq4.iq4_mx_grouped_gemm(w, e, n, k, FMT[fmt], q, ldq, d, lds, count, dev(off.astype(np.int32)),
                                dev(pairs.astype(np.int32)), top, total, y, iq4.IQ4_F32, n)
        assert np.array_equal(host(y), r), "far apart"


@pytest.mark.parametrize("tokens,hidden,inter,experts,top", [(4, 512, 256, 16, 4), (90, 512, 384, 12, 3)])
def test_layer(tokens, hidden, inter, experts, top):
    """A run of the calls as a layer makes them: norm (residual added) to rows, routing,
    gather, gate and up products by expert, SwiGLU, rows again, down products, weighted
    sum -- each step against the oracle on the step's own inputs."""
    note(f"mx layer: {tokens} tokens, {experts} experts")
    rng = np.random.default_rng(77)
    x, res = (rng.standard_normal((tokens, hidden)).astype(np.float32) for _ in range(2))
    gain = (1 + 0.1 * rng.standard_normal(hidden)).astype(np.float32)
    logits = rng.standard_normal((tokens, experts)).astype(np.float32)
    up = [real_weights(500 + i, 2 * inter, hidden) for i in range(experts)]
    down = [real_weights(900 + i, hidden, inter) for i in range(experts)]
    eu, ed = iq4.iq4_mx_packed_bytes(2 * inter, hidden), iq4.iq4_mx_packed_bytes(hidden, inter)
    wu = torch.empty(experts * eu, dtype=torch.uint8, device="cuda")
    wd = torch.empty(experts * ed, dtype=torch.uint8, device="cuda")
    for i in range(experts):
        iq4.iq4_mx_pack_weights(dev(up[i][0]), hidden // 2, dev(up[i][1]), hidden // 32, 2 * inter, hidden, wu[i * eu:])
        iq4.iq4_mx_pack_weights(dev(down[i][0]), inter // 2, dev(down[i][1]), inter // 32, hidden, inter, wd[i * ed:])

    f8, P = FMT["mxfp8"], tokens * top
    cq, cs = iq4.iq4_rows_bytes(f8, hidden)
    hq, hs = iq4.iq4_rows_bytes(f8, inter)
    t = lambda *shape, dt=torch.float32: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
    xd, rd, gd, ld = dev(x), dev(res), dev(gain), dev(logits)
    h, q, d = t(tokens, hidden), t(tokens, cq, dt=torch.uint8), t(tokens, cs, dt=torch.uint8)
    ids, wt = t(tokens, top, dt=torch.int32), t(tokens, top)
    cnt, off = t(experts, dt=torch.int32), t(experts + 1, dt=torch.int32)
    pairs, slot = t(P, dt=torch.int32), t(P, dt=torch.int32)
    gu, a = t(P, 2 * inter), t(P, inter)
    q2, d2, y = t(P, hq, dt=torch.uint8), t(P, hs, dt=torch.uint8), t(P, hidden)

    def layer():
        iq4.iq4_rmsnorm(xd, hidden, rd, hidden, iq4.IQ4_F32, tokens, hidden, gd, 1e-6, h, hidden, None, 0, 0, f8, q, cq, d, cs)
        iq4.iq4_route_topk(ld, tokens, experts, top, ids, wt)
        iq4.iq4_moe_gather(ids, P, experts, cnt, off, pairs, slot)
        iq4.iq4_mx_grouped_gemm(wu, experts, 2 * inter, hidden, f8, q, cq, d, cs, tokens, off, pairs, top, P, gu, iq4.IQ4_F32, 2 * inter)
        torch.mul(torch.nn.functional.silu(gu[:, :inter]), gu[:, inter:], out=a)
        iq4.iq4_quantize_rows(a, iq4.IQ4_F32, P, inter, inter, f8, q2, hq, d2, hs)
        iq4.iq4_mx_grouped_gemm(wd, experts, hidden, inter, f8, q2, hq, d2, hs, P, off, None, 0, P, y, iq4.IQ4_F32, hidden)
        return (y[slot.long()].view(tokens, top, hidden) * wt.unsqueeze(-1)).sum(1)

    out = host(layer())
    # the oracle, step by step on what the step was given
    hr, yr = oracle.rmsnorm(x, res, gain, 1e-6, rounder("f32"))
    assert np.array_equal(host(h), hr.astype(np.float32))
    cx, sx = oracle.quantize_rows(yr, "mxfp8")
    assert np.array_equal(host(q)[:, :hidden], cx) and np.array_equal(host(d)[:, : hidden // 32], sx)
    dx = value("mxfp8", cx, sx)
    rid, rw = oracle.route_topk(logits, top)
    assert np.array_equal(host(ids), rid)
    pr, of = host(pairs), host(off)
    expert = np.searchsorted(of, np.arange(P), side="right") - 1
    gur = host(gu).astype(np.float64)
    for i in range(P):
        r, tol = bound(value("mxfp4", *up[expert[i]]), dx[pr[i] // top][None], hidden, "f32")
        assert np.all(np.abs(gur[i] - r[0]) <= tol[0]), i
    ca, sa = oracle.quantize_rows(host(a), "mxfp8")
    assert np.array_equal(host(q2)[:, :inter], ca) and np.array_equal(host(d2)[:, : inter // 32], sa)
    da = value("mxfp8", ca, sa)
    yh = host(y).astype(np.float64)
    for i in range(P):
        r, tol = bound(value("mxfp4", *down[expert[i]]), da[i][None], inter, "f32")
        assert np.all(np.abs(yh[i] - r[0]) <= tol[0]), i
    want = (yh[host(slot)].reshape(tokens, top, hidden) * host(wt).astype(np.float64)[:, :, None]).sum(1)
    # top products and top - 1 sums in binary32
    slack = 2 * top * 2.0**-24 * (np.abs(yh[host(slot)]).reshape(tokens, top, hidden) * host(wt)[:, :, None]).sum(1)
    assert np.all(np.abs(out - want) <= slack)

    # the library's calls captured into a graph and replayed, eager work in between
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = layer()
    s.synchronize()
    assert bits_equal(host(first), out)
    keep = [host(v).copy() for v in (h, gu, y)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for turn in range(3):
        for v in (h, q, d, gu, a, q2, d2, y):
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for v, want in zip((h, gu, y), keep):
            assert bits_equal(host(v), want), turn
        assert bits_equal(host(layer()), out)


def test_calls_on_two_streams_at_once():
    note("mx: the same calls on two streams at once")
    n, k, m = 520, 1024, 70
    cw, sw = exact_weights(1, n, k)
    w = packed(cw, sw, n, k)
    xs = [exact_rows(i, "mxfp4", m, k) for i in (10, 20)]
    bufs = [stored("mxfp4", *x, k) for x in xs]
    want = [oracle.mx_product(value("mxfp4", cw, sw), value("mxfp4", *x)) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    ys = [torch.zeros(m, n, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for (q, d, ldq, lds), y, s in zip(bufs, ys, streams):
            iq4.iq4_mx_gemm(w, n, k, FMT["mxfp4"], q, ldq, d, lds, m, y, iq4.IQ4_F32, n, stream=s)
    torch.cuda.synchronize()
    for y, r in zip(ys, want):
        assert np.array_equal(host(y), r)
