"""Rows in 8 or 4 bits and the RMS norm on the GPU against the oracle.

Everything here is a function of the inputs bit for bit: the codes and scales are decided
in exact arithmetic from the row's float32 values, the norm's mean is held in 64 bits and
its other steps are single binary32 roundings that the definition names.  So codes, scales
and all float outputs must equal the oracle's exactly; no tolerance is used.
"""
import numpy as np
import pytest
import torch

import dequant_matmul_iq4_amd as iq4
import oracle
from gpu_util import bits_equal, host, note
from rows_util import FMT, TYPES, floats, rounder, row_buffers, split_rows, stored, value

pytestmark = pytest.mark.gpu


def acts(seed, m, k):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)) * np.exp(rng.standard_normal((m, 1)))
    x[:, rng.random(k) < 1 / 32] *= 20
    return x.astype(np.float32)


def special_rows():
    """Blocks where a rounding or a scale can go wrong, as rows of 12 x 32."""
    rng = np.random.default_rng(3)
    b = [rng.standard_normal(32) * s for s in (1e-30, 1e-5, 1.0, 3e4)]
    b.append(np.arange(-16, 16) / 4.0)
    b.append(np.concatenate([[7.9, -7.9, 6.0, 5.0, 4.99, -2.5, 0.25, 0.75], np.zeros(24)]))
    b.append(np.zeros(32))
    b.append(np.full(32, -0.0))
    b.append(np.concatenate([[480.0, 449.0, -464.0, 465.0, 2.0**-10, 1.5 * 2.0**-10, 2.0**-9], np.full(25, 3 * 2.0**-10)]))
    b.append(np.concatenate([[1.0], np.full(31, np.nextafter(np.float32(0.25), np.float32(1)))]))
    b.append(np.full(32, 2.0**-14))
    b.append(np.concatenate([[254.0, -127.0], 0.5 + np.arange(30)]))
    x = np.stack(b).reshape(1, -1)
    return np.concatenate([x, x * 2.0**7, -x]).astype(np.float32)


def quantise(x, t, fmt, ldx=None, ldq=None, lds=None):
    m, k = x.shape
    q, d, ldq, lds = row_buffers(fmt, m, k, ldq, lds)
    xd = floats(x, t, ldx)
    iq4.iq4_quantize_rows(xd, TYPES[t][0], m, k, xd.shape[1], FMT[fmt], q, ldq, d, lds)
    return q, d


def same_rows(fmt, k, q, d, want):
    codes, scales = split_rows(fmt, k, q, d)
    assert np.array_equal(codes, want[0])
    if fmt == "q8_1":
        a, b = scales, want[1]
        assert np.array_equal(np.isnan(a), np.isnan(b)) and bits_equal(np.nan_to_num(a, nan=0), np.nan_to_num(b, nan=0))
    else:
        assert np.array_equal(scales, want[1])


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("m,k", [(1, 32), (3, 64), (5, 96), (2, 128), (4, 160), (1, 512), (7, 544), (3, 2592), (33, 4096)])
def test_quantise_and_back(fmt, t, m, k):
    note(f"rows: quantise {m} x {k} {t} -> {fmt} and back")
    x = rounder(t)(acts(m * k, m, k).astype(np.float64)).astype(np.float32)
    q, d = quantise(x, t, fmt)
    want = oracle.quantize_rows(x, fmt)
    same_rows(fmt, k, q, d, want)
    v = value(fmt, *want)
    for out in TYPES:
        o = floats(np.zeros((m, k)), out, k + 8)
        o[:] = -7.0
        iq4.iq4_dequant_rows(q, q.shape[1], d, d.shape[1], FMT[fmt], m, k, TYPES[out][0], o, k + 8)
        got = host(o.double())
        assert np.array_equal(got[:, :k], rounder(out)(v)) and np.all(got[:, k:] == -7.0)


@pytest.mark.parametrize("fmt", list(FMT))
def test_special_blocks_strides_and_gaps(fmt):
    note(f"rows: special blocks, strides, {fmt}")
    x = special_rows()
    m, k = x.shape
    c, s = iq4.iq4_rows_bytes(FMT[fmt], k)
    q, d = quantise(x, "f32", fmt, ldx=k + 12, ldq=c + 16, lds=s + 32)
    same_rows(fmt, k, q, d, oracle.quantize_rows(x, fmt))
    assert np.all(host(q)[:, c:] == 0xEE) and np.all(host(d)[:, s:] == 0xEE)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("t", list(TYPES))
def test_infinities_and_nans(fmt, t):
    note(f"rows: infinities and NaN, {fmt} {t}")
    x = acts(4, 4, 128)
    x[0, 5], x[1, 40], x[2, 127], x[2, 64] = np.inf, np.nan, -np.inf, np.nan
    x = rounder(t)(x.astype(np.float64)).astype(np.float32)
    q, d = quantise(x, t, fmt)
    want = oracle.quantize_rows(x, fmt)
    same_rows(fmt, 128, q, d, want)
    o = torch.zeros(4, 128, device="cuda")
    iq4.iq4_dequant_rows(q, q.shape[1], d, d.shape[1], FMT[fmt], 4, 128, iq4.IQ4_F32, o, 128)
    assert np.array_equal(host(o).astype(np.float64), value(fmt, *want), equal_nan=True)


def test_smallest_and_largest_values():
    note("rows: subnormal and huge float32 blocks, every scale byte")
    k = 32 * 256
    x = np.zeros((1, k), dtype=np.float32)
    for e in range(256):  # one block per binary32 exponent
        blk = x[0, 32 * e:32 * e + 32]
        bits = (np.uint32(min(e, 254)) << np.uint32(23)) | np.random.default_rng(e).integers(0, 1 << 23, 32).astype(np.uint32)
        blk[:] = bits.view(np.float32) * np.where(np.arange(32) % 2, -1, 1)
        blk[8:] /= np.float32(2) ** np.arange(24, dtype=np.float32)
    for fmt in ("mxfp4", "mxfp8"):
        q, d = quantise(x, "f32", fmt)
        want = oracle.quantize_rows(x, fmt)
        same_rows(fmt, k, q, d, want)
        o = torch.zeros(1, k, device="cuda")
        iq4.iq4_dequant_rows(q, q.shape[1], d, d.shape[1], FMT[fmt], 1, k, iq4.IQ4_F32, o, k)
        assert np.array_equal(host(o).astype(np.float64), value(fmt, *want))
    # every code and scale byte, decoded; codes above the quantiser's range too
    codes = np.arange(256, dtype=np.uint8).reshape(1, 256)
    for s in (0, 1, 60, 127, 200, 247, 255):
        scales = np.full((1, 8), s, dtype=np.uint8)
        q, d, ldq, lds = stored("mxfp8", codes, scales, 256)
        o = torch.zeros(1, 256, device="cuda")
        iq4.iq4_dequant_rows(q, ldq, d, lds, FMT["mxfp8"], 1, 256, iq4.IQ4_F32, o, 256)
        with np.errstate(over="ignore"):
            want = value("mxfp8", codes, scales).astype(np.float32)
        assert np.array_equal(host(o), want, equal_nan=True), s


# ---- norm ---------------------------------------------------------------------------------


def norm(x, res, t, gain, eps, y_t=None, fmt=None, store_h=True, over=None):
    """Runs iq4_rmsnorm; returns (h, y, codes, scales) as far as they were asked for."""
    m, k = x.shape
    xd = floats(x, t, k + 16)
    rd = None if res is None else floats(res, t, k + 8)
    ldr = k + 8
    h, ldh = None, 0
    if over == "x":
        h, ldh = xd, k + 16
    elif over == "res":
        h, ldh = rd, k + 8
    elif store_h:
        h, ldh = floats(np.zeros((m, k)), t, k + 24), k + 24
    y = None if y_t is None else floats(np.zeros((m, k)), y_t, k + 8)
    q = d = None
    ldq = lds = 0
    if fmt:
        q, d, ldq, lds = row_buffers(fmt, m, k)
    g = None if gain is None else torch.from_numpy(gain).cuda()
    iq4.iq4_rmsnorm(xd, k + 16, rd, ldr, TYPES[t][0], m, k, g, eps, h, ldh, y, TYPES[y_t or t][0], k + 8,
                    FMT[fmt or "q8_1"], q, ldq, d, lds)
    out = []
    for b in (h, y):
        if b is None:
            out.append(None)
            continue
        v = host(b.double())
        assert np.isnan(v[:, k:]).all()
        out.append(v[:, :k])
    return out[0], out[1], q, d


def norm_oracle(x, res, t, gain, eps):
    return oracle.rmsnorm(x.astype(np.float64), None if res is None else res.astype(np.float64), gain, eps, rounder(t))


def inputs(seed, m, k, t):
    r = rounder(t)
    x = r(acts(seed, m, k).astype(np.float64)).astype(np.float32)
    res = r(3 * acts(seed + 1, m, k).astype(np.float64)).astype(np.float32)
    gain = (1 + 0.3 * np.random.default_rng(seed + 2).standard_normal(k)).astype(np.float32)
    return x, res, gain


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("fmt,m,k", [("q8_1", 1, 32), ("mxfp4", 3, 96), ("mxfp8", 2, 512), ("mxfp4", 5, 544), ("q8_1", 4, 2048),
                                     ("mxfp8", 3, 2592), ("mxfp8", 2, 4096), ("q8_1", 2, 8192), ("mxfp4", 1, 8224),
                                     ("mxfp8", 2, 16384), ("mxfp4", 2, 16416), ("q8_1", 1, 20000)])
def test_norm(t, fmt, m, k):
    note(f"norm: {m} x {k} {t} -> {fmt}")
    x, res, gain = inputs(m + k, m, k, t)
    h, y, q, d = norm(x, res, t, gain, 1e-6, y_t="f32", fmt=fmt)
    hr, yr = norm_oracle(x, res, t, gain, 1e-6)
    assert np.array_equal(h, hr) and np.array_equal(y, yr.astype(np.float64))
    same_rows(fmt, k, q, d, oracle.quantize_rows(yr, fmt))


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("y_t", list(TYPES))
def test_norm_output_types(t, y_t):
    note(f"norm: {t} -> {y_t}, no residual, no gain, no codes")
    x, _, _ = inputs(9, 3, 160, t)
    _, y, _, _ = norm(x, None, t, None, 1e-5, y_t=y_t, store_h=False)
    _, yr = norm_oracle(x, None, t, None, 1e-5)
    assert np.array_equal(y, rounder(y_t)(yr.astype(np.float64)))


@pytest.mark.parametrize("k", [256, 4096, 16640])
@pytest.mark.parametrize("over", ["x", "res", None])
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_norm_sum_in_place(over, t, k):
    note(f"norm: h over {over}, {t}, k = {k}")
    x, res, gain = inputs(12, 3, k, t)
    h, y, q, d = norm(x, res, t, gain, 1e-6, y_t="f32", fmt="mxfp8", store_h=False, over=over)
    hr, yr = norm_oracle(x, res, t, gain, 1e-6)
    assert np.array_equal(y, yr.astype(np.float64))
    same_rows("mxfp8", k, q, d, oracle.quantize_rows(yr, "mxfp8"))
    assert h is None or np.array_equal(h, hr)


@pytest.mark.parametrize("fmt", list(FMT))
def test_norm_zero_rows_nan_rows_and_extremes(fmt):
    note(f"norm: zero, NaN, infinite, tiny and huge rows, {fmt}")
    x, res, gain = inputs(21, 8, 256, "f32")
    res[:] = 0
    x[0] = 0
    x[1, 7] = np.nan
    x[2, 255] = np.inf
    x[3] *= np.float32(1e-30)
    x[4] *= np.float32(1e30)
    x[5] = -0.0
    x[6] = 3.0e38
    for eps in (1e-6, 0.0):
        if eps == 0.0:
            x[0] = x[5] = 1.0
        h, y, q, d = norm(x, res, "f32", gain, eps, y_t="f32", fmt=fmt)
        hr, yr = norm_oracle(x, res, "f32", gain, eps)
        assert np.array_equal(y, yr.astype(np.float64), equal_nan=True)
        assert np.isnan(y[1]).all() and np.isnan(y[2]).all() and np.isfinite(y[[0, 3, 4, 5, 6, 7]]).all()
        same_rows(fmt, 256, q, d, oracle.quantize_rows(yr, fmt))


def test_norm_long_zero_row_with_zero_eps_is_nan():
    note("norm: a zero row with eps = 0 (1 / 0 times 0)")
    x = np.zeros((2, 64), dtype=np.float32)
    x[1] = 1
    _, y, q, d = norm(x, None, "f32", None, 0.0, y_t="f32", fmt="mxfp4", store_h=False)
    assert np.isnan(y[0]).all() and np.all(y[1] == 1)
    assert host(d)[0, 0] == 255 and host(d)[1, 0] != 255


def test_norm_equals_norm_then_quantise():
    note("norm: the fused rows equal the plain row quantised by the row and the q8_1 calls")
    x, res, gain = inputs(31, 4, 4096, "f32")
    for fmt in FMT:
        _, y, q, d = norm(x, res, "f32", gain, 1e-6, y_t="f32", fmt=fmt)
        q2, d2 = quantise(y.astype(np.float32), "f32", fmt)
        assert bits_equal(host(q), host(q2)) and bits_equal(host(d), host(d2))
    q3 = torch.empty(4, 4096, dtype=torch.int8, device="cuda")
    d3 = torch.empty(4, 128, dtype=torch.float16, device="cuda")
    yd = torch.from_numpy(y.astype(np.float32)).cuda()
    iq4.iq4_quantize_q8_1(yd, 4, 4096, 4096, q3, d3)
    assert bits_equal(host(q).view(np.int8), host(q3)) and bits_equal(host(d).view(np.float16), host(d3))


def test_rows_do_not_depend_on_each_other():
    note("norm: 37 rows at once equal the rows one at a time")
    x, res, gain = inputs(41, 37, 1056, "bf16")
    h, y, q, d = norm(x, res, "bf16", gain, 1e-6, y_t="bf16", fmt="mxfp4")
    for r in (0, 17, 36):
        h1, y1, q1, d1 = norm(x[r:r + 1], res[r:r + 1], "bf16", gain, 1e-6, y_t="bf16", fmt="mxfp4")
        assert bits_equal(h1, h[r:r + 1]) and bits_equal(y1, y[r:r + 1])
        assert bits_equal(host(q1), host(q[r:r + 1])) and bits_equal(host(d1), host(d[r:r + 1]))


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("fmt", list(FMT))
def test_large_calls_equal_small_ones(t, fmt):
    """Rows of more than 64 MB are read and written past the L2; their values are those of small calls."""
    m, k = (4100, 4128) if t == "f32" else (8200, 4128)
    note(f"rows: {m} x {k} {t} {fmt} at once and in parts")
    g = torch.Generator(device="cuda").manual_seed(7)
    x = (torch.randn(m, k, device="cuda", generator=g) * 3).to(TYPES[t][1])
    res = torch.randn(m, k, device="cuda", generator=g).to(TYPES[t][1])
    gain = torch.rand(k, device="cuda", generator=g) + 0.5

    def run(a, b):
        """h, y, codes, scales of the norm; codes, scales of x; x decoded, twice; of rows a .. b - 1."""
        xs, rs, n = x[a:b], res[a:b].clone(), b - a
        y = torch.empty(n, k, dtype=TYPES[t][1], device="cuda")
        q, d, ldq, lds = row_buffers(fmt, n, k)
        iq4.iq4_rmsnorm(xs, k, rs, k, TYPES[t][0], n, k, gain, 1e-6, rs, k, y, TYPES[t][0], k, FMT[fmt], q, ldq, d, lds)
        q2, d2, _, _ = row_buffers(fmt, n, k)
        iq4.iq4_quantize_rows(xs, TYPES[t][0], n, k, k, FMT[fmt], q2, ldq, d2, lds)
        back = torch.empty(n, k, dtype=TYPES[t][1], device="cuda")
        iq4.iq4_dequant_rows(q2, ldq, d2, lds, FMT[fmt], n, k, TYPES[t][0], back, k)
        return rs, y, q, d, q2, d2, back

    whole = run(0, m)
    for a, b in ((0, 700), (m // 2, m // 2 + 333), (m - 512, m)):
        for w, p in zip(whole, run(a, b)):
            assert torch.equal(w[a:b].contiguous().view(torch.uint8), p.contiguous().view(torch.uint8))


def test_rows_more_than_32_bits_apart():
    note("rows and norm: two rows 4.3 GB apart")
    k, far = 512, (1 << 30) + 64
    x, res, gain = inputs(51, 2, k, "f32")
    b = torch.zeros(far + k, device="cuda")
    b[:k], b[far:] = torch.from_numpy(x[0]).cuda(), torch.from_numpy(x[1]).cuda()
    q, d, ldq, lds = row_buffers("mxfp8", 2, k)
    iq4.iq4_quantize_rows(b, iq4.IQ4_F32, 2, k, far, FMT["mxfp8"], q, ldq, d, lds)
    want = oracle.quantize_rows(x, "mxfp8")
    same_rows("mxfp8", k, q, d, want)
    o = torch.full((far + k,), -7.0, device="cuda")
    iq4.iq4_dequant_rows(q, ldq, d, lds, FMT["mxfp8"], 2, k, iq4.IQ4_F32, o, far)
    got = np.stack([host(o[:k]), host(o[far:])])
    assert np.array_equal(got.astype(np.float64), value("mxfp8", *want)) and bool((o[k:far] == -7.0).all())
    # the norm with x and its sum there, and codes as far apart
    fq = (1 << 32) + 128
    q = torch.full((fq + 512,), 0xEE, dtype=torch.uint8, device="cuda")
    d = torch.full((2, lds), 0xEE, dtype=torch.uint8, device="cuda")
    rd = torch.from_numpy(res).cuda()
    iq4.iq4_rmsnorm(b, far, rd, k, iq4.IQ4_F32, 2, k, torch.from_numpy(gain).cuda(), 1e-6, b, far, o, iq4.IQ4_F32, far,
                    FMT["mxfp8"], q, fq, d, lds)
    hr, yr = norm_oracle(x, res, "f32", gain, 1e-6)
    assert np.array_equal(np.stack([host(b[:k]), host(b[far:])]).astype(np.float64), hr)
    assert np.array_equal(np.stack([host(o[:k]), host(o[far:])]).astype(np.float64), yr.astype(np.float64))
    two = torch.stack([q[:512], q[fq:]])
    same_rows("mxfp8", k, two, d, oracle.quantize_rows(yr, "mxfp8"))
    assert bool((q[512:fq] == 0xEE).all())


@pytest.mark.parametrize("m,k", [(1 << 14, 1 << 20), ((1 << 14) + 1, (1 << 20) - 64), (1 << 21, 1 << 13)])
def test_largest_calls(m, k):
    """m * k up to the documented 2^34: the binary32 decode alone would take 2^32 lanes.  Every call's rows
    are those of calls of a few thousand rows."""
    note(f"rows: {m} x {k}, decoded, quantised and normed at once and in parts")
    assert (1 << 34) - m * k <= 1 << 20 and m * k <= 1 << 34
    step = (1 << 30) // k
    f4, f8 = FMT["mxfp4"], FMT["mxfp8"]
    q, d, ldq, lds = row_buffers("mxfp4", m, k)
    n = min(step, 1024)
    g = torch.Generator(device="cuda").manual_seed(11)
    codes = torch.randint(0, 256, (n, ldq), dtype=torch.uint8, device="cuda", generator=g)
    codes[:, k // 2:] = 0
    d[:, : k // 32] = torch.randint(120, 134, (1, k // 32), dtype=torch.uint8, device="cuda", generator=g)
    d[:, k // 32:] = 0
    for i in range(0, m, n):  # every run of rows its own
        q[i:i + n] = (codes ^ ((7 * (i // n) + 1) % 256))[: m - i]
    q[:, k // 2:] = 0
    out = torch.full((m, k), -7.0, device="cuda")
    iq4.iq4_dequant_rows(q, ldq, d, lds, f4, m, k, iq4.IQ4_F32, out, k)
    small = torch.empty(step, k, device="cuda")
    for i in range(0, m, step):
        rows = min(step, m - i)
        iq4.iq4_dequant_rows(q[i:], ldq, d[i:], lds, f4, rows, k, iq4.IQ4_F32, small, k)
        assert torch.equal(out[i:i + rows].view(torch.int32), small[:rows].view(torch.int32)), i
    for i in (0, m // 2 - 1, m // 2, m - 1):
        want = oracle.dequant_rows(host(q[i:i + 1, : k // 2]), host(d[i:i + 1, : k // 32]), "mxfp4")
        assert np.array_equal(host(out[i]).astype(np.float64), want[0]), i
    del q, d, small
    for norm_too in (False, True):
        q, d, ldq, lds = row_buffers("mxfp8", m, k)
        q2, d2, _, _ = row_buffers("mxfp8", step, k)

        def call(x, rows, q, d):
            if norm_too:
                iq4.iq4_rmsnorm(x, k, None, 0, iq4.IQ4_F32, rows, k, None, 1e-6, None, 0, None, 0, 0, f8, q, ldq, d, lds)
            else:
                iq4.iq4_quantize_rows(x, iq4.IQ4_F32, rows, k, k, f8, q, ldq, d, lds)

        call(out, m, q, d)
        for i in range(0, m, step):
            rows = min(step, m - i)
            call(out[i:], rows, q2, d2)
            assert torch.equal(q[i:i + rows], q2[:rows]) and torch.equal(d[i:i + rows], d2[:rows]), i
        del q, d, q2, d2


@pytest.mark.parametrize("k", [256, 16640])
@pytest.mark.parametrize("t", list(TYPES))
def test_norm_of_twice_a_row_in_place(t, k):
    note(f"norm: x, its residual and their sum one buffer, {t}, k = {k}")
    x, _, gain = inputs(61, 3, k, t)
    b = floats(x, t)
    q, d, ldq, lds = row_buffers("mxfp8", 3, k)
    iq4.iq4_rmsnorm(b, k, b, k, TYPES[t][0], 3, k, torch.from_numpy(gain).cuda(), 1e-6, b, k, None, 0, 0, FMT["mxfp8"], q, ldq,
                    d, lds)
    hr, yr = norm_oracle(x, x, t, gain, 1e-6)
    assert np.array_equal(host(b.double()), hr)
    same_rows("mxfp8", k, q, d, oracle.quantize_rows(yr, "mxfp8"))
