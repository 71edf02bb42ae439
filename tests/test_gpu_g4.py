"""Products with 4-bit weights of group scales on the GPU against the oracle.

Most cases hold whole numbers: activations of a few bits and scales that are powers of two, so
that every product and every partial sum, in any order, is a binary32 number and the result has
to be the exact one (rounded once for 16-bit results).

Where the inputs are real, the bound is by the number of additions: a result is a sum of k
products (and of each group's sum times its scale), and each addition is off by at most a whole
step of the magnitudes' sum M (2^-23 M; a matrix instruction may truncate), each group's scaling
by half a step: (k + 2 k / 32 + 64) 2^-23 M, and half a step of y's type of the result itself.
An activation of binary32 enters as two parts (at most 1.001 of its own magnitude), which miss 2^-23 of it
(half a step of what the first leaves, 2^-11 of the value at most) or, of a slice's smallest, 2^-39 of the
slice's largest magnitude: 2^-23 M + 2^-39 max |x| sum |w|.  One of bfloat16 counts in M with the weights
that the sums are made of: |s| (16 + q) in the products, |s| (16 + z) in what is taken off.
"""
import numpy as np
import pytest
import torch

import dequant_matmul_iq4_amd as iq4
import oracle
from gpu_util import bits_equal, dev, host, note
from rows_util import HALF_STEP, TYPES, floats, rounder

pytestmark = pytest.mark.gpu


def weights(seed, n, k, group, zeros, scale, whole):
    """(codes, scales as float64 values of their type, zero points or None)."""
    rng = np.random.default_rng(seed)
    groups = -(-k // group)
    codes = rng.integers(0, 256, (n, k // 2)).astype(np.uint8)
    s = 2.0 ** rng.integers(-1, 2, (n, groups)) if whole else rounder(scale)(0.02 * np.exp(rng.standard_normal((n, groups))))
    return codes, s * rng.choice([1, -1], s.shape), rng.integers(0, 16, (n, groups)).astype(np.uint8) if zeros else None


def pack(codes, scales, zeros, group, scale, out=None):
    n, k = codes.shape[0], 2 * codes.shape[1]
    size = iq4.iq4_g4_packed_bytes(n, k, group, zeros is not None)
    p = torch.full((size,), 0xEE, dtype=torch.uint8, device="cuda") if out is None else out
    d = dev(scales).to(TYPES[scale][1])
    z = None if zeros is None else dev(zeros)
    iq4.iq4_g4_pack_weights(dev(codes), codes.shape[1], d, d.shape[1], z, d.shape[1], n, k, group, p)
    torch.cuda.synchronize()
    return p


def product(p, n, k, group, zeros, scale, x, t, y_t, ldx=None, ldy=None):
    """Y as float64; what lies between its rows is checked to be left alone."""
    m = len(x)
    xd = floats(x, t, ldx)
    y = torch.full((m, ldy or n), -7.0, dtype=TYPES[y_t][1], device="cuda")
    iq4.iq4_g4_qmv(p, n, k, group, TYPES[scale][0], zeros is not None, xd, TYPES[t][0], xd.shape[1], m, y, TYPES[y_t][0], y.shape[1])
    got = host(y.double())
    assert np.all(got[:, n:] == -7.0)
    return got[:, :n]


def unpacked(p, n, k, group, zeros):
    """Codes, scale bytes and zero points read back out of the documented layout."""
    b = host(p)
    kt, rt, per = -(-k // 128), -(-n // 16), 128 // group
    w = b[: rt * kt * 1024].view(np.uint32).reshape(rt, kt, 4, 16, 4)  # row tile, code tile, g, row, block
    q = np.empty((rt, 16, kt, 4, 4, 8), dtype=np.uint8)  # row, code tile, block, g, element
    for nib, e in enumerate((0, 2, 4, 6, 1, 3, 5, 7)):
        q[..., e] = (w >> np.uint32(4 * nib) & np.uint32(15)).transpose(0, 3, 1, 4, 2)
    at = rt * kt * 1024
    s = b[at: at + rt * kt * 16 * per * 2].view(np.uint16).reshape(rt, kt, 16, per).transpose(0, 2, 1, 3).reshape(rt * 16, -1)
    at += rt * kt * 16 * per * 2
    z = b[at: at + rt * kt * 16 * per].reshape(rt, kt, 16, per).transpose(0, 2, 1, 3).reshape(rt * 16, -1) if zeros else None
    return q.reshape(rt * 16, -1), s, z


@pytest.mark.parametrize("n,k,group,zeros", [(1, 32, 32, True), (16, 512, 128, False), (17, 160, 64, True), (35, 1056, 128, True), (48, 640, 32, False)])
def test_packed_layout(n, k, group, zeros):
    note(f"g4: pack {n} x {k} by {group}, zeros {zeros}")
    codes, s, z = weights(n + k, n, k, group, zeros, "f16", False)
    q, sb, zb = unpacked(pack(codes, s, z, group, "f16"), n, k, group, zeros)
    want = np.stack((codes & 15, codes >> 4), 2).reshape(n, k)
    assert np.array_equal(q[:n, :k], want) and not q[n:].any() and not q[:, k:].any()
    groups = s.shape[1]
    assert bits_equal(sb[:n, :groups], s.astype(np.float16).view(np.uint16)) and not sb[n:].any() and not sb[:, groups:].any()
    if zeros:
        assert np.array_equal(zb[:n, :groups], z) and not zb[n:].any() and not zb[:, groups:].any()


def test_pack_takes_any_alignment_and_strides():
    note("g4: pack from unaligned, strided sources")
    n, k, group = 19, 224, 64
    codes, s, z = weights(3, n, k, group, True, "bf16", False)
    want = pack(codes, s, z, group, "bf16")
    buf = torch.zeros(n * 200 + 1, dtype=torch.uint8, device="cuda")
    c = buf[1:].view(n, 200)
    c[:, : k // 2] = dev(codes)
    d = torch.zeros(n * 14 + 1, dtype=torch.uint8, device="cuda")
    d[1:].view(n, 14)[:, :8] = dev(s).to(torch.bfloat16).view(torch.uint8).view(n, 8)
    zz = torch.full((n, 9), 0xFF, dtype=torch.uint8, device="cuda")
    zz[:, :4] = dev(z) | 0xF0  # the low four bits count
    p = torch.full_like(want, 0xEE)
    iq4.iq4_g4_pack_weights(c, 200, d.data_ptr() + 1, 7, zz, 9, n, k, group, p)
    size = 2 * 2 * (1024 + 16 * 2 * 3)  # two row tiles, two code tiles
    assert torch.equal(p[:size], want[:size])


SHAPES = [(1, 32, 32), (16, 128, 128), (17, 160, 32), (5, 544, 64), (48, 672, 128), (100, 2592, 32), (33, 6144, 128), (130, 4096, 64),
          (7, 16416, 32)]


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("n,k,group", SHAPES)
def test_whole_numbers_are_exact(n, k, group, zeros, t):
    # |sum| <= 16416 * 15 * 2 * 4 < 2^22 in steps of 1/2: exact in binary32 in any order
    scale = "bf16" if (n + k) % 3 else "f16"
    codes, s, z = weights(n * k, n, k, group, zeros, scale, True)
    p = pack(codes, s, z, group, scale)
    w = oracle.g4_weights(codes, s, z, group)
    rng = np.random.default_rng(k)
    for i, m in enumerate((1, 2, 3, 4, 5, 8, 15, 16, 17, 31, 33, 64, 65, 130)):
        y_t = list(TYPES)[(i + n) % 3]
        note(f"g4: exact {m} x {n} x {k} by {group}, zeros {zeros}, {t} -> {y_t}, scales {scale}")
        x = rng.integers(-4, 5, (m, k)).astype(np.float64)
        got = product(p, n, k, group, z, scale, x, t, y_t, ldx=k + (i % 4) * 3, ldy=n + i % 3)
        assert np.array_equal(got, rounder(y_t)(oracle.g4_product(w, x))), m


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n,k,group", [(4100, 160, 32), (4100, 640, 128), (4100, 1056, 32), (2100, 2048, 64), (2100, 3584, 128), (2100, 4096, 32),
                                       (20, 6400, 64), (1030, 6400, 128), (600, 8768, 32)])
def test_more_columns_and_longer_rows(n, k, group, t):
    # |sum| <= 8768 * 15 * 2 * 4 < 2^21 in steps of 1/2
    codes, s, z = weights(n * k, n, k, group, True, "f16", True)
    p = pack(codes, s, z, group, "f16")
    w = oracle.g4_weights(codes, s, z, group)
    rng = np.random.default_rng(k)
    for m in (1, 12, 17, 33, 47, 64, 130):
        note(f"g4: exact {m} x {n} x {k} by {group}, {t}")
        x = rng.integers(-4, 5, (m, k)).astype(np.float64)
        assert np.array_equal(product(p, n, k, group, z, "f16", x, t, "f32", ldx=k + m % 2), oracle.g4_product(w, x)), m


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("group", [32, 64, 128])
def test_real_inputs(group, t):
    n, k = 96, 2560
    for m in (1, 4, 7, 23, 64):
        for zeros in (True, False):
            scale = "f16" if zeros else "bf16"
            note(f"g4: real {m} x {n} x {k} by {group}, zeros {zeros}, {t}")
            codes, s, z = weights(m + group, n, k, group, zeros, scale, False)
            rng = np.random.default_rng(m)
            x = rounder(t)(rng.standard_normal((m, k)) * np.exp(rng.standard_normal((m, 1))))
            x = x.astype(np.float32).astype(np.float64) if t == "f32" else x
            w = oracle.g4_weights(codes, s, z, group)
            want, mags = oracle.g4_product(w, x), oracle.g4_product(abs(w), abs(x))
            y_t = "f32" if m != 7 else t
            got = product(pack(codes, s, z, group, scale), n, k, group, z, scale, x, t, y_t)
            own = 0
            if t == "f32":
                own = 2.0**-23 * mags + 2.0**-39 * abs(x).max(1, keepdims=True) * abs(w).sum(1)
            if t == "bf16":
                q = np.stack((codes & 15, codes >> 4), 2).reshape(n, k)
                wide = lambda v: np.repeat(v, group, axis=1)  # noqa: E731
                mags = oracle.g4_product(abs(wide(s)) * (32 + q + (wide(z) if zeros else 8)), abs(x))
            err = (1.001 * (k + 2 * k / 32) + 64) * 2.0**-23 * mags + own
            bound = err + (HALF_STEP[y_t] * (abs(want) + err) if y_t != "f32" else 0)
            assert np.all(abs(got - want) <= bound)
            # what such a bound would hide, the norm of all errors shows: they are of either sign
            if y_t == "f32":
                assert np.linalg.norm(got - want) <= 2e-6 * np.linalg.norm(want)


def test_every_bit_of_an_activation_counts():
    """One activation a row that is not zero, at every place: its product with each code, 29 bits
    of it at most, is off by what its two parts miss (2^-23) and the rounding of their sum (2^-24)."""
    note("g4: single activations over all of binary32")
    n, k, group = 16, 256, 32
    codes, s, z = weights(5, n, k, group, True, "f16", True)
    p = pack(codes, s, z, group, "f16")
    w = oracle.g4_weights(codes, s, z, group)
    rng = np.random.default_rng(6)
    x = np.zeros((k, k))
    size = (rng.integers(0, 1 << 23, k).astype(np.uint32) | (rng.integers(30, 245, k).astype(np.uint32) << np.uint32(23))).view(np.float32)
    x[np.arange(k), np.arange(k)] = size * rng.choice([1, -1], k)
    want = oracle.g4_product(w, x)
    got = product(p, n, k, group, z, "f16", x, "f32", "f32")
    assert np.all(abs(got - want) <= 2 * 2.0**-23 * abs(want))
    for t in ("f16", "bf16"):  # exact: 8 or 11 bits by 4
        v = rounder(t)(np.diag(rng.standard_normal(k) * 2.0 ** rng.integers(-13, 13, k)))
        assert np.array_equal(product(p, n, k, group, z, "f16", v, t, "f32"), oracle.g4_product(w, v))


def test_smallest_and_largest_activations():
    note("g4: subnormal binary16 and huge binary32 and bfloat16 activations")
    n, k, group = 16, 128, 128
    codes = np.full((n, k // 2), 0x99, dtype=np.uint8)  # every weight 1
    s = np.ones((n, 1))
    p = pack(codes, s, None, group, "f16")
    x = np.zeros((3, k))
    x[0, 5], x[1, 7], x[2, 9] = 2.0**-24, 3 * 2.0**-24, -(2.0**-20)
    assert np.array_equal(product(p, n, k, group, None, "f16", x, "f16", "f32"), np.repeat(x.sum(1)[:, None], n, 1))
    for t in ("f32", "bf16"):
        x[0, 5], x[1, 7], x[2, 9] = float(torch.finfo(TYPES[t][1]).max), 2.0**127, -(2.0**-100)
        assert np.array_equal(product(p, n, k, group, None, "f16", x, t, "f32"), np.repeat(x.sum(1)[:, None], n, 1))


@pytest.mark.parametrize("t", list(TYPES))
def test_infinities_and_nan_stay_in_their_rows(t):
    note(f"g4: infinities and NaN, {t}")
    n, k, group = 33, 544, 32
    codes, s, z = weights(8, n, k, group, True, "f16", True)
    p = pack(codes, s, z, group, "f16")
    w = oracle.g4_weights(codes, s, z, group)
    rng = np.random.default_rng(9)
    for m in (3, 20):
        x = rng.integers(-4, 5, (m, k)).astype(np.float64)
        x[0, 40], x[1, 543] = np.inf, -np.inf
        x[2, 17] = np.nan
        got = product(p, n, k, group, z, "f16", x, t, "f32")
        with np.errstate(invalid="ignore"):
            want = np.stack([np.where(w[:, 40] == 0, np.nan, w[:, 40] * np.inf), np.where(w[:, 543] == 0, np.nan, w[:, 543] * -np.inf)])
        assert np.array_equal(got[:2], want, equal_nan=True) and np.isnan(got[2]).all()
        assert np.array_equal(got[3:], oracle.g4_product(w, x[3:]))


# ---- by expert ----------------------------------------------------------------------------


def bank(seed, experts, n, k, group, zeros, scale):
    each = iq4.iq4_g4_packed_bytes(n, k, group, zeros)
    p = torch.full((experts * each,), 0xEE, dtype=torch.uint8, device="cuda")
    ws = []
    for e in range(experts):
        codes, s, z = weights(seed + e, n, k, group, zeros, scale, True)
        pack(codes, s, z, group, scale, p[e * each:(e + 1) * each])
        ws.append(oracle.g4_weights(codes, s, z, group))
    return p, ws


def grouped(p, experts, n, k, group, zeros, scale, x, t, y_t, offsets, pairs, top, n_pairs, ldx=None, ldy=None, stream=None):
    xd = floats(x, t, ldx)
    y = torch.full((n_pairs, ldy or n), -7.0, dtype=TYPES[y_t][1], device="cuda")
    iq4.iq4_g4_grouped_qmv(p, experts, n, k, group, TYPES[scale][0], zeros, xd, TYPES[t][0], xd.shape[1], len(x),
                           dev(np.asarray(offsets, dtype=np.int32)), None if pairs is None else dev(np.asarray(pairs, dtype=np.int32)), top,
                           n_pairs, y, TYPES[y_t][0], y.shape[1], stream=stream)
    got = host(y.double())
    assert np.all(got[:, n:] == -7.0)
    return got[:, :n]


COUNTS = [[1], [0, 0, 3, 0], [4, 1, 0, 2, 9], [17, 0, 65, 1, 3, 140, 0], [2] * 70, [0] * 300 + [5, 0, 33], [3] * 260]


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_by_expert(counts, gather, t):
    e, pairs_n = len(counts), sum(counts)
    n, k, group, zeros = (37, 160, 32, True) if e % 2 else (50, 608, 128, False)
    note(f"g4: {pairs_n} pairs of {e} experts, gather {gather}, {t}")
    p, ws = bank(e, e, n, k, group, zeros, "f16")
    rng = np.random.default_rng(pairs_n)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    top = 3 if gather else 1
    rows = -(-pairs_n // top) if gather else pairs_n
    x = rng.integers(-4, 5, (rows, k)).astype(np.float64)
    order = rng.permutation(rows * top)[:pairs_n] if gather else None
    extra = 5  # rows behind the last expert's: left as they were
    if gather:
        extra = min(extra, rows * top - pairs_n)
        order = np.concatenate([order, np.zeros(extra, dtype=order.dtype)])
    else:
        x = np.concatenate([x, np.full((extra, k), np.nan)])
    y_t = ["f32", "bf16", "f16"][e % 3]
    got = grouped(p, e, n, k, group, zeros, "f16", x, t, y_t, offsets, order, top, pairs_n + extra, ldx=k + e % 5, ldy=n + 1)
    of = np.repeat(np.arange(e), counts)
    for i in range(pairs_n):
        src = x[order[i] // top] if gather else x[i]
        assert np.array_equal(got[i], rounder(y_t)(oracle.g4_product(ws[of[i]], src[None]))[0]), i
    assert np.all(got[pairs_n:] == -7.0)


def test_wrong_offsets_and_pairs_touch_nothing_else():
    note("g4: offsets and pair ids out of range")
    n, k, group, e, m = 32, 128, 32, 4, 12
    p, _ = bank(3, e, n, k, group, False, "f16")
    x = np.ones((6, k))
    for offsets, pairs in (([-5, 3, 2, 40, 99], [-1, 1000] * 6), ([0, 12, 12, 12, 12], [2**31 - 1, -(2**31)] * 6)):
        got = grouped(p, e, n, k, group, False, "f16", x, "f32", "f32", offsets, pairs, 2, m, ldy=n + 8)
        assert got.shape == (m, n)


# ---- as a program has them ------------------------------------------------------------------


def test_captured_and_on_other_streams():
    """A graph of dense and grouped calls, replayed between eager calls, and two streams at once."""
    note("g4: graph and streams")
    n, k, group = 256, 4096, 128
    codes, s, z = weights(11, n, k, group, True, "f16", True)
    p = pack(codes, s, z, group, "f16")
    w = oracle.g4_weights(codes, s, z, group)
    rng = np.random.default_rng(12)
    x = floats(rng.integers(-4, 5, (4, k)), "f32")
    y = torch.zeros(4, n, device="cuda")

    def call(out, stream=None):
        iq4.iq4_g4_qmv(p, n, k, group, iq4.IQ4_F16, 1, x, iq4.IQ4_F32, k, 4, out, iq4.IQ4_F32, n, stream=stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(y)
    for i in range(4):
        v = rng.integers(-4, 5, (4, k)).astype(np.float64)
        x.copy_(dev(v.astype(np.float32)))
        y.fill_(-1)
        graph.replay()
        want = oracle.g4_product(w, v)
        assert np.array_equal(host(y), want)
        eager = torch.zeros(4, n, device="cuda")
        call(eager)
        assert np.array_equal(host(eager), want)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.zeros(4, n, device="cuda") for _ in range(6)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        call(o, a if i % 2 else b)
    torch.cuda.synchronize()
    assert all(np.array_equal(host(o), want) for o in outs)
