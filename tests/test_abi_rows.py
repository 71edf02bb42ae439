"""Host-side checks of the row-format calls: refusals before anything is enqueued."""
import ctypes

import pytest

import dequant_matmul_iq4_amd as iq4

FAKE = 1 << 20
A, AL, U = iq4.IQ4_E_ARG, iq4.IQ4_E_ALIGN, iq4.IQ4_E_UNSUPPORTED
MX4, MX8, Q8 = iq4.IQ4_ROWS_MXFP4, iq4.IQ4_ROWS_MXFP8, iq4.IQ4_ROWS_Q8_1


def _rc(name, *args):
    return getattr(iq4.lib(), name)(*args)


def test_row_bytes():
    assert iq4.iq4_rows_bytes(MX4, 4096) == (2048, 128)
    assert iq4.iq4_rows_bytes(MX8, 4096) == (4096, 128)
    assert iq4.iq4_rows_bytes(Q8, 4096) == (4096, 256)
    assert iq4.iq4_rows_bytes(MX4, 32) == (64, 16) and iq4.iq4_rows_bytes(MX8, 544) == (640, 32)
    assert iq4.iq4_rows_bytes(Q8, 32) == (32, 2)
    for bad in ((3, 32), (-1, 32), (MX4, 0)):
        with pytest.raises(iq4.IQ4Error) as e:
            iq4.iq4_rows_bytes(*bad)
        assert e.value.code == A
    with pytest.raises(iq4.IQ4Error) as e:
        iq4.iq4_rows_bytes(MX4, 48)
    assert e.value.code == U
    assert _rc("iq4_rows_bytes", MX4, 32, None, None) == A


def test_quantize_and_dequant_refusals():
    def quant(x=FAKE, t=0, m=2, k=128, ldx=128, fmt=MX8, q=FAKE, ldq=128, d=FAKE, lds=16):
        return _rc("iq4_quantize_rows", x, t, m, k, ldx, fmt, q, ldq, d, lds, None)

    def back(q=FAKE, ldq=128, d=FAKE, lds=16, fmt=MX8, m=2, k=128, t=0, out=FAKE, ldo=128):
        return _rc("iq4_dequant_rows", q, ldq, d, lds, fmt, m, k, t, out, ldo, None)

    for f in (quant, back):
        assert f(fmt=3) == A and f(t=3) == A and f(m=-1) == A and f(k=0) == A
        assert f(k=100) == U and f(m=(1 << 21) + 1) == U and f(m=1 << 20, k=1 << 20) == U
        assert f(q=None) == A and f(d=None) == A and f(ldq=112) == A and f(lds=0) == A
        assert f(q=FAKE + 8) == AL and f(d=FAKE + 8) == AL and f(ldq=136) == AL and f(lds=24) == AL
        assert f(m=0, q=None, d=None) == iq4.IQ4_OK
    assert quant(x=None) == A and quant(ldx=96) == A and quant(x=FAKE + 8) == AL
    assert quant(ldx=130) == AL and quant(t=1, ldx=132) == AL and quant(t=2, ldx=132) == AL
    assert back(out=None) == A and back(ldo=96) == A and back(out=FAKE + 4) == AL and back(t=2, ldo=132) == AL
    # Q8_1 rows: 8-byte codes, 2-byte scales, no padding
    assert quant(fmt=Q8, ldq=124, lds=8) == A and quant(fmt=Q8, lds=6) == A
    assert quant(fmt=Q8, q=FAKE + 4, lds=8) == AL and quant(fmt=Q8, d=FAKE + 1, lds=8) == AL


def test_rmsnorm_refusals():
    def norm(x=FAKE, ldx=128, res=FAKE, ldr=128, t=0, m=2, k=128, gain=FAKE, eps=1e-6, h=FAKE * 2, ldh=128, y=FAKE * 3,
             yt=0, ldy=128, fmt=MX8, q=FAKE * 4, ldq=128, d=FAKE * 5, lds=16):
        return _rc("iq4_rmsnorm", x, ldx, res, ldr, t, m, k, gain, eps, h, ldh, y, yt, ldy, fmt, q, ldq, d, lds, None)

    assert norm(t=3) == A and norm(yt=5) == A and norm(m=-1) == A and norm(k=0) == A and norm(k=40) == U
    assert norm(eps=-1.0) == A and norm(eps=float("nan")) == A and norm(eps=float("inf")) == A
    assert norm(x=None) == A and norm(y=None, q=None) == A and norm(fmt=7) == A
    assert norm(ldx=64) == A and norm(ldr=64) == A and norm(ldh=64) == A and norm(ldy=64) == A
    assert norm(x=FAKE + 4) == AL and norm(res=FAKE + 4) == AL and norm(h=FAKE + 4) == AL and norm(y=FAKE + 4) == AL
    assert norm(t=1, ldx=132) == AL and norm(yt=1, ldy=132) == AL and norm(gain=FAKE + 4) == AL
    assert norm(q=FAKE + 8) == AL and norm(d=FAKE + 8) == AL and norm(d=None) == A and norm(ldq=64) == A
    # the sum stored over an addend: row for row, and only if there is a sum
    assert norm(h=FAKE, ldh=256) == A and norm(res=FAKE * 2, h=FAKE * 2, ldh=256) == A
    assert norm(h=FAKE, res=None) == A
    assert norm(m=0, x=None, y=None, q=None) == iq4.IQ4_OK


def test_mx_packed_bytes():
    assert iq4.iq4_mx_packed_bytes(16, 512) == 4 * 1024 + 256
    assert iq4.iq4_mx_packed_bytes(4096, 4096) == 4096 * 4096 * 17 // 32
    assert iq4.iq4_mx_packed_bytes(1, 32) == 1024 + 256
    assert iq4.iq4_mx_packed_bytes(17, 544) == 2 * 5 * 1024 + 2 * 2 * 256
    for n, k in ((0, 32), (16, 0), (16, 40), (1 << 25, 32), (16, 1 << 21)):
        assert iq4.iq4_mx_packed_bytes(n, k) == -1


def test_mx_pack_refusals():
    big = FAKE * 64

    def pack(q=FAKE, ldq=64, d=FAKE, lds=4, n=16, k=128, p=big):
        return _rc("iq4_mx_pack_weights", q, ldq, d, lds, n, k, p, None)

    assert pack(n=0) == A and pack(k=-32) == A and pack(k=48) == U and pack(n=1 << 25) == U
    assert pack(ldq=63) == A and pack(lds=3) == A and pack(q=None) == A and pack(d=None) == A and pack(p=None) == A
    assert pack(p=big + 16) == AL
    assert pack(q=big) == A and pack(d=big + 256) == A  # overlap


def test_mx_gemm_refusals():
    def gemm(p=FAKE, n=16, k=128, fmt=MX4, q=FAKE, ldq=64, d=FAKE, lds=16, m=4, y=FAKE, yt=0, ldy=16):
        return _rc("iq4_mx_gemm", p, n, k, fmt, q, ldq, d, lds, m, y, yt, ldy, None)

    def grouped(p=FAKE, e=4, n=16, k=128, fmt=MX4, q=FAKE, ldq=64, d=FAKE, lds=16, rows=8, off=FAKE, pairs=FAKE, top=2, m=16,
                y=FAKE, yt=0, ldy=16):
        return _rc("iq4_mx_grouped_gemm", p, e, n, k, fmt, q, ldq, d, lds, rows, off, pairs, top, m, y, yt, ldy, None)

    for f in (gemm, grouped):
        assert f(n=0) == A and f(k=0) == A and f(k=100) == U and f(n=1 << 25) == U and f(m=-1) == A and f(m=(1 << 21) + 1) == U
        assert f(fmt=Q8) == A and f(fmt=9) == A and f(yt=3) == A and f(ldy=15) == A
        assert f(p=None) == A and f(q=None) == A and f(d=None) == A and f(y=None) == A
        assert f(p=FAKE + 16) == AL and f(q=FAKE + 8) == AL and f(d=FAKE + 8) == AL and f(y=FAKE + 2) == AL
        assert f(yt=1, y=FAKE + 1) == AL and f(ldq=72) == AL and f(lds=20) == AL and f(ldq=48) == A
        assert f(fmt=MX8) == A  # ldq of MXFP4 rows
    assert gemm(m=0, q=None, y=None) == iq4.IQ4_OK
    assert gemm(n=1 << 24, m=1 << 21, ldy=1 << 24) == U and "workgroups" in iq4.iq4_last_error()
    assert grouped(m=0, off=None, y=None) == iq4.IQ4_OK
    assert grouped(e=0) == A and grouped(e=1025) == A and grouped(top=0) == A and grouped(off=None) == A
    assert grouped(off=FAKE + 2) == AL and grouped(pairs=FAKE + 1) == AL
    assert grouped(rows=(1 << 21) + 1) == U and grouped(rows=(1 << 30) + 1, pairs=None) == A
    assert grouped(rows=7) == A and grouped(rows=8, pairs=None, m=9) == A and grouped(rows=-1) == A


def test_binding_raises():
    with pytest.raises(iq4.IQ4Error) as e:
        iq4.iq4_mx_gemm(FAKE, 16, 100, MX4, FAKE, 64, FAKE, 16, 1, FAKE, 0, 16, stream=0)
    assert e.value.code == U and "multiple of 32" in str(e.value)
    n = ctypes.c_int64(0)
    assert _rc("iq4_rows_bytes", MX4, 96, ctypes.byref(n), ctypes.byref(n)) == iq4.IQ4_OK
