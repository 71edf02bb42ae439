"""Host-side checks of the group-scaled products, the experts' rows and SwiGLU: refusals
before anything is enqueued."""
import pytest

import dequant_matmul_iq4_amd as iq4

FAKE = 1 << 20
A, AL, U = iq4.IQ4_E_ARG, iq4.IQ4_E_ALIGN, iq4.IQ4_E_UNSUPPORTED
MX4, MX8, Q8 = iq4.IQ4_ROWS_MXFP4, iq4.IQ4_ROWS_MXFP8, iq4.IQ4_ROWS_Q8_1


def _rc(name, *args):
    return getattr(iq4.lib(), name)(*args)


def test_g4_packed_bytes():
    # code tiles of 16 x 128: 1024 bytes of codes, 16 rows x 1, 2 or 4 scales of two bytes and zero points of one
    assert iq4.iq4_g4_packed_bytes(16, 512, 128, 0) == 4 * (1024 + 32) + 128  # (a multiple of 256)
    assert iq4.iq4_g4_packed_bytes(16, 512, 32, 0) == 4 * (1024 + 128)
    assert iq4.iq4_g4_packed_bytes(16, 512, 64, 1) == 4 * (1024 + 96) + 128
    assert iq4.iq4_g4_packed_bytes(1, 32, 32, 1) == 1024 + 192 + 64 and iq4.iq4_g4_packed_bytes(17, 544, 32, 1) == 10 * 1216 + 128
    for n, k, g in ((0, 32, 32), (16, 0, 32), (16, 40, 32), (16, 128, 16), (16, 128, 256), (1 << 25, 32, 32), (16, 1 << 21, 32)):
        assert iq4.iq4_g4_packed_bytes(n, k, g, 0) == -1


def test_g4_pack_refusals():
    big = FAKE * 64

    def pack(q=FAKE, ldq=64, d=FAKE, lds=4, z=FAKE, ldz=4, n=16, k=128, g=32, p=big):
        return _rc("iq4_g4_pack_weights", q, ldq, d, lds, z, ldz, n, k, g, p, None)

    assert pack(n=0) == A and pack(k=-32) == A and pack(k=48) == U and pack(n=1 << 25) == U and pack(g=16) == U and pack(g=0) == U
    assert pack(ldq=63) == A and pack(lds=3) == A and pack(ldz=3) == A and pack(q=None) == A and pack(d=None) == A and pack(p=None) == A
    assert pack(p=big + 16) == AL and pack(n=1 << 24, k=1 << 20, ldq=1 << 19, lds=1 << 15, ldz=1 << 15) == U
    assert pack(q=big) == A and pack(d=big + 256) == A and pack(z=big + 1024) == A  # overlap


def test_g4_product_refusals():
    def dense(p=FAKE, n=16, k=128, g=32, st=1, z=0, x=FAKE, xt=0, ldx=128, m=4, y=FAKE, yt=0, ldy=16):
        return _rc("iq4_g4_qmv", p, n, k, g, st, z, x, xt, ldx, m, y, yt, ldy, None)

    def grouped(p=FAKE, e=4, n=16, k=128, g=32, st=1, z=0, x=FAKE, xt=0, ldx=128, rows=8, off=FAKE, pairs=FAKE, top=2, m=16, y=FAKE,
                yt=0, ldy=16):
        return _rc("iq4_g4_grouped_qmv", p, e, n, k, g, st, z, x, xt, ldx, rows, off, pairs, top, m, y, yt, ldy, None)

    for f in (dense, grouped):
        assert f(n=0) == A and f(k=0) == A and f(k=100) == U and f(n=1 << 25) == U and f(m=-1) == A and f(m=(1 << 21) + 1) == U
        assert f(g=48) == U and f(st=0) == A and f(st=3) == A and f(xt=3) == A and f(yt=-1) == A and f(ldx=127) == A and f(ldy=15) == A
        assert f(p=None) == A and f(x=None) == A and f(y=None) == A
        assert f(p=FAKE + 16) == AL and f(x=FAKE + 2) == AL and f(y=FAKE + 2) == AL and f(xt=1, x=FAKE + 1) == AL and f(yt=2, y=FAKE + 1) == AL
        assert f(x=FAKE * 4, y=FAKE * 4) == A and f(p=FAKE * 4, x=FAKE * 8, y=FAKE * 4 + 256) == A  # overlaps
    assert dense(m=0, p=None, x=None, y=None) == iq4.IQ4_OK and grouped(m=0, p=None, off=None, y=None) == iq4.IQ4_OK
    assert grouped(e=0) == A and grouped(e=1025) == A and grouped(top=0) == A and grouped(off=None) == A
    assert grouped(off=FAKE + 2) == AL and grouped(pairs=FAKE + 1) == AL
    assert grouped(rows=7) == A and grouped(rows=8, pairs=None, m=9) == A and grouped(rows=-1) == A and grouped(rows=(1 << 30) + 1) == A


def test_slots_refusals():
    far = FAKE * 4

    def disp(x=FAKE, xt=0, ldx=64, t=4, h=64, s=FAKE, w=FAKE, top=2, n=8, r=far, rt=0, ldr=64):
        return _rc("iq4_moe_dispatch", x, xt, ldx, t, h, s, w, top, n, r, rt, ldr, None)

    def comb(r=FAKE, rt=0, ldr=64, n=8, s=FAKE, w=FAKE, t=4, top=2, h=64, add=FAKE, lda=64, o=far, xt=0, ldo=64):
        return _rc("iq4_moe_combine", r, rt, ldr, n, s, w, t, top, h, add, lda, o, xt, ldo, None)

    def grad(x=FAKE, xt=0, ldx=64, r=FAKE, rt=0, ldr=64, n=8, s=FAKE, w=FAKE, t=4, top=2, h=64, dr=far, ldg=64, dw=far * 2):
        return _rc("iq4_moe_combine_grad", x, xt, ldx, r, rt, ldr, n, s, w, t, top, h, dr, ldg, dw, None)

    for f in (disp, comb, grad):
        assert f(t=-1) == A and f(n=-1) == A and f(h=0) == A and f(top=0) == A and f(top=17) == A and f(xt=3) == A and f(rt=-1) == A
        assert f(t=(1 << 23) + 1) == U and f(n=(1 << 24) + 1) == U and f(h=(1 << 20) + 1) == U
        assert f(ldr=63) == A and f(r=None) == A and f(s=None) == A and f(r=FAKE + 2) == AL and f(rt=1, r=FAKE + 1) == AL
        assert f(s=FAKE + 2) == AL and f(w=FAKE + 1) == AL
        assert f(t=0, s=None, r=None) == iq4.IQ4_OK
    for f in (disp, grad):
        assert f(ldx=63) == A and f(x=None) == A and f(x=FAKE + 2) == AL
    assert disp(n=0, x=None, r=None) == iq4.IQ4_OK
    assert comb(o=None) == A and comb(ldo=63) == A and comb(lda=63) == A and comb(add=FAKE + 2) == AL and comb(o=far + 2) == AL
    assert comb(add=far, lda=128) == A  # over the addend, but not row for row
    assert disp(r=FAKE + 64) == A and comb(o=FAKE + 64) == A and grad(dr=FAKE + 64) == A  # overlaps
    assert comb(add=far + 128, o=far) == A and comb(add=far, lda=64, o=far, ldo=128) == A
    assert grad(dr=None, dw=None) == A and grad(ldg=63) == A and grad(dr=far + 1) == AL and grad(dw=far + 2) == AL


def test_swiglu_refusals():
    def fwd(g=FAKE, ldg=128, u=FAKE, ldu=128, t=0, m=2, k=128, y=FAKE * 3, yt=0, ldy=128, fmt=MX8, q=FAKE * 4, ldq=128, d=FAKE * 5, lds=16):
        return _rc("iq4_swiglu", g, ldg, u, ldu, t, m, k, y, yt, ldy, fmt, q, ldq, d, lds, None)

    def grad(dh=FAKE, dt=0, lddh=128, g=FAKE, ldg=128, u=FAKE, ldu=128, t=0, m=2, k=128, dg=FAKE * 3, lddg=128, du=FAKE * 4, lddu=128):
        return _rc("iq4_swiglu_grad", dh, dt, lddh, g, ldg, u, ldu, t, m, k, dg, lddg, du, lddu, None)

    for f in (fwd, grad):
        assert f(t=3) == A and f(m=-1) == A and f(k=0) == A and f(k=(1 << 20) + 32) == U and f(m=(1 << 21) + 1) == U
        assert f(m=1 << 20, k=1 << 20) == U and f(g=None) == A and f(u=None) == A and f(ldg=127) == A and f(ldu=127) == A
        assert f(g=FAKE + 2) == AL and f(t=1, u=FAKE + 1) == AL and f(m=0, g=None, u=None) == iq4.IQ4_OK
    assert fwd(yt=3) == A and fwd(y=None, q=None) == A and fwd(ldy=127) == A and fwd(y=FAKE * 3 + 2) == AL and fwd(k=100) == U
    assert fwd(fmt=7) == A and fwd(d=None) == A and fwd(ldq=64) == A and fwd(q=FAKE + 8) == AL and fwd(fmt=MX4, lds=24) == AL
    assert fwd(fmt=Q8, lds=6) == A
    assert fwd(q=FAKE + 256) == A and fwd(d=FAKE - 16) == A and fwd(q=FAKE * 3 + 512) == A and fwd(d=FAKE * 4 + 128) == A  # overlaps
    assert fwd(y=FAKE) == A and fwd(g=FAKE * 3 + 64) == A and fwd(u=FAKE * 3 - 64) == A  # overlaps
    assert grad(dg=FAKE) == A and grad(du=FAKE * 3) == A and grad(dh=FAKE * 4 + 64, dt=1) == A
    assert grad(dg=FAKE * 3, lddg=256, du=FAKE * 3 + 256, lddu=256) == A  # halves of a buffer's rows, too narrow
    assert grad(dt=3) == A and grad(dh=None) == A and grad(dg=None) == A and grad(du=None) == A
    assert grad(lddh=127) == A and grad(lddg=127) == A and grad(lddu=127) == A and grad(dg=FAKE * 3 + 1) == AL


def test_binding_raises():
    with pytest.raises(iq4.IQ4Error) as e:
        iq4.iq4_g4_qmv(FAKE, 16, 128, 16, 1, 0, FAKE, 0, 128, 1, FAKE, 0, 16, stream=0)
    assert e.value.code == U and "32, 64 or 128" in str(e.value)
