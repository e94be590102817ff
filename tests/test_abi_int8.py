"""Argument checks of the 8-bit path at the C boundary, before any HIP call (CPU only)."""

import math

import pytest

from activation_sparsity_fp4_amd import _lib

A, B, C, D, E_, F, G, H = (0x10000 * i for i in range(1, 9))  # fake, aligned device addresses: never dereferenced
OK, EINVAL, EALIGN, ENOTIMPL = _lib.SHARQ_OK, _lib.SHARQ_EINVAL, _lib.SHARQ_EALIGN, _lib.SHARQ_ENOTIMPL


def quant(x=A, dtype=1, E=1, R=4, K=64, ldx=64, codes=B, scales=C):
    return _lib.call("sharq_quantize_int8", x, dtype, E, R, K, ldx, codes, scales, 0)


def test_quantize():
    assert quant(R=0) == OK and quant(E=0, x=0, codes=0) == OK
    for bad in (dict(dtype=3), dict(dtype=-1), dict(E=-1), dict(R=-1), dict(K=0), dict(ldx=63), dict(x=0),
                dict(codes=0), dict(scales=0), dict(R=1 << 25), dict(E=1 << 10, R=1 << 22), dict(E=1 << 40)):
        assert quant(**bad) == EINVAL, bad
    assert quant(K=1 << 17, ldx=1 << 17) == ENOTIMPL
    for bad in (dict(x=A + 1), dict(x=A + 2, dtype=0), dict(codes=B + 8), dict(scales=C + 2)):
        assert quant(**bad) == EALIGN, bad


def rms(x=A, T=4, K=64, ldx=64, gamma=B, eps=1e-5, r=0, codes=C, scales=D):
    return _lib.call("sharq_quantize_int8_rms", x, T, K, ldx, gamma, eps, r, codes, scales, 0)


def test_quantize_rms():
    assert rms(T=0) == OK
    for bad in (dict(eps=0.0), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan), dict(K=0), dict(ldx=32),
                dict(x=0), dict(codes=0), dict(scales=0), dict(T=-1), dict(T=1 << 25)):
        assert rms(**bad) == EINVAL, bad
    assert rms(K=1 << 17, ldx=1 << 17) == ENOTIMPL
    for bad in (dict(x=A + 1), dict(gamma=B + 1), dict(codes=C + 4), dict(scales=D + 1), dict(r=E_ + 2)):
        assert rms(**bad) == EALIGN, bad


@pytest.mark.parametrize("name", ["sharq_pack_int8", "sharq_unpack_int8"])
def test_pack(name):
    def pack(src=A, E=1, R=4, K=64, dst=B):
        return _lib.call(name, src, E, R, K, dst, 0)

    assert pack(R=0, src=0) == OK
    for bad in (dict(src=0), dict(dst=0), dict(R=-1), dict(K=0), dict(E=-2)):
        assert pack(**bad) == EINVAL, bad
    assert pack(K=1 << 17) == ENOTIMPL
    assert (pack(dst=B + 8) if name == "sharq_pack_int8" else pack(src=A + 8)) == EALIGN


def linear(ac=A, asc=B, wc=C, ws=D, bias=0, T=4, O=8, K=65, y=E_, ldy=8, dtype=0):
    return _lib.call("sharq_linear_int8", ac, asc, wc, ws, bias, T, O, K, y, ldy, dtype, 0)


def test_linear():
    assert linear(T=0, ac=0, y=0) == OK and linear(O=0) == OK
    for bad in (dict(T=-1), dict(O=-1), dict(K=0), dict(ldy=7), dict(dtype=2), dict(dtype=-1), dict(ac=0),
                dict(asc=0), dict(wc=0), dict(ws=0), dict(y=0), dict(T=1 << 25), dict(O=1 << 25, ldy=1 << 25),
                dict(T=1 << 20, O=1 << 19, ldy=1 << 19)):
        assert linear(**bad) == EINVAL, bad
    assert linear(K=1 << 17) == ENOTIMPL
    for bad in (dict(ac=A + 8), dict(asc=B + 1), dict(wc=C + 4), dict(ws=D + 2), dict(bias=F + 1), dict(y=E_ + 4)):
        assert linear(**bad) == EALIGN, bad


def silu(ac=A, asc=B, wc=C, ws=D, T=4, I=5, K=64, hc=E_, hs=F, work=G, nbytes=1 << 20):
    return _lib.call("sharq_linear_silu_int8", ac, asc, wc, ws, T, I, K, hc, hs, work, nbytes, 0)


def test_silu():
    size = lambda T, I: _lib.call("sharq_linear_silu_int8_workspace_bytes", T, I)  # noqa: E731
    assert size(4, 5) == 4 * 8 * 2 and size(0, 5) == 0 and size(3, 4096) == 3 * 4096 * 2
    for bad in ((-1, 5), (4, 0), (4, -1), (1 << 25, 8), (4, 1 << 40)):
        assert size(*bad) == 0
    assert silu(T=0, work=0, nbytes=0) == OK
    for bad in (dict(T=-1), dict(I=0), dict(I=-8), dict(K=0), dict(I=1 << 24), dict(ac=0), dict(ws=0), dict(hc=0),
                dict(hs=0), dict(work=0, nbytes=0), dict(work=0), dict(nbytes=63), dict(nbytes=-1),
                dict(T=1 << 23, I=1 << 16)):
        assert silu(**bad) == EINVAL, bad
    assert silu(K=1 << 17) == ENOTIMPL and silu(I=1 << 17) == ENOTIMPL
    for bad in (dict(hc=E_ + 8), dict(hs=F + 2), dict(wc=C + 1), dict(work=G + 8)):
        assert silu(**bad) == EALIGN, bad


def grouped(ac=A, asc=B, T=4, rows=0, seg=C, E=2, wc=D, ws=E_, P=4, O=8, K=65, y=F, dtype=0):
    return _lib.call("sharq_linear_grouped_int8", ac, asc, T, rows, seg, E, wc, ws, P, O, K, y, dtype, 0)


def grouped_silu(ac=A, asc=B, T=4, rows=0, seg=C, E=2, wc=D, ws=E_, P=4, I=7, K=64, hc=F, hs=G, work=H,
                 nbytes=1 << 20):
    return _lib.call("sharq_linear_grouped_silu_int8", ac, asc, T, rows, seg, E, wc, ws, P, I, K, hc, hs, work, nbytes,
                     0)


def test_grouped():
    assert grouped(P=0, T=0) == OK and grouped(O=0) == OK
    for bad in (dict(E=0), dict(P=-1), dict(P=5), dict(T=-1), dict(O=-1), dict(K=0), dict(seg=0), dict(ac=0),
                dict(wc=0), dict(y=0), dict(dtype=2), dict(T=1 << 25), dict(P=1 << 31, rows=G),
                dict(P=1 << 30, rows=G, O=1 << 20)):
        assert grouped(**bad) == EINVAL, bad
    assert grouped(K=1 << 17) == ENOTIMPL
    for bad in (dict(rows=G + 2), dict(seg=C + 1), dict(y=F + 8), dict(ws=E_ + 1)):
        assert grouped(**bad) == EALIGN, bad
    assert grouped_silu(P=0, T=0) == OK
    for bad in (dict(I=0), dict(hc=0), dict(hs=0), dict(P=1 << 25, rows=H), dict(E=-1), dict(work=0, nbytes=0),
                dict(nbytes=4 * 8 * 2 - 1)):
        assert grouped_silu(**bad) == EINVAL, bad
    for bad in (dict(hc=F + 4), dict(hs=G + 1), dict(work=H + 4)):
        assert grouped_silu(**bad) == EALIGN, bad
