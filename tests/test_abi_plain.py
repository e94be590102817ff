"""Argument checks of the plain MXFP4 products, the norming quantiser, the bf16
combine and the routing at the C boundary, before any HIP call (CPU only)."""

import math

import pytest

from activation_sparsity_fp4_amd import _lib

A, B, C, D, E_, F, G, H = (0x10000 * i for i in range(1, 9))  # fake, aligned device addresses: never dereferenced
OK, EINVAL, EALIGN, ENOTIMPL = _lib.SHARQ_OK, _lib.SHARQ_EINVAL, _lib.SHARQ_EALIGN, _lib.SHARQ_ENOTIMPL


def linear(ac=A, asc=B, wc=C, ws=D, T=4, O=8, K=64, y=E_, ldy=8, dtype=0, work=0, nbytes=0):
    return _lib.call("sharq_linear_mxfp4", ac, asc, wc, ws, T, O, K, y, ldy, dtype, work, nbytes, 0)


def test_linear():
    assert linear(T=0) == OK and linear(O=0) == OK
    assert linear(T=0, ac=0, y=0) == OK
    for bad in (dict(T=-1), dict(O=-1), dict(K=0), dict(K=48), dict(ldy=7), dict(dtype=2), dict(dtype=-1),
                dict(ac=0), dict(asc=0), dict(wc=0), dict(ws=0), dict(y=0), dict(nbytes=-1), dict(nbytes=16),
                dict(T=1 << 25), dict(O=1 << 25, ldy=1 << 25), dict(T=1 << 24, O=1 << 16, ldy=1 << 16)):
        assert linear(**bad) == EINVAL, bad
    for bad in (dict(ac=A + 8), dict(asc=B + 1), dict(wc=C + 4), dict(ws=D + 2), dict(y=E_ + 4),
                dict(work=F + 8, nbytes=64)):
        assert linear(**bad) == EALIGN, bad


def test_workspace_sizes():
    size = lambda T, O, K: _lib.call("sharq_linear_mxfp4_workspace_bytes", T, O, K)  # noqa: E731
    assert size(1, 8192, 28672) > 0  # one token, long K: split
    assert size(1, 8192, 28672) % (8192 * 4) == 0
    assert size(4096, 28672, 4096) == 0  # tiles fill the GPU
    for bad in ((-1, 8, 64), (1, -1, 64), (1, 8, 48), (1, 8, 0), (0, 8, 4096), (1, 0, 4096), (1 << 40, 8, 64)):
        assert size(*bad) == 0
    silu = lambda T, I, K: _lib.call("sharq_linear_silu_mxfp4_workspace_bytes", T, I, K)  # noqa: E731
    assert silu(1, 4096, 28672) == size(1, 8192, 28672)
    assert silu(1, -4, 64) == 0 and silu(1, 1 << 40, 64) == 0


def silu(ac=A, asc=B, wc=C, ws=D, T=4, I=32, K=64, hc=E_, hs=F, work=0, nbytes=0):
    return _lib.call("sharq_linear_silu_mxfp4", ac, asc, wc, ws, T, I, K, hc, hs, work, nbytes, 0)


def test_silu():
    assert silu(T=0) == OK
    for bad in (dict(T=-1), dict(I=0), dict(I=-32), dict(I=16), dict(K=16), dict(I=1 << 24), dict(hc=0), dict(hs=0),
                dict(ac=0), dict(ws=0), dict(nbytes=16), dict(T=1 << 24, I=1 << 16)):
        assert silu(**bad) == EINVAL, bad
    for bad in (dict(hc=E_ + 8), dict(hs=F + 4), dict(wc=C + 1), dict(work=G + 1)):
        assert silu(**bad) == EALIGN, bad


def grouped(ac=A, asc=B, T=4, rows=0, seg=C, E=2, wc=D, ws=E_, P=4, O=8, K=64, y=F, dtype=0):
    return _lib.call("sharq_linear_grouped_mxfp4", ac, asc, T, rows, seg, E, wc, ws, P, O, K, y, dtype, 0)


def grouped_silu(ac=A, asc=B, T=4, rows=0, seg=C, E=2, wc=D, ws=E_, P=4, I=32, K=64, hc=F, hs=G):
    return _lib.call("sharq_linear_grouped_silu_mxfp4", ac, asc, T, rows, seg, E, wc, ws, P, I, K, hc, hs, 0)


def test_grouped():
    assert grouped(P=0, T=0) == OK and grouped(O=0) == OK
    for bad in (dict(E=0), dict(P=-1), dict(P=5), dict(T=-1), dict(O=-1), dict(K=40), dict(seg=0), dict(ac=0),
                dict(wc=0), dict(y=0), dict(dtype=2), dict(T=1 << 25), dict(P=1 << 31, rows=G),
                dict(P=1 << 30, rows=G, O=1 << 20)):
        assert grouped(**bad) == EINVAL, bad
    assert grouped(rows=G + 2) == EALIGN and grouped(seg=C + 1) == EALIGN and grouped(y=F + 8) == EALIGN
    assert grouped_silu(P=0, T=0) == OK
    for bad in (dict(I=0), dict(I=48), dict(hc=0), dict(hs=0), dict(P=1 << 25, rows=H), dict(E=-1)):
        assert grouped_silu(**bad) == EINVAL, bad
    assert grouped_silu(hc=F + 4) == EALIGN and grouped_silu(hs=G + 4) == EALIGN


def quant(x=A, T=4, K=64, ldx=64, gamma=B, eps=1e-5, r=0, codes=C, scales=D):
    return _lib.call("sharq_quantize_mxfp4_rms", x, T, K, ldx, gamma, eps, r, codes, scales, 0)


def test_quantize_rms():
    assert quant(T=0) == OK
    for bad in (dict(eps=0.0), dict(eps=-1.0), dict(eps=math.inf), dict(eps=math.nan), dict(K=48), dict(ldx=32),
                dict(x=0), dict(codes=0), dict(scales=0), dict(T=-1)):
        assert quant(**bad) == EINVAL, bad
    assert quant(K=1 << 18, ldx=1 << 18) == ENOTIMPL
    for bad in (dict(ldx=68), dict(x=A + 2), dict(gamma=B + 2), dict(codes=C + 1), dict(scales=D + 8), dict(r=E_ + 2)):
        assert quant(**bad) == EALIGN, bad


def combine(y=A, P=4, H=8, idx=B, w=C, T=2, k=2, out=D, out16=0):
    return _lib.call("sharq_moe_combine_bf16", y, P, H, idx, w, T, k, out, out16, 0)


def test_combine_bf16():
    assert combine(T=0) == OK
    for bad in (dict(H=6), dict(H=0), dict(k=0), dict(k=65), dict(out=0), dict(y=0), dict(idx=0), dict(w=0),
                dict(P=-1), dict(T=-1)):
        assert combine(**bad) == EINVAL, bad
    for bad in (dict(y=A + 8), dict(out=D + 4), dict(out=0, out16=E_ + 8), dict(idx=B + 2), dict(w=C + 1)):
        assert combine(**bad) == EALIGN, bad


def route(x=A, dtype=0, T=4, E=8, ld=8, bias=0, k=2, score=0, groups=1, top=1, gscore=0, renorm=1, scale=1.0, n=0,
          ids=B, w=C, seg=D, rows=E_, idx=F, work=0, nbytes=0):
    return _lib.call("sharq_moe_route", x, dtype, T, E, ld, bias, k, score, groups, top, gscore, renorm, scale, n, ids,
                     w, seg, rows, idx, work, nbytes, 0)


def test_route():
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(ld=7), dict(dtype=3), dict(score=2), dict(gscore=2),
                dict(groups=3), dict(groups=0), dict(groups=4, top=5), dict(groups=4, top=0),
                dict(groups=4, top=1, k=3), dict(scale=math.nan), dict(scale=math.inf), dict(x=0), dict(ids=0),
                dict(w=0), dict(seg=0), dict(rows=0), dict(idx=0), dict(nbytes=16), dict(T=1 << 30, k=4),
                dict(T=1 << 31), dict(T=65)):
        assert route(**bad) == EINVAL, bad
    assert route(E=1025, ld=1025) == ENOTIMPL
    assert route(E=128, ld=128, k=65) == ENOTIMPL
    for bad in (dict(x=A + 2), dict(x=A + 1, dtype=1), dict(bias=G + 1), dict(n=G + 2), dict(ids=B + 1),
                dict(w=C + 2), dict(seg=D + 1), dict(rows=E_ + 2), dict(idx=F + 3), dict(T=65, work=G + 4, nbytes=1 << 20)):
        assert route(**bad) == EALIGN, bad


@pytest.mark.parametrize("T", [0, 1, 64, 65, 4096, 16384, 1 << 20])
def test_route_workspace(T):
    size = _lib.call("sharq_moe_route_workspace_bytes", T, 128)
    assert size % (128 * 4) == 0 and size <= 256 * 128 * 4
    assert (size == 0) == (T <= 64)
    assert _lib.call("sharq_moe_route_workspace_bytes", T, 0) == 0
    assert _lib.call("sharq_moe_route_workspace_bytes", -1, 8) == 0
