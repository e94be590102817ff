"""Pins of the 8-bit oracle (CPU): codes against enumeration of every code, the
scale rule, ties, degenerate rows; products against Python integers."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import linear_grouped_int8_ref, linear_int8_ref, quantize_int8_ref


def _nearest(x, s):
    """The code nearest to x / s by enumeration in exact arithmetic, ties to the even one."""
    x, s = Fraction(float(x)), Fraction(float(s))
    return min(range(-127, 128), key=lambda q: (abs(x - q * s), q % 2))


@pytest.mark.parametrize("seed", range(4))
def test_codes_are_the_nearest(seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((3, 40)).astype(np.float32)
    if seed == 1:  # subnormal rows: the scale has few bits
        x = (x * np.float32(2.0 ** -135)).astype(np.float32)
    if seed == 2:
        x *= np.float32(1e37)
    codes, scales = quantize_int8_ref(x)
    for i in range(3):
        assert scales[i] == np.float32(Fraction(float(np.abs(x[i]).max())) / 127)
        for k in range(40):
            assert codes[i, k] == _nearest(x[i, k], scales[i])


def test_ties_go_to_the_even_code():
    s = np.float32(0.25)
    x = np.array([[127 * s, 0.5 * s, 1.5 * s, -2.5 * s, -3.5 * s, 125.5 * s, -126.5 * s]], np.float32)
    codes, scales = quantize_int8_ref(x)
    assert scales[0] == s and codes[0].tolist() == [127, 0, 2, -2, -4, 126, -126]


def test_degenerate_rows():
    x = np.zeros((5, 3), np.float32)
    x[1, 1] = np.nan
    x[2, 2] = -np.inf
    x[3] = [2.0 ** -149, 0, -2.0 ** -149]  # amax / 127 rounds to zero
    x[4] = [0, -5, 0]
    codes, scales = quantize_int8_ref(x)
    assert scales[0] == 0 and scales[3] == 0 and np.isnan(scales[1]) and np.isnan(scales[2])
    assert not codes[:4].any() and codes[4].tolist() == [0, -127, 0]


def test_products():
    rng = np.random.default_rng(7)
    qa, qw = rng.integers(-128, 128, (3, 20)).astype(np.int8), rng.integers(-128, 128, (4, 20)).astype(np.int8)
    sa, sw = rng.random(3).astype(np.float32), rng.random(4).astype(np.float32)
    y, p = linear_int8_ref(qa, sa, qw, sw, np.ones(4))
    for t in range(3):
        for o in range(4):
            want = sum(int(a) * int(w) for a, w in zip(qa[t], qw[o])) * float(sa[t]) * float(sw[o])
            assert y[t, o] == pytest.approx(want + 1, rel=1e-15) and p[t, o] == pytest.approx(abs(want), rel=1e-15)
    rows = np.array([2, 0, 7, 1])
    y, _ = linear_grouped_int8_ref(qa, sa, np.stack([qw, qw[::-1]]), np.stack([sw, sw]), [0, 1, 3], rows, 4)
    assert np.array_equal(y[0], linear_int8_ref(qa[2:], sa[2:], qw, sw)[0][0])
    assert np.array_equal(y[1], linear_int8_ref(qa[:1], sa[:1], qw[::-1], sw)[0][0])
    assert not y[2].any() and np.isnan(y[3]).all()
