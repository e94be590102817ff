"""CPU oracle of the 8-bit integer path (NumPy).

Coding by distances: of the 255 multiples of a row's scale the nearest to the
entry, ties to the even one; exact in float64, where an entry and a midpoint
(k + 1/2) s of float32 s are both held without rounding. Products of codes are
summed in int64.
"""

from __future__ import annotations

import numpy as np

__all__ = ["quantize_int8_ref", "linear_int8_ref", "linear_grouped_int8_ref"]


def quantize_int8_ref(x):
    """(codes int8 [R, K], scales float32 [R]) of rows x (values exact in float32)."""
    x = np.asarray(x, dtype=np.float64)
    codes = np.zeros(x.shape, np.int8)
    scales = np.zeros(x.shape[0], np.float32)
    for i, row in enumerate(x):
        if not np.isfinite(row).all():
            scales[i] = np.nan
            continue
        scales[i] = np.float32(np.abs(row).max() / 127.0)
        s = np.float64(scales[i])
        if s == 0:
            continue
        a = np.abs(row)
        k = np.minimum(np.floor(a / s), 127.0)  # may be one off where the quotient rounds: settled below
        k -= k * s > a
        k += (k + 1) * s <= a
        k = np.minimum(k, 127.0)
        middle = (k + 0.5) * s
        k += (a > middle) | ((a == middle) & (k % 2 == 1))
        codes[i] = (np.sign(row) * np.minimum(k, 127.0)).astype(np.int8)
    return codes, scales


def linear_int8_ref(qa, sa, qw, sw, bias=None):
    """(Y, P): the product in float64 and its size |Y - bias|, from row-major codes."""
    s = np.asarray(qa, np.int64) @ np.asarray(qw, np.int64).T
    p = s * np.asarray(sa, np.float64)[:, None] * np.asarray(sw, np.float64)
    return p + (0.0 if bias is None else np.asarray(bias, np.float64)), np.abs(p)


def linear_grouped_int8_ref(qa, sa, qw, sw, seg, rows, P):
    """(Y, |Y|) [P, O]: row p is activation row rows[p] (p without rows; zeros outside the activation) times the
    weight of the expert whose segment holds it; rows of no segment are NaN."""
    y = np.full((P, qw.shape[1]), np.nan)
    src = np.arange(P) if rows is None else np.asarray(rows)
    for e in range(len(seg) - 1):
        for p in range(max(seg[e], 0), min(seg[e + 1], P)):
            inside = 0 <= src[p] < len(qa)
            y[p] = linear_int8_ref(qa[src[p]][None], sa[src[p]][None], qw[e], sw[e])[0][0] if inside else 0.0
    return y, np.abs(y)
