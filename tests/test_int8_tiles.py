"""The sizes that the GPU parity tests of the 8-bit products run at reach every
tile, whatever the costs that choose one are fitted to (CPU only: the library is
asked, nothing is launched)."""

import ctypes

import pytest

from activation_sparsity_fp4_amd import _lib
from int8_tiles import BEHIND, BF16, DENSE, FP32, GROUPED, SILU, columns, tile, weight_rows

KINDS = (FP32, BF16, SILU)
RING = 6  # the most stages that a tile keeps in flight


@pytest.mark.parametrize("kind", KINDS)
def test_every_dense_tile_is_reached(kind):
    partial = set()
    for T, K, O in DENSE:
        o = weight_rows(O, kind)
        t = tile(T, 0, o, K, kind)
        assert -(-K // 64) > 2 * RING
        filled = T % t[2] == 0 or (o // 2 % (t[3] // 2) if kind == SILU else o % t[3]) == 0 or K % 64 == 0
        if not filled:
            partial.add(t[0])
    assert partial == set(range(t[1]))


def last_heights(sizes, height):
    """Of the row tiles of segments: the full height, and for a last one with fewer rows the loop that it takes (whole,
    half or a quarter of the height, 32 rows at least)."""
    for n in sizes:
        if n >= height:
            yield height
        last = n % height
        if last:
            yield next((h for h in (max(height // 4, 32), height // 2) if last <= h), "whole")


@pytest.mark.parametrize("kind", KINDS)
def test_every_grouped_tile_is_reached(kind):
    """In both orders of the column tiles (in eights and not), and with last row tiles of every height."""
    orders, heights, tall = set(), {}, {}
    for sizes, K, O in GROUPED:
        o = weight_rows(O, kind)
        t = tile(sum(sizes) + BEHIND, len(sizes), o, K, kind)
        orders.add((t[0], columns(o, kind, t) % 8 == 0))
        assert -(-K // 64) > 2 * RING
        if t[2] > 16:  # thin tiles have one height
            tall[t[0]] = t[2]
            heights.setdefault(t[0], set()).update(last_heights(sizes, t[2]))
    assert orders == {(n, eights) for n in range(t[1]) for eights in (False, True)}
    for number, height in tall.items():
        assert heights[number] == {height, height // 2, max(height // 4, 32), "whole"}, number


def test_wide_weights_off_the_eights_are_among_them():
    assert {columns(o, FP32, tile(sum(s) + BEHIND, len(s), o, k, FP32)) for s, k, o in GROUPED} >= {43, 54}


def test_refusals():
    t = (ctypes.c_int32 * 4)()

    def ask(rows=64, E=0, O=256, K=512, kind=0, out=ctypes.addressof(t)):
        return _lib.call("sharq_int8_tile", rows, E, O, K, kind, out)

    assert ask() == ask(E=4) == ask(kind=2) == _lib.SHARQ_OK
    for bad in (dict(rows=0), dict(rows=-1), dict(E=-1), dict(O=0), dict(K=0), dict(kind=3), dict(kind=-1),
                dict(kind=2, O=255), dict(out=0), dict(rows=1 << 25), dict(O=1 << 25), dict(rows=1 << 31, E=4),
                dict(rows=1 << 24, O=1 << 24), dict(rows=1 << 30, E=4, O=1 << 20)):
        assert ask(**bad) == _lib.SHARQ_EINVAL, bad
    assert ask(K=1 << 17) == _lib.SHARQ_ENOTIMPL
