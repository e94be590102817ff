"""Sizes of 8-bit products that reach every tile the library chooses from, in every
kind of output, with rows and columns that do not fill the last tile, K no
multiple of 64 and more stages than a tile keeps in flight."""

import ctypes

from activation_sparsity_fp4_amd import _lib

FP32, BF16, SILU = range(3)

# T, K, O; for the gate|up product O is 2 I with I = O // 2
DENSE = [
    (13, 1345, 777), (16, 2100, 513),  # 16 x 32
    (29, 4133, 3001), (17, 1000, 1602),  # 32 x 32
    (61, 16111, 4501), (190, 16111, 1363),  # 64 x 32
    (333, 4127, 1001), (150, 1999, 3001),  # 64 x 64, K in two
    (99, 913, 9001),  # 64 x 128
    (70, 2055, 8501), (70, 2300, 8501),  # 64 x 128, K in two: odd and even numbers of stages
    (200, 955, 11293), (2500, 1031, 8101),  # 128 x 128
    (200, 2055, 11001), (133, 1970, 11055),  # 128 x 128, K in two
    (401, 1981, 9385),  # 128 x 256
    (1297, 941, 8863), (4000, 1000, 8001),  # 256 x 128
    (325, 2499, 11375), (2001, 3101, 4001),  # 256 x 128, K in two
    (389, 4235, 24703), (470, 4300, 24590),  # 256 x 256
]

# rows of each expert, K, O as above
GROUPED = [
    ([0, 1, 16, 17, 3, 8], 1111, 213), ([0, 1, 16, 17, 3, 8], 911, 505),  # 16 x 32
    ([16, 200, 0, 257], 915, 455), ([16, 200, 0, 257], 915, 571),  # 16 x 64
    ([84, 104, 107], 945, 989), ([300, 72, 337], 945, 1101),  # 64 x 128
    ([2053, 1854], 909, 911), ([820] * 9 + [763, 741, 710, 640, 821] * 2 + [900], 907, 141),  # 128 x 128
    ([1280 + 30, 1280 + 60, 1201], 909, 2040), ([1, 2, 0, 1] * 6, 927, 3109),  # 128 x 256
    ([520, 500, 400, 613], 1000, 11008), ([512, 487, 500, 501], 1000, 13801),
    ([640, 256, 700, 690] * 3 + [1300, 1233, 1200], 1855, 533), ([1100, 1204, 1290, 1024, 1199, 1094], 1861, 917),  # 256 x 128
    ([5200, 5301, 5302], 957, 781), ([1100, 1068, 1000, 512, 1200, 1257, 1300], 965, 1905),  # 256 x 256
    ([200, 300, 256, 420, 30, 350, 0, 492], 4096, 11008), ([200, 300, 256, 420, 30, 350, 0, 492], 4100, 13824),
]
BEHIND = 9  # rows behind the last segment


def tile(rows, E, O, K, kind):
    """(number, how many, tokens, weight rows) of the tile of a product."""
    t = (ctypes.c_int32 * 4)()
    status = _lib.call("sharq_int8_tile", rows, E, O, K, kind, ctypes.addressof(t))
    assert status == 0, (status, rows, E, O, K, kind)
    return tuple(t)


def weight_rows(O, kind):
    return O // 2 * 2 if kind == SILU else O


def columns(O, kind, t):
    """Column tiles of a product on tile t."""
    return -(-(O // 2) // (t[3] // 2)) if kind == SILU else -(-O // t[3])
