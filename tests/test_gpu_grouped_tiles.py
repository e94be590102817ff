"""Every tile of the grouped fused gate|up call is written: outputs are filled
with a pattern first, then compared bit for bit with the chain linear_grouped ->
silu_mul -> prepare, and rows behind the last segment keep the pattern. Segments
whose last row tiles just fill the grid's bound of ceil(P / 128) + E row tiles
(few experts, narrow h), and plans that the routing makes."""

import numpy as np
import pytest

from oracle import moe_route_ref
from synth import bf16_round
from gpu_util import bf16_to_gpu, f32_to_gpu, i32_to_gpu, to_np

pytestmark = pytest.mark.gpu

CODES = ("bb_codes", "bb_scales", "res_codes", "res_scales")
FILL = 0xA5


@pytest.fixture(scope="module")
def sq():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import activation_sparsity_fp4_amd as sq
    return sq


def _inputs(sq, rng, T, E, K, I):
    x = bf16_to_gpu(bf16_round(rng.standard_normal((T, K)).astype(np.float32)))
    w = bf16_to_gpu(bf16_round((rng.standard_normal((E * 2 * I, K)) * 0.05).astype(np.float32)))
    return sq.prepare(x, None, 2, 4), sq.quantize_mxfp4(w.view(E, 2 * I, K))


def _check(sq, p, w, seg, a_rows, P, I, n, m):
    import torch
    rows = int(to_np(seg)[-1])
    want_h = sq.silu_mul(sq.linear_grouped(p, w, seg, a_rows))
    want = sq.prepare(want_h, None, n, m)
    out = sq.prepare(torch.zeros((P, I), dtype=torch.bfloat16, device="cuda"), None, n, m)
    for f in (*CODES, "mask"):
        getattr(out, f).fill_(FILL)
    hp, h = sq.linear_grouped_silu_prepare(p, w, seg, a_rows, n, m, with_h=True, out=out)
    assert hp is out
    assert torch.equal(h[:rows].view(torch.int16), want_h[:rows].view(torch.int16)), "h"
    for f in CODES:
        got = getattr(out, f)
        assert torch.equal(got[:, :rows], getattr(want, f)[:, :rows]), f
        assert (got[:, rows:] == FILL).all(), f
    assert torch.equal(out.mask[:rows], want.mask[:rows]) and (out.mask[rows:] == FILL).all()


@pytest.mark.parametrize("I,counts", [(256, [640]), (128, [1152]), (128, [600, 553]), (640, [129, 257]),
                                      (384, [1, 385, 0, 513, 129]), (128, [129] * 16), (128, [128] * 3 + [897]),
                                      (256, [0, 0, 1300]), (128, [1])])
@pytest.mark.parametrize("n,m", [(2, 4), (8, 16)])
def test_segments_that_fill_the_grid(sq, I, counts, n, m):
    print(f"grouped fused I={I} counts={counts} {n}:{m}", flush=True)
    rng = np.random.default_rng(I + len(counts))
    P = sum(counts)
    p, w = _inputs(sq, rng, P, len(counts), 128, I)
    _check(sq, p, w, i32_to_gpu(np.concatenate([[0], np.cumsum(counts)])), None, P, I, n, m)


@pytest.mark.parametrize("T,E,k,I,pad", [(1, 5, 3, 128, 0), (40, 5, 2, 128, 3), (700, 2, 1, 128, 60),
                                         (650, 3, 2, 256, 1), (1000, 16, 2, 128, 24), (300, 8, 8, 384, 0),
                                         (640, 1, 1, 256, 0)])
def test_routed_plans(sq, T, E, k, I, pad):
    """A padded batch routed on the device, rows gathered: the h of every pair, and nothing behind the pairs."""
    print(f"routed grouped fused T={T} E={E} k={k} I={I} pad={pad}", flush=True)
    rng = np.random.default_rng(T + E)
    p, w = _inputs(sq, rng, T + pad, E, 256, I)
    logits = (2 * rng.standard_normal(E) + rng.standard_normal((T + pad, E))).astype(np.float32)
    r = sq.moe_route(f32_to_gpu(logits), k, num_tokens=i32_to_gpu([T]))
    ref = moe_route_ref(logits, k, num_tokens=T)
    assert np.array_equal(to_np(r.seg_offsets), ref["seg_offsets"]) and np.array_equal(to_np(r.a_rows), ref["a_rows"])
    _check(sq, p, w, r.seg_offsets, r.a_rows, (T + pad) * k, I, 2, 4)
