"""Pins of the plain-product and routing oracles: hand-worked rows, invariants
of the plan, and agreement with the generator of the synthetic workloads."""

import math

import numpy as np
import pytest

from oracle import linear_mxfp4_ref, linear_ref, moe_route_ref, quantize_weight_ref
from synth import bf16_round, moe_combine_index, moe_routing


def test_product_is_the_two_path_product_without_a_residual():
    rng = np.random.default_rng(0)
    a = quantize_weight_ref(bf16_round(rng.standard_normal((5, 96)).astype(np.float32)))
    w = quantize_weight_ref(bf16_round(rng.standard_normal((7, 96)).astype(np.float32)))
    y, bound = linear_mxfp4_ref(*a, *w)
    y2, bound2 = linear_ref(*a, np.zeros_like(a[0]), np.zeros_like(a[1]), *w)
    assert np.array_equal(y, y2) and np.allclose(bound, bound2)


def test_hand_worked_row():
    r = moe_route_ref(np.array([[0.0, math.log(3.0), math.log(2.0), -math.inf]]), 2)
    assert r["expert"].tolist() == [[1, 2]]
    assert np.allclose(r["weight"], [[0.6, 0.4]])
    r = moe_route_ref(np.array([[0.0, math.log(3.0), math.log(2.0), -math.inf]]), 2, renormalize=False, scale=2.0)
    assert np.allclose(r["weight"], [[1.0, 2 / 3]])


def test_bias_moves_the_choice_but_not_the_weight():
    r = moe_route_ref(np.array([[0.0, 1.0, 2.0]]), 1, score="sigmoid", bias=np.array([5.0, 0.0, 0.0]),
                      renormalize=False)
    assert r["expert"].tolist() == [[0]] and np.allclose(r["weight"], [[0.5]])


def test_groups():
    x = np.array([[9.0, 0.0, 5.0, 5.0, 8.0, -9.0]])
    # largest values 9, 5, 8: groups 0 and 2 stay
    assert moe_route_ref(x, 3, groups=3, top_groups=2)["expert"].tolist() == [[0, 4, 1]]
    # sums of sigmoid scores 1.4999, 1.9866, 0.9998: group 1 alone
    r = moe_route_ref(x, 2, score="sigmoid", groups=3, top_groups=1, group_score="sum2")
    assert r["expert"].tolist() == [[2, 3]]


def test_ties_masks_and_padding():
    x = np.array([[1.0, 1.0, 1.0, math.nan], [-math.inf] * 4, [0.0, math.inf, math.inf, 0.0], [1.0, 2.0, 3.0, 4.0]])
    r = moe_route_ref(x, 3, num_tokens=3)
    assert r["expert"].tolist() == [[0, 1, 2], [-1, -1, -1], [1, 2, 0], [-1, -1, -1]]
    assert r["weight"][1].tolist() == [0.0] * 3 and np.allclose(r["weight"][2], [0.5, 0.5, 0.0])
    assert r["seg_offsets"].tolist() == [0, 2, 4, 6, 6]
    assert r["a_rows"].tolist() == [0, 2, 0, 2, 0, 2] + [-1] * 6
    assert r["pair_index"].tolist() == [[0, 2, 4], [-1] * 3, [3, 5, 1], [-1] * 3]


@pytest.mark.parametrize("T,E,k", [(40, 8, 3), (17, 16, 8)])
def test_plan_agrees_with_the_synthetic_routing(T, E, k):
    a_rows, seg, _, wts = moe_routing(np.random.default_rng(5), T, E, k)
    logits = np.random.default_rng(5).standard_normal((T, E), dtype=np.float32)
    r = moe_route_ref(logits, k, renormalize=False)
    assert np.array_equal(r["a_rows"], a_rows) and np.array_equal(r["seg_offsets"], seg)
    idx, w = moe_combine_index(a_rows, wts, T, k)
    for t in range(T):
        mine = dict(zip(r["pair_index"][t].tolist(), r["weight"][t].tolist()))
        want = dict(zip(idx[t].tolist(), w[t].tolist()))
        assert mine.keys() == want.keys()
        assert all(abs(mine[p] - want[p]) < 1e-6 for p in mine)
