"""Routing with biases at the ends of float32's range (an expert taken out of
service by its type's lowest value, infinities): the sums that groups are judged
by pass float32's range, and the choice is still float64's. Against the float64
oracle, as the other routing tests."""

import numpy as np
import pytest

from oracle import moe_route_ref
from gpu_util import f32_to_gpu, to_np

pytestmark = pytest.mark.gpu

LOWEST = float(np.finfo(np.float32).min)


@pytest.fixture(scope="module")
def sq():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import activation_sparsity_fp4_amd as sq
    return sq


def _check(sq, x, k, **kw):
    bias = kw.pop("bias")
    r = sq.moe_route(f32_to_gpu(x), k, bias=f32_to_gpu(bias), **kw)
    ref = moe_route_ref(x, k, bias=bias, **kw)
    for name in ("expert", "seg_offsets", "a_rows", "pair_index"):
        assert np.array_equal(to_np(getattr(r, name)), ref[name]), name
    w = to_np(r.weight).astype(np.float64)
    assert np.all(np.abs(w - ref["weight"]) <= np.abs(ref["weight"]) * (2.0 ** -24 + 2.0 ** -45) + 2.0 ** -150)
    return ref


# per group: the bias of its experts (None: their logits are -inf, so that nothing of it can be chosen)
GROUPS = {"lowest behind a group of nothing": [None, LOWEST, LOWEST, None],
          "sums below the lowest value": [-3e38, -2e38, None, -2.5e38],
          "sums past the largest": [2e38, 3e38, 2.5e38, 0.0],
          "infinity beside a sum past the largest": [3e38, np.inf, 3e38, np.inf],
          "one group in service": [LOWEST, LOWEST, 0.25, LOWEST],
          "mixed": [None, LOWEST, 3e38, -2e38]}


@pytest.mark.parametrize("E", [16, 60, 128, 256, 1024])
@pytest.mark.parametrize("pattern", sorted(GROUPS))
@pytest.mark.parametrize("gscore", ["sum2", "max"])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_group_sums_past_the_range(sq, E, pattern, gscore, score):
    print(f"group sums E={E} {pattern} {gscore} {score}", flush=True)
    rng = np.random.default_rng(E)
    x = rng.standard_normal((9, E)).astype(np.float32)
    bias = np.zeros(E, np.float32)
    for g, b in enumerate(GROUPS[pattern]):
        part = slice(g * (E // 4), (g + 1) * (E // 4))
        if b is None:
            x[:, part] = -np.inf
        else:
            bias[part] = b
    for top in (1, 2, 3):
        _check(sq, x, 3, score=score, bias=bias, groups=4, top_groups=top, group_score=gscore)


def test_single_experts_out_of_service(sq):
    """The lowest value as the bias of some experts, others in service in every group."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)).astype(np.float32)
    bias = (0.1 * rng.standard_normal(64)).astype(np.float32)
    out = rng.choice(64, 20, replace=False)
    bias[out] = LOWEST
    for gscore in ("sum2", "max"):
        ref = _check(sq, x, 6, score="sigmoid", bias=bias, groups=8, top_groups=3, group_score=gscore)
        assert not np.isin(ref["expert"], out).any()
    _check(sq, x, 50, score="sigmoid", bias=bias)
