"""quantize_mxfp4 of a stack of expert weights equals the experts quantised one
by one, for any number of rows: an expert's scale block in the stack then need
not begin on a 16-byte boundary."""

import numpy as np
import pytest

from synth import bf16_round
from gpu_util import bf16_to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sq():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    import activation_sparsity_fp4_amd as sq
    return sq


def test_stack_of_single_rows(sq):
    import torch
    rng = np.random.default_rng(2)
    x = bf16_to_gpu(bf16_round(rng.standard_normal((1, 320)).astype(np.float32)))
    experts = torch.stack([x, 2 * x, -x]).transpose(0, 1).contiguous().transpose(0, 1)  # [3, 1, 320]
    got = sq.quantize_mxfp4(experts)
    for e in range(3):
        one = sq.quantize_mxfp4(experts[e].clone())
        assert torch.equal(got.codes[e], one.codes) and torch.equal(got.scales[e], one.scales)


@pytest.mark.parametrize("E,O,K", [(3, 33, 96), (2, 257, 2080), (5, 7, 128), (4, 1, 32), (3, 8, 256)])
def test_stack_of_any_rows(sq, E, O, K):
    """The whole stack, into a given output with a guard behind it too, and a grouped product against it."""
    import torch
    print(f"stack E={E} O={O} K={K}", flush=True)
    rng = np.random.default_rng(O)
    w = bf16_to_gpu(bf16_round(rng.standard_normal((E * O, K)).astype(np.float32))).view(E, O, K)
    one = [sq.quantize_mxfp4(w[e]) for e in range(E)]
    G = sq.stages(K)
    whole = sq.MXFP4(torch.full((E + 1, G, O, 64), 0xA5, dtype=torch.uint8, device="cuda"),
                     torch.full((E + 1, G, O, 4), 0xA5, dtype=torch.uint8, device="cuda"), K)
    got = sq.quantize_mxfp4(w, sq.MXFP4(whole.codes[:E], whole.scales[:E], K))
    fresh = sq.quantize_mxfp4(w)
    for e in range(E):
        for t in (got, fresh):
            assert torch.equal(t.codes[e], one[e].codes) and torch.equal(t.scales[e], one[e].scales)
    assert (whole.codes[E] == 0xA5).all() and (whole.scales[E] == 0xA5).all()
    a = sq.quantize_mxfp4(w[0])
    seg = torch.arange(E + 1, dtype=torch.int32, device="cuda")
    rows = torch.zeros(E, dtype=torch.int32, device="cuda")
    y = sq.linear_grouped_mxfp4(a, got, seg, rows)
    for e in range(E):
        assert torch.equal(y[e], sq.linear_mxfp4(sq.MXFP4(a.codes[:, :1].contiguous(), a.scales[:, :1].contiguous(), K),
                                                 one[e], split_k=False)[0])
