"""A single row has no leading dimension: the plain quantiser takes a [1, K]
tensor of whatever stride it reports, as the norming one does."""

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


def test_plain_quantiser(sq):
    import torch
    rng = np.random.default_rng(2)
    x = bf16_to_gpu(bf16_round(rng.standard_normal((1, 320)).astype(np.float32)))
    column = x.reshape(320, 1).t()
    odd = torch.as_strided(x, (1, 320), (333, 1))
    assert column.stride() != x.stride() and odd.stride(0) % 8
    want = sq.quantize_mxfp4(x)
    for row in (column, odd, x.expand(1, 320)):
        got = sq.quantize_mxfp4(row)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
