"""Codes of tensors whose rows lie closer together than K entries equal those of
their copies, bit for bit."""

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,strides", [((3, 1, 200), (0, 0, 1)), ((3, 1, 200), (8, 8, 1)), ((3, 2, 200), (0, 0, 1)),
                                           ((3, 2, 200), (16, 8, 1)), ((5, 200), (0, 1)), ((5, 200), (3, 1))])
def test_quantize_overlapping_rows(shape, strides):
    import torch
    import activation_sparsity_fp4_amd as sq
    print(f"quantize {shape} strides {strides}", flush=True)
    memory = torch.randn(4096, device="cuda", generator=torch.Generator(device="cuda").manual_seed(0)).bfloat16()
    x = memory.as_strided(shape, strides)
    got, want = sq.quantize_int8(x), sq.quantize_int8(x.clone(memory_format=torch.contiguous_format))
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    if len(shape) == 2:
        got = sq.quantize_int8(x, rms_eps=1e-5)
        want = sq.quantize_int8(x.clone(memory_format=torch.contiguous_format), rms_eps=1e-5)
        assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
