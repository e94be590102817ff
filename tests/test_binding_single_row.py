"""A single row has no leading dimension: whatever stride its tensor reports,
the library is told the row's length (CPU: the calls are recorded, not made)."""

import pytest
import torch

import activation_sparsity_fp4_amd as sq
from host_stub import on_gpu, record, OnGpu
from test_binding_devices import K, O, u8

# the reported stride of a row: a transposed column, an odd one, an expanded row
STRIDES = [1, 333, 0]


def _row(n, dtype, stride):
    t = torch.zeros(n, dtype=dtype).as_strided((1, n), (stride, 1))
    assert t.stride(0) == stride
    return on_gpu(t)


def _operands():
    g = sq.stages(K)
    prep = sq.Prepared(u8(g, 1, 64, index=0), u8(g, 1, 4, index=0), u8(g, 1, 64, index=0), u8(g, 1, 4, index=0), None, K)
    nv = sq.NVPrepared(u8(g, 1, 64, index=0), u8(g, 1, 8, index=0), u8(g, 1, 64, index=0), u8(g, 1, 8, index=0), None, K,
                       1.0)
    mx = sq.MXFP4(prep.bb_codes, prep.bb_scales, K)
    w = sq.MXFP4(u8(g, O, 64, index=0), u8(g, O, 4, index=0), K)
    return prep, nv, mx, w, sq.NVFP4(w.codes, u8(g, O, 8, index=0), K, 1.0)


@pytest.mark.parametrize("stride", STRIDES)
def test_inputs(monkeypatch, stride):
    calls = record(monkeypatch, sq)
    x = _row(K, torch.bfloat16, stride)
    for f in (lambda: sq.prepare(x), lambda: sq.prepare(x, rms_eps=1e-5), lambda: sq.quantize_mxfp4(x),
              lambda: sq.quantize_mxfp4(x, rms_eps=1e-5), lambda: sq.prepare_nvfp4(x, 1.0),
              lambda: sq.quantize_nvfp4(x, 1.0)):
        del calls[:]
        f()
        entry, args, _ = calls[0]
        assert args[:4] == (x.data_ptr(), 1, K, K), entry


@pytest.mark.parametrize("stride", STRIDES)
@pytest.mark.parametrize("workspace", [0, 4096])
def test_outputs(monkeypatch, stride, workspace):
    calls = record(monkeypatch, sq, workspace)
    prep, nv, mx, w, nvw = _operands()
    y = _row(O, torch.float32, stride)
    for f in (lambda: sq.linear(prep, w, y), lambda: sq.linear_scratchfree(prep, w, y),
              lambda: sq.linear_nvfp4(nv, nvw, y), lambda: sq.linear_mxfp4(mx, w, y)):
        del calls[:]
        f()
        entry, args, _ = calls[0]
        assert args[args.index(y.data_ptr()) + 1] == O, entry


def test_several_rows_keep_theirs(monkeypatch):
    calls = record(monkeypatch, sq)
    x = on_gpu(torch.zeros(2, K + 8, dtype=torch.bfloat16)[:, :K])
    assert isinstance(x, OnGpu)
    for f in (sq.prepare, sq.quantize_mxfp4):
        del calls[:]
        f(x)
        assert calls[0][1][:4] == (x.data_ptr(), 2, K, K + 8)
