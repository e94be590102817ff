"""Rows of a quantised tensor that lie closer together than K entries (expanded
tensors, sliding windows): copied to rows of their own, whatever the number of
rows of an expert (CPU: the library calls are recorded, not made)."""

import pytest
import torch

import activation_sparsity_fp4_amd as sq
from host_stub import on_gpu, record

K = 40

SHAPES = {  # shape, strides
    "experts of one row, all the same": ((3, 1, K), (0, 0, 1)),
    "experts of one row, overlapping": ((3, 1, K), (8, 8, 1)),
    "experts of one row, any stride of the row": ((3, 1, K), (7, 999, 1)),
    "experts of two rows, all the same": ((3, 2, K), (0, 0, 1)),
    "experts of two rows, each the same": ((3, 2, K), (2 * K, 0, 1)),
    "experts of two rows, overlapping": ((3, 2, K), (16, 8, 1)),
    "one expert, rows all the same": ((1, 4, K), (0, 0, 1)),
    "a matrix of equal rows": ((4, K), (0, 1)),
    "a matrix of overlapping rows": ((4, K), (3, 1)),
}


@pytest.mark.parametrize("name", sorted(SHAPES))
def test_rows_closer_than_their_length_are_copied(monkeypatch, name):
    calls = record(monkeypatch, sq)
    shape, strides = SHAPES[name]
    memory = torch.arange(4096, dtype=torch.float32)
    x = on_gpu(memory.as_strided(shape, strides))
    sq.quantize_int8(x)
    (entry, args, _), = calls
    E, R = (1, shape[0]) if len(shape) == 2 else shape[:2]
    assert entry == "sharq_quantize_int8" and args[2:6] == (E, R, K, K)
    assert args[0] != memory.data_ptr()


def test_normed_rows_closer_than_their_length_are_copied(monkeypatch):
    calls = record(monkeypatch, sq)
    memory = torch.zeros(4096, dtype=torch.bfloat16)
    sq.quantize_int8(on_gpu(memory.as_strided((4, K), (0, 1))), rms_eps=1e-5)
    (entry, args, _), = calls
    assert entry == "sharq_quantize_int8_rms" and args[1:4] == (4, K, K) and args[0] != memory.data_ptr()


@pytest.mark.parametrize("shape,strides,ld", [((3, 1, K), (48, 1, 1), 48), ((3, 2, K), (96, 48, 1), 48),
                                              ((4, K), (K, 1), K), ((3, 1, K), (K, 0, 1), K)])
def test_rows_apart_are_read_where_they_are(monkeypatch, shape, strides, ld):
    calls = record(monkeypatch, sq)
    memory = torch.zeros(4096)
    sq.quantize_int8(on_gpu(memory.as_strided(shape, strides)))
    assert calls[0][1][0] == memory.data_ptr() and calls[0][1][5] == ld
