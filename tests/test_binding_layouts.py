"""Arguments whose layout the kernels do not read are refused: strided segments
and gathers, stacks of experts that are no contiguous block, outputs of another
shape (CPU: the library calls are recorded, not made)."""

import pytest
import torch

import activation_sparsity_fp4_amd as sq
from host_stub import on_gpu, record
from test_binding_devices import E, K, O, P, T, tensors, u8


def _every_other(t):
    """The values of t at a stride of 2."""
    wide = torch.zeros(2 * t.numel(), dtype=t.dtype)
    return on_gpu(wide.as_strided((t.numel(),), (2,)))


def _stacks(w):
    """Stacks [E, ..] of w's shape that are not one contiguous block: one expert for all, and a slice of every other."""
    G, R = w.codes.shape[1:3]
    one = sq.MXFP4(on_gpu(torch.zeros(1, G, R, 64, dtype=torch.uint8).expand(E, G, R, 64)), w.scales, K)
    two = sq.MXFP4(w.codes, on_gpu(torch.zeros(2 * E, G, R, 4, dtype=torch.uint8).as_strided(
        (E, G, R, 4), (2 * G * R * 4, R * 4, 4, 1))), K)
    return one, two, sq.MXFP4(w.codes, u8(E - 1, G, R, 4, index=0), K)


CALLS = {"linear_grouped": (sq.linear_grouped, "prep", "we"),
         "linear_grouped_silu_prepare": (sq.linear_grouped_silu_prepare, "prep", "gue"),
         "linear_grouped_mxfp4": (sq.linear_grouped_mxfp4, "mx", "we"),
         "linear_grouped_silu_mxfp4": (sq.linear_grouped_silu_mxfp4, "mx", "gue")}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_grouped(monkeypatch, name):
    calls = record(monkeypatch, sq)
    f, a, w = CALLS[name]
    t = tensors(0)
    a, w, seg, rows = t[a], t[w], t["seg"], t["rows"]
    f(a, w, seg, rows)
    assert len(calls) == 1
    bad = [(a, w, _every_other(seg), rows), (a, w, seg, _every_other(rows)),
           (a, w, on_gpu(torch.zeros(E, dtype=torch.int32)), rows)]
    for args in bad + [(a, s, seg, rows) for s in _stacks(w)]:
        with pytest.raises(ValueError):
            f(*args)
    assert len(calls) == 1


def test_silu_prepare_into(monkeypatch):
    calls = record(monkeypatch, sq)
    t = tensors(0)
    gu, g = t["gu"], sq.stages(K)
    for bad in (gu._replace(scales=u8(g, O, 4, index=0)), gu._replace(scales=gu.scales.as_subclass(torch.Tensor)),
                gu._replace(codes=on_gpu(torch.zeros(g, 4 * O, 64, dtype=torch.uint8)[:, ::2]))):
        with pytest.raises(ValueError):
            sq.linear_silu_prepare_into(t["prep"], bad, t["hp"])
    with pytest.raises(TypeError):
        sq.linear_silu_prepare_into(t["prep"], gu._replace(scales=on_gpu(gu.scales.float())), t["hp"])
    assert not calls


def test_compact_backbone(monkeypatch):
    calls = record(monkeypatch, sq)
    t = tensors(0)
    cb, row = t["cb"], t["cb"].meta.shape[1]
    strided = lambda n: on_gpu(torch.zeros(T, 2 * n, dtype=torch.uint8)[:, :n])  # noqa: E731
    for bad in (cb._replace(codes=strided(K // 4)), cb._replace(meta=strided(row))):
        with pytest.raises(ValueError):
            sq.compress_backbone(t["prep"], out=bad)
        with pytest.raises(ValueError):
            sq.expand_backbone(bad)
    for bad in (cb._replace(codes=u8(T, K // 4 - 1, index=0)), cb._replace(meta=u8(T, row - 1, index=0)),
                cb._replace(meta=u8(T - 1, row, index=0))):
        with pytest.raises(ValueError):
            sq.expand_backbone(bad)
    with pytest.raises(TypeError):
        sq.compress_backbone(t["prep"], out=cb._replace(meta=on_gpu(cb.meta.int())))
    assert not calls


def test_stack_outputs(monkeypatch):
    """quantize_mxfp4 of a stack writes an output of as many experts and of that K."""
    calls = record(monkeypatch, sq)
    x = on_gpu(torch.zeros(E, O, K, dtype=torch.bfloat16))
    w = tensors(0)["we"]
    sq.quantize_mxfp4(x, w)
    assert len(calls) == E
    g = sq.stages(K)
    for bad in (sq.MXFP4(u8(E + 1, g, O, 64, index=0), u8(E + 1, g, O, 4, index=0), K),
                sq.MXFP4(w.codes, u8(E + 1, g, O, 4, index=0), K),
                sq.MXFP4(u8(E - 1, g, O, 64, index=0), u8(E - 1, g, O, 4, index=0), K), w._replace(K=K - 32)):
        with pytest.raises(ValueError):
            sq.quantize_mxfp4(x, bad)
    with pytest.raises(ValueError):
        sq.quantize_mxfp4(on_gpu(torch.zeros(T, K, dtype=torch.bfloat16)), tensors(0)["mx"]._replace(K=K - 32))
    assert len(calls) == E
    assert P == T  # the outputs above stand for pairs as well
