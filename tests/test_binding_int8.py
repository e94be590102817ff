"""The binding of the 8-bit path: types, shapes, layouts, devices and streams of
its arguments (CPU: the library calls are recorded, not made)."""

import pytest
import torch

import activation_sparsity_fp4_amd as sq
from host_stub import on_gpu, record

T, K, I, E, P = 6, 200, 72, 3, 6
G = 4


def int8(index, k, *rows):
    return sq.Int8(on_gpu(torch.zeros((*rows[:-1], (k + 63) // 64, rows[-1], 64), dtype=torch.int8), index),
                   on_gpu(torch.zeros(rows), index), k)


def tensors(index):
    f = lambda t: on_gpu(t, index)  # noqa: E731
    return dict(x=f(torch.zeros(T, K, dtype=torch.bfloat16)), xe=f(torch.zeros(E, T, K)),
                gamma=f(torch.ones(K, dtype=torch.bfloat16)), q=int8(index, K, T), w=int8(index, K, 2 * I),
                we=int8(index, K, E, 2 * I), h=int8(index, I, T), bias=f(torch.zeros(2 * I)),
                y=f(torch.zeros(T, 2 * I)), seg=f(torch.zeros(E + 1, dtype=torch.int32)),
                rows=f(torch.zeros(P, dtype=torch.int32)), rm=f(torch.zeros(T, K, dtype=torch.int8)),
                rms=f(torch.zeros(T)))


CALLS = {
    "quantize": (lambda x, q: sq.quantize_int8(x, q), ("x", "q")),
    "quantize_norm": (lambda x, q, gamma: sq.quantize_int8(x, q, gamma, 1e-5), ("x", "q", "gamma")),
    "quantize_stack": (lambda xe: sq.quantize_int8(xe), ("xe",)),
    "pack": (lambda rm, rms: sq.pack_int8(rm, rms), ("rm", "rms")),
    "unpack": (lambda q: sq.unpack_int8(q), ("q",)),
    "unpack_stack": (lambda we: sq.unpack_int8(we), ("we",)),
    "linear": (lambda q, w, y, bias: sq.linear_int8(q, w, y, bias=bias), ("q", "w", "y", "bias")),
    "silu": (lambda q, w, h: sq.linear_silu_int8(q, w, h), ("q", "w", "h")),
    "grouped": (lambda q, we, seg, rows, y: sq.linear_grouped_int8(q, we, seg, rows, y),
                ("q", "we", "seg", "rows", "y")),
    "grouped_silu": (lambda q, we, seg, rows, h: sq.linear_grouped_silu_int8(q, we, seg, rows, h),
                     ("q", "we", "seg", "rows", "h")),
}


def pick(names, index, other=None, at=-1):
    here, there = tensors(index), tensors(index if other is None else other)
    return [(there if i == at else here)[n] for i, n in enumerate(names)]


@pytest.mark.parametrize("name", sorted(CALLS))
def test_runs_on_the_device_of_its_tensors(monkeypatch, name):
    calls = record(monkeypatch, sq, 4096)
    f, names = CALLS[name]
    for index in (0, 1, 3):
        del calls[:]
        f(*pick(names, index))
        assert len(calls) == 1
        entry, args, device = calls[0]
        assert device == index and args[-1] == 1000 + index


@pytest.mark.parametrize("name", sorted(n for n, (_, names) in CALLS.items() if len(names) > 1))
def test_refuses_tensors_of_two_devices(monkeypatch, name):
    calls = record(monkeypatch, sq)
    f, names = CALLS[name]
    for at in range(len(names)):
        with pytest.raises(ValueError, match="all tensors must be on"):
            f(*pick(names, 0, 1, at))
    assert not calls


@pytest.mark.parametrize("name,arg", [("linear", 0), ("linear", 1), ("silu", 2), ("quantize", 1), ("unpack", 0)])
def test_refuses_scales_on_another_device(monkeypatch, name, arg):
    record(monkeypatch, sq)
    f, names = CALLS[name]
    args = pick(names, 0)
    args[arg] = args[arg]._replace(scales=pick(names, 1)[arg].scales)
    with pytest.raises(ValueError, match="all tensors must be on"):
        f(*args)


def refused(error, f, *args, **kw):
    with pytest.raises(error):
        f(*args, **kw)


def test_refuses_what_does_not_fit(monkeypatch):
    calls = record(monkeypatch, sq)
    t = tensors(0)
    x, q, w, we, seg, rows = t["x"], t["q"], t["w"], t["we"], t["seg"], t["rows"]
    zeros = lambda *s, dtype=torch.float32: on_gpu(torch.zeros(s, dtype=dtype))  # noqa: E731
    # the quantiser
    refused(TypeError, sq.quantize_int8, [1.0])
    refused(TypeError, sq.quantize_int8, zeros(T, K, dtype=torch.float64))
    refused(TypeError, sq.quantize_int8, zeros(T, K), rms_eps=1e-5)  # the norm reads bfloat16
    refused(ValueError, sq.quantize_int8, torch.zeros(T, K))  # on the CPU
    refused(ValueError, sq.quantize_int8, zeros(K))
    refused(ValueError, sq.quantize_int8, zeros(T, 0))
    refused(ValueError, sq.quantize_int8, on_gpu(torch.zeros(K, T).t()))
    refused(ValueError, sq.quantize_int8, x, gamma=t["gamma"])
    refused(ValueError, sq.quantize_int8, x, gamma=zeros(K - 1, dtype=torch.bfloat16), rms_eps=1e-5)
    refused(TypeError, sq.quantize_int8, x, gamma=zeros(K), rms_eps=1e-5)
    refused(ValueError, sq.quantize_int8, zeros(E, T, K, dtype=torch.bfloat16), rms_eps=1e-5)
    refused(ValueError, sq.quantize_int8, x, int8(0, K, T + 1))
    refused(ValueError, sq.quantize_int8, x, int8(0, K + 1, T))
    # operands
    for bad in (q._replace(K=K + 64), q._replace(K=K - 64), q._replace(scales=zeros(T + 1)),
                q._replace(codes=on_gpu(torch.zeros(T, G, 64, dtype=torch.int8).transpose(0, 1))),
                q._replace(scales=zeros(2 * T)[::2])):
        refused(ValueError, sq.linear_int8, bad, w)
    for bad in (q._replace(codes=zeros(G, T, 64, dtype=torch.uint8)), q._replace(scales=zeros(T, dtype=torch.float64))):
        refused(TypeError, sq.linear_int8, bad, w)
    refused(ValueError, sq.linear_int8, q, int8(0, K + 1, 2 * I))
    refused(ValueError, sq.linear_int8, q, we)
    refused(TypeError, sq.linear_int8, q, w, dtype=torch.float16)
    refused(TypeError, sq.linear_int8, q, w, zeros(T, 2 * I), dtype=torch.bfloat16)
    refused(ValueError, sq.linear_int8, q, w, zeros(T, 2 * I - 1))
    refused(ValueError, sq.linear_int8, q, w, on_gpu(torch.zeros(2 * I, T).t()))
    refused(ValueError, sq.linear_int8, q, w, bias=zeros(2 * I + 1))
    refused(ValueError, sq.linear_int8, q, w, bias=zeros(4 * I)[::2])
    refused(TypeError, sq.linear_int8, q, w, bias=zeros(2 * I, dtype=torch.bfloat16))
    # gate|up
    refused(ValueError, sq.linear_silu_int8, q, int8(0, K, 2 * I - 1))
    refused(ValueError, sq.linear_silu_int8, q, int8(0, K, 0))
    refused(ValueError, sq.linear_silu_int8, q, w, int8(0, I, T + 1))
    refused(ValueError, sq.linear_silu_int8, q, w, int8(0, I + 1, T))
    # segments
    refused(ValueError, sq.linear_grouped_int8, q, w, seg)
    refused(ValueError, sq.linear_grouped_int8, q, we, zeros(E, dtype=torch.int32))
    refused(TypeError, sq.linear_grouped_int8, q, we, zeros(E + 1, dtype=torch.int64))
    refused(TypeError, sq.linear_grouped_int8, q, we, seg, zeros(P))
    refused(ValueError, sq.linear_grouped_int8, q, we, seg, zeros(2 * P, dtype=torch.int32)[::2])
    refused(ValueError, sq.linear_grouped_int8, q, we, seg, rows, zeros(P, 4 * I)[:, :2 * I])
    refused(ValueError, sq.linear_grouped_silu_int8, q, int8(0, K, E, 2 * I + 1), seg, rows)
    refused(ValueError, sq.linear_grouped_silu_int8, q, we, seg, rows, int8(0, I, E, T))
    # packing
    refused(TypeError, sq.pack_int8, zeros(T, K), t["rms"])
    refused(ValueError, sq.pack_int8, t["rm"], zeros(T + 1))
    refused(ValueError, sq.pack_int8, on_gpu(torch.zeros(K, T, dtype=torch.int8).t()), t["rms"])
    assert not calls


@pytest.mark.parametrize("stride", [1, 333, 0])
def test_a_single_row_has_no_leading_dimension(monkeypatch, stride):
    calls = record(monkeypatch, sq)
    x = on_gpu(torch.zeros(K, dtype=torch.bfloat16).as_strided((1, K), (stride, 1)))
    for f in (lambda: sq.quantize_int8(x), lambda: sq.quantize_int8(x, rms_eps=1e-5)):
        del calls[:]
        f()
        name, args, _ = calls[0]
        assert args[5 if name == "sharq_quantize_int8" else 3] == K
    out = on_gpu(torch.zeros(2 * I).as_strided((1, 2 * I), (stride, 1)))
    del calls[:]
    sq.linear_int8(int8(0, K, 1), int8(0, K, 2 * I), out)
    assert calls[0][1][9] == 2 * I


def test_strided_stacks(monkeypatch):
    calls = record(monkeypatch, sq)
    wide = torch.zeros(E, T, K + 8)
    sq.quantize_int8(on_gpu(wide[:, :, :K]))  # rows of K + 8, experts side by side
    assert calls[0][1][2:6] == (E, T, K, K + 8) and calls[0][1][0] == wide.data_ptr()
    sq.quantize_int8(on_gpu(wide.transpose(0, 1)[:, :, :K]))  # the other way round: copied first
    assert calls[1][1][2:6] == (T, E, K, K)
