"""Every entry point of the binding works on the device of its tensors, whatever
device is current, and refuses tensors of several devices (CPU: no GPU needed,
the library calls are recorded, not made)."""

import pytest
import torch

import activation_sparsity_fp4_amd as sq
from host_stub import on_gpu, record

T, K, O, E, P = 8, 256, 128, 2, 8


def u8(*shape, index):
    return on_gpu(torch.zeros(shape, dtype=torch.uint8), index)


def tensors(index):
    """The arguments of every entry point, on GPU `index`."""
    g = sq.stages(K)
    prep = sq.Prepared(u8(g, T, 64, index=index), u8(g, T, 4, index=index), u8(g, T, 64, index=index),
                       u8(g, T, 4, index=index), u8(T, K // 8, index=index), K)
    hp = sq.Prepared(u8(1, T, 64, index=index), u8(1, T, 4, index=index), u8(1, T, 64, index=index),
                     u8(1, T, 4, index=index), u8(T, O // 8, index=index), O)
    nv = sq.NVPrepared(u8(g, T, 64, index=index), u8(g, T, 8, index=index), u8(g, T, 64, index=index),
                       u8(g, T, 8, index=index), None, K, 1.0)
    f = lambda t: on_gpu(t, index)  # noqa: E731
    return dict(
        x=f(torch.zeros(T, K, dtype=torch.bfloat16)), gamma=f(torch.ones(K, dtype=torch.bfloat16)), prep=prep, hp=hp,
        nv=nv, w=sq.MXFP4(u8(g, O, 64, index=index), u8(g, O, 4, index=index), K),
        gu=sq.MXFP4(u8(g, 2 * O, 64, index=index), u8(g, 2 * O, 4, index=index), K),
        we=sq.MXFP4(u8(E, g, O, 64, index=index), u8(E, g, O, 4, index=index), K),
        gue=sq.MXFP4(u8(E, g, 2 * O, 64, index=index), u8(E, g, 2 * O, 4, index=index), K),
        nvw=sq.NVFP4(u8(g, O, 64, index=index), u8(g, O, 8, index=index), K, 1.0),
        seg=f(torch.zeros(E + 1, dtype=torch.int32)), rows=f(torch.zeros(P, dtype=torch.int32)),
        y=f(torch.zeros(T, O)), gate=f(torch.zeros(T, 2 * O)), h=f(torch.zeros(T, O, dtype=torch.bfloat16)),
        pairs=f(torch.zeros(T, 1, dtype=torch.int32)), weights=f(torch.zeros(T, 1)),
        rm=u8(T, K // 2, index=index), rms=u8(T, K // 32, index=index), nrms=u8(T, K // 16, index=index),
        mx=sq.MXFP4(u8(g, T, 64, index=index), u8(g, T, 4, index=index), K),
        cb=sq.CompactBackbone(u8(T, K // 4, index=index),
                              u8(T, sq._lib.call("sharq_backbone_meta_row_bytes", K, 2, 4), index=index), 2, 4, K))


# a call, and the arguments (names of `tensors`) that it takes
CALLS = {
    "prepare": (lambda x, gamma, prep: sq.prepare(x, gamma, out=prep), ("x", "gamma", "prep")),
    "prepare_rms": (lambda x, gamma: sq.prepare(x, gamma, rms_eps=1e-5), ("x", "gamma")),
    "quantize": (lambda x, mx: sq.quantize_mxfp4(x, mx), ("x", "mx")),
    "quantize_rms": (lambda x, mx, gamma: sq.quantize_mxfp4(x, mx, gamma, 1e-5), ("x", "mx", "gamma")),
    "linear": (lambda prep, w, y: sq.linear(prep, w, y), ("prep", "w", "y")),
    "linear_whole": (lambda prep, w, y: sq.linear(prep, w, y, split_k=False), ("prep", "w", "y")),
    "linear_scratchfree": (lambda prep, w, y: sq.linear_scratchfree(prep, w, y), ("prep", "w", "y")),
    "linear_grouped": (lambda prep, we, seg, rows, y: sq.linear_grouped(prep, we, seg, rows, y),
                       ("prep", "we", "seg", "rows", "y")),
    "linear_silu_prepare": (lambda prep, gu: sq.linear_silu_prepare(prep, gu, with_h=True), ("prep", "gu")),
    "linear_silu_prepare_into": (lambda prep, gu, hp: sq.linear_silu_prepare_into(prep, gu, hp, split_k=False),
                                 ("prep", "gu", "hp")),
    "linear_grouped_silu_prepare": (
        lambda prep, gue, seg, rows, hp: sq.linear_grouped_silu_prepare(prep, gue, seg, rows, out=hp),
        ("prep", "gue", "seg", "rows", "hp")),
    "compress": (lambda prep, cb: sq.compress_backbone(prep, out=cb), ("prep", "cb")),
    "expand": (lambda cb, mask: sq.expand_backbone(cb, mask=mask), ("cb", "prep.mask")),
    "combine": (lambda y, pairs, weights: sq.moe_combine(y, pairs, weights), ("y", "pairs", "weights")),
    "combine_bf16": (lambda h, pairs, weights: sq.moe_combine(h, pairs, weights), ("h", "pairs", "weights")),
    "silu_mul": (lambda gate, h: sq.silu_mul(gate, h), ("gate", "h")),
    "prepare_nvfp4": (lambda x, gamma, nv: sq.prepare_nvfp4(x, 1.0, gamma, out=nv), ("x", "gamma", "nv")),
    "quantize_nvfp4": (lambda x: sq.quantize_nvfp4(x, 1.0), ("x",)),
    "linear_nvfp4": (lambda nv, nvw, y: sq.linear_nvfp4(nv, nvw, y), ("nv", "nvw", "y")),
    "pack_mxfp4": (lambda rm, rms: sq.pack_mxfp4(rm, rms, K), ("rm", "rms")),
    "pack_nvfp4": (lambda rm, nrms: sq.pack_nvfp4(rm, nrms, K, 1.0), ("rm", "nrms")),
    "unpack": (lambda mx: sq.unpack_stage_major(mx.codes, mx.scales, K), ("mx",)),
    "linear_mxfp4": (lambda mx, w, y: sq.linear_mxfp4(mx, w, y), ("mx", "w", "y")),
    "linear_silu_mxfp4": (lambda mx, gu: sq.linear_silu_mxfp4(mx, gu), ("mx", "gu")),
    "linear_grouped_mxfp4": (lambda mx, we, seg, rows: sq.linear_grouped_mxfp4(mx, we, seg, rows),
                             ("mx", "we", "seg", "rows")),
    "linear_grouped_silu_mxfp4": (lambda mx, gue, seg, rows: sq.linear_grouped_silu_mxfp4(mx, gue, seg, rows),
                                  ("mx", "gue", "seg", "rows")),
    "moe_route": (lambda y: sq.moe_route(y, 2), ("y",)),
}


def pick(names, index, other=None, at=-1):
    """The named arguments on GPU `index`, the one at `at` on GPU `other`."""
    here, there = tensors(index), tensors(index if other is None else other)
    out = []
    for i, name in enumerate(names):
        name, _, field = name.partition(".")
        t = (there if i == at else here)[name]
        out.append(getattr(t, field) if field else t)
    return out


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("workspace", [0, 4096])
def test_runs_on_the_device_of_its_tensors(monkeypatch, name, workspace):
    calls = record(monkeypatch, sq, workspace)
    f, names = CALLS[name]
    for index in (0, 1, 3):
        del calls[:]
        f(*pick(names, index))
        assert len(calls) == 1
        entry, args, device = calls[0]
        assert device == index, f"{entry} was called with GPU {device} current, its tensors lie on GPU {index}"
        assert args[-1] == 1000 + index  # that device's stream


@pytest.mark.parametrize("name", sorted(n for n, (_, names) in CALLS.items() if len(names) > 1))
def test_refuses_tensors_of_two_devices(monkeypatch, name):
    calls = record(monkeypatch, sq)
    f, names = CALLS[name]
    for at in range(len(names)):
        with pytest.raises(ValueError, match="all tensors must be on"):
            f(*pick(names, 0, 1, at))
    assert not calls


@pytest.mark.parametrize("name,arg,fields", [("linear", 0, ("bb_scales", "res_codes", "res_scales")),
                                             ("linear", 1, ("scales",)), ("linear_mxfp4", 0, ("scales",)),
                                             ("prepare", 2, ("bb_scales", "res_codes", "res_scales", "mask")),
                                             ("quantize", 1, ("codes", "scales")),
                                             ("linear_nvfp4", 1, ("scales",)), ("unpack", 0, ("scales",))])
def test_refuses_parts_on_another_device(monkeypatch, name, arg, fields):
    """The codes and scales of one operand on two devices."""
    calls = record(monkeypatch, sq)
    f, names = CALLS[name]
    for field in fields:
        args, other = pick(names, 0), pick(names, 1)
        args[arg] = args[arg]._replace(**{field: getattr(other[arg], field)})
        with pytest.raises(ValueError, match="all tensors must be on"):
            f(*args)
    assert not calls
