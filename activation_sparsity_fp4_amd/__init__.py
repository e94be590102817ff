"""SharQ linear hot path for AMD MI355X (gfx950).

Thin PyTorch-facing wrappers over the C ABI in ``include/sharq.h``: they check
tensor dtypes/devices, allocate outputs with ``torch.empty`` and pass raw device
pointers and the current HIP stream. All arithmetic runs in libsharq.so.

    prep = prepare(x, gamma=None, n=2, m=4)        # x: bf16 [T, K] on the GPU
    wq = quantize_mxfp4(w)                         # w: bf16 [O, K]
    y = linear(prep, wq)                           # fp32 [T, O]

The plain MXFP4 path (one operand, no decomposition) and expert routing:

    y = linear_mxfp4(quantize_mxfp4(x), wq)        # fp32 or bf16 [T, O]
    r = moe_route(logits, k)                       # experts, weights, dispatch plan
"""

from __future__ import annotations

import functools
from typing import NamedTuple, Optional

from . import _lib
from ._lib import SCRATCHFREE_MAX_BYTES, SharqError, status_string  # noqa: F401

__all__ = [
    "Prepared",
    "MXFP4",
    "prepare",
    "quantize_mxfp4",
    "linear",
    "linear_scratchfree",
    "linear_grouped",
    "linear_silu_prepare",
    "linear_silu_prepare_into",
    "linear_grouped_silu_prepare",
    "CompactBackbone",
    "compress_backbone",
    "expand_backbone",
    "moe_combine",
    "silu_mul",
    "NVPrepared",
    "NVFP4",
    "prepare_nvfp4",
    "quantize_nvfp4",
    "linear_nvfp4",
    "pack_mxfp4",
    "pack_nvfp4",
    "unpack_stage_major",
    "linear_mxfp4",
    "linear_silu_mxfp4",
    "linear_grouped_mxfp4",
    "linear_grouped_silu_mxfp4",
    "Routing",
    "moe_route",
    "SharqError",
    "status_string",
]


class Prepared(NamedTuple):
    """Outputs of the prepare operator (uint8 device tensors) and K.

    Codes and scales are stage-major with G = ceil(K/128) stages of 128 K
    entries: the 16 code bytes of block b = k // 32 of row t sit at
    codes[b // 4, t, 16 * (b % 4):][:16] and its scale byte at
    scales[b // 4, t, b % 4]; blocks past K // 32 are zero."""
    bb_codes: "object"    # [G, T, 64]
    bb_scales: "object"   # [G, T, 4]
    res_codes: "object"   # [G, T, 64]
    res_scales: "object"  # [G, T, 4]
    mask: "object"        # [T, K/8] (row-major bitmap) or None
    K: int
    rms_scale: "object" = None  # fp32 [T] per-row 1/rms when the RMSNorm was absorbed


class MXFP4(NamedTuple):
    """A block-scaled FP4 tensor, stage-major: codes [G, R, 64] and scales
    [G, R, 4]; for expert weights codes [E, G, O, 64] and scales [E, G, O, 4]."""
    codes: "object"
    scales: "object"
    K: int


def stages(K: int) -> int:
    """Number of 128-entry K stages (the leading dimension of a scale tensor)."""
    return (K + 127) // 128


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:  # an import statement on every call would cost what a check does
        import torch
        _torch_module = torch
    return _torch_module


def _stream(device) -> int:
    """The device's current stream (without making a torch.cuda.Stream of it, which takes 2 us a call)."""
    return _torch()._C._cuda_getCurrentRawStream(device.index)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _ld(t):
    """Leading dimension of a [rows, columns] tensor; a single row has none, whatever stride it reports."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _need(t, dtype, name, ndim=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def _same_device(first, *others):
    index = first.get_device()  # -1 off the GPU; cheaper than a torch.device
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on {first.device}, got one on {t.device}")


def _parts(prep):
    """The tensors of a Prepared or NVPrepared that an entry point reads or writes."""
    return prep.bb_codes, prep.bb_scales, prep.res_codes, prep.res_scales, prep.mask


def _run(name, device, *args):
    """Enqueue an entry point on the device's current stream and raise on a bad status."""
    torch = _torch()
    if device.index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            st = _lib.call(name, *args, _stream(device))
    else:
        st = _lib.call(name, *args, _stream(device))
    if st:
        _lib.check(name, st)


def _check_stage_major(codes, scales, R, K, name):
    G = stages(K)
    if tuple(codes.shape) != (G, R, 64) or tuple(scales.shape) != (G, R, 4):
        raise ValueError(f"{name}: expected stage-major codes [{G}, {R}, 64] and scales [{G}, {R}, 4], "
                         f"got {tuple(codes.shape)} and {tuple(scales.shape)}")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name}: codes and scales must be contiguous")


def _check_matrix(t, dtype, rows, cols, name, contiguous=False):
    """A [rows, cols] device tensor of dtype with unit column stride (and
    contiguous rows when the entry point takes no leading dimension): the
    kernels write rows x cols entries through it, so nothing smaller passes."""
    _need(t, dtype, name, 2)
    if tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name}: expected shape ({rows}, {cols}), got {tuple(t.shape)}")
    if t.stride(1) != 1 or (contiguous and not t.is_contiguous()):
        raise ValueError(f"{name} must be {'contiguous' if contiguous else 'contiguous along its rows'}")


def _check_prepared(prep):
    torch = _torch()
    for name in ("bb_codes", "res_codes", "bb_scales", "res_scales"):
        _need(getattr(prep, name), torch.uint8, name, 3)
    T = prep.bb_codes.shape[1]
    _check_stage_major(prep.bb_codes, prep.bb_scales, T, prep.K, "backbone")
    _check_stage_major(prep.res_codes, prep.res_scales, T, prep.K, "residual")
    if prep.mask is not None:
        _check_matrix(prep.mask, torch.uint8, T, prep.K // 8, "mask", contiguous=True)


def prepare(x, gamma=None, n: int = 2, m: int = 4, with_mask: bool = True, out: Optional[Prepared] = None,
            rms_eps: Optional[float] = None) -> Prepared:
    """Fused prepare: N:M mask, MXFP4 backbone, residual against it, MXFP4 residual.
    With rms_eps the whole RMSNorm (per-row 1/rms, then gamma) is absorbed
    first; the per-row scales are returned in ``rms_scale``."""
    torch = _torch()
    _need(x, torch.bfloat16, "x", 2)
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous along K")
    T, K = x.shape
    if gamma is not None:
        _need(gamma, torch.bfloat16, "gamma", 1)
        if gamma.numel() != K:  # the kernels read K entries of gamma
            raise ValueError(f"gamma must hold K = {K} entries, got {gamma.numel()}")
        gamma = gamma.contiguous()
    if out is None:
        kw = dict(dtype=torch.uint8, device=x.device)
        G = stages(K)
        out = Prepared(torch.empty((G, T, 64), **kw), torch.empty((G, T, 4), **kw),
                       torch.empty((G, T, 64), **kw), torch.empty((G, T, 4), **kw),
                       torch.empty((T, K // 8), **kw) if with_mask else None, K,
                       torch.empty((T,), dtype=torch.float32, device=x.device) if rms_eps is not None else None)
    else:
        if out.K != K:
            raise ValueError("out was allocated for another K")
        _check_prepared(out)
        if out.bb_codes.shape[1] != T:
            raise ValueError("out was allocated for another number of rows")
    if rms_eps is not None:
        if out.rms_scale is None:
            raise ValueError("out has no rms_scale buffer")
        _need(out.rms_scale, torch.float32, "rms_scale", 1)
        if out.rms_scale.numel() != T or not out.rms_scale.is_contiguous():
            raise ValueError("rms_scale must be a contiguous fp32 [T] tensor")
        _same_device(x, gamma, *_parts(out), out.rms_scale)
        _run("sharq_prepare_rms", x.device, x.data_ptr(), T, K, _ld(x), _ptr(gamma), float(rms_eps), n, m,
             out.rms_scale.data_ptr(), out.bb_codes.data_ptr(), out.bb_scales.data_ptr(),
             out.res_codes.data_ptr(), out.res_scales.data_ptr(), _ptr(out.mask))
        return out
    _same_device(x, gamma, *_parts(out))
    _run("sharq_prepare", x.device, x.data_ptr(), T, K, _ld(x), _ptr(gamma), n, m,
         out.bb_codes.data_ptr(), out.bb_scales.data_ptr(), out.res_codes.data_ptr(),
         out.res_scales.data_ptr(), _ptr(out.mask))
    return out


def quantize_mxfp4(x, out: Optional[MXFP4] = None, gamma=None, rms_eps: Optional[float] = None) -> MXFP4:
    """Plain MXFP4 along the last axis of a bf16 [R, K] tensor (e.g. a weight
    [O, K]), or of a stack of expert weights [E, O, K] (one call per expert,
    so each expert owns a contiguous [G, O, 4] scale block). With rms_eps the
    rows of a [R, K] tensor are RMS-normed first (per-row 1/rms, then gamma
    when given), as prepare(rms_eps=...) norms them."""
    torch = _torch()
    if gamma is not None and rms_eps is None:
        raise ValueError("gamma is the weight of the norm: it needs rms_eps")
    if x.dim() == 3:
        if rms_eps is not None:
            raise ValueError("the norm is for [R, K] activations")
        E, R, K = x.shape
        if out is None:
            out = MXFP4(torch.empty((E, stages(K), R, 64), dtype=torch.uint8, device=x.device),
                        torch.empty((E, stages(K), R, 4), dtype=torch.uint8, device=x.device), K)
        elif out.K != K:
            raise ValueError("out was allocated for another K")
        _need(out.codes, torch.uint8, "out.codes", 4)
        _need(out.scales, torch.uint8, "out.scales", 4)
        if out.codes.shape[0] != E or out.scales.shape[0] != E:
            raise ValueError(f"out must hold {E} experts")
        for e in range(E):
            scales = out.scales[e]
            # the library wants a scale block on a 16-byte boundary; in a stack of odd sizes it may lie off one
            block = torch.empty_like(scales) if scales.data_ptr() % 16 else scales
            quantize_mxfp4(x[e], MXFP4(out.codes[e], block, K))
            if block is not scales:
                scales.copy_(block)
        return out
    _need(x, torch.bfloat16, "x", 2)
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous along K")
    R, K = x.shape
    if out is None:
        out = MXFP4(torch.empty((stages(K), R, 64), dtype=torch.uint8, device=x.device),
                    torch.empty((stages(K), R, 4), dtype=torch.uint8, device=x.device), K)
    elif out.K != K:
        raise ValueError("out was allocated for another K")
    _need(out.codes, torch.uint8, "out.codes", 3)
    _need(out.scales, torch.uint8, "out.scales", 3)
    _check_stage_major(out.codes, out.scales, R, K, "out")
    if rms_eps is not None:
        if gamma is not None:
            _need(gamma, torch.bfloat16, "gamma", 1)
            if gamma.numel() != K:  # the kernels read K entries of gamma
                raise ValueError(f"gamma must hold K = {K} entries, got {gamma.numel()}")
            gamma = gamma.contiguous()
        _same_device(x, gamma, out.codes, out.scales)
        _run("sharq_quantize_mxfp4_rms", x.device, x.data_ptr(), R, K, _ld(x), _ptr(gamma),
             float(rms_eps), 0, out.codes.data_ptr(), out.scales.data_ptr())
        return out
    _same_device(x, out.codes, out.scales)
    _run("sharq_quantize_mxfp4", x.device, x.data_ptr(), R, K, _ld(x), out.codes.data_ptr(),
         out.scales.data_ptr())
    return out


def _scratch(device, nbytes):
    """Workspace of one call, from the allocator that orders it with the
    stream's work (in a graph, from the graph's own memory); None for 0."""
    torch = _torch()
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 0 else None


def linear(prep: Prepared, w: MXFP4, out=None, split_k: bool = True):
    """Two-path FP4 GEMM: Y = deq(backbone) W^T + deq(residual) W^T, fp32 [T, O].
    With split_k, K is split over a workspace (sharq_linear_ws) where
    the library's plan expects it to be faster (too few output tiles to fill
    the GPU, K long enough); the result is deterministic."""
    torch = _torch()
    _check_prepared(prep)
    _need(w.codes, torch.uint8, "w.codes", 3)
    _need(w.scales, torch.uint8, "w.scales", 3)
    T, K = prep.bb_codes.shape[1], prep.K
    O = w.codes.shape[1]
    if w.K != K:
        raise ValueError("weight K does not match the activation K")
    _check_stage_major(w.codes, w.scales, O, K, "w")
    if out is None:
        out = torch.empty((T, O), dtype=torch.float32, device=prep.bb_codes.device)
    _check_matrix(out, torch.float32, T, O, "out")
    _same_device(*_parts(prep), w.codes, w.scales, out)
    nbytes = _lib.call("sharq_linear_workspace_bytes", T, O, K) if split_k else 0
    if nbytes > 0:
        ws = _scratch(out.device, nbytes)
        _run("sharq_linear_ws", out.device, prep.bb_codes.data_ptr(), prep.bb_scales.data_ptr(),
             prep.res_codes.data_ptr(), prep.res_scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(),
             T, O, K, out.data_ptr(), _ld(out), ws.data_ptr(), ws.numel())
        return out
    _run("sharq_linear", out.device, prep.bb_codes.data_ptr(), prep.bb_scales.data_ptr(), prep.res_codes.data_ptr(),
         prep.res_scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(), T, O, K,
         out.data_ptr(), _ld(out))
    return out


def linear_scratchfree(prep: Prepared, w: MXFP4, out):
    """linear() with any K split's partials in the library's static scratch
    array instead of a workspace: nothing is allocated, so `out` (fp32
    [T, O]) is required. Raises SharqError (SHARQ_ESCRATCH) when the split
    plan needs more than SCRATCHFREE_MAX_BYTES. Calls that overlap in time on
    one GPU share the array and race."""
    torch = _torch()
    _check_prepared(prep)
    _need(w.codes, torch.uint8, "w.codes", 3)
    _need(w.scales, torch.uint8, "w.scales", 3)
    T, K = prep.bb_codes.shape[1], prep.K
    O = w.codes.shape[1]
    if w.K != K:
        raise ValueError("weight K does not match the activation K")
    _check_stage_major(w.codes, w.scales, O, K, "w")
    _check_matrix(out, torch.float32, T, O, "out")
    _same_device(*_parts(prep), w.codes, w.scales, out)
    _run("sharq_linear_scratchfree", out.device, prep.bb_codes.data_ptr(), prep.bb_scales.data_ptr(),
         prep.res_codes.data_ptr(), prep.res_scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(),
         T, O, K, out.data_ptr(), _ld(out))
    return out


def linear_grouped(prep: Prepared, w: MXFP4, seg_offsets, a_rows=None, out=None):
    """Grouped two-path GEMM over expert segments. w.codes is [E, G, O, 64];
    seg_offsets int32 [E+1]; a_rows int32 [P] (source row of each sorted pair) or None."""
    torch = _torch()
    _check_prepared(prep)
    E, _, O, _ = _check_mx(w, "w", 4)
    K = prep.K
    if w.K != K:
        raise ValueError("weight K does not match the activation K")
    P = _check_plan(seg_offsets, E, a_rows, prep.bb_codes.shape[1])
    if out is None:
        out = torch.empty((P, O), dtype=torch.float32, device=w.codes.device)
    _check_matrix(out, torch.float32, P, O, "out", contiguous=True)
    _same_device(*_parts(prep), w.codes, w.scales, seg_offsets, a_rows, out)
    _run("sharq_linear_grouped", out.device, prep.bb_codes.data_ptr(), prep.bb_scales.data_ptr(),
         prep.res_codes.data_ptr(), prep.res_scales.data_ptr(), prep.bb_codes.shape[1], _ptr(a_rows),
         seg_offsets.data_ptr(), E, w.codes.data_ptr(), w.scales.data_ptr(), P, O, K, out.data_ptr())
    return out


def linear_silu_prepare(prep: Prepared, w_gu: MXFP4, n: int = 2, m: int = 4, with_h: bool = False,
                        with_prepared: bool = True, with_mask: bool = True, split_k: bool = True):
    """Fused gate|up projection: Y = two-path GEMM of prep against w_gu (rows:
    I gate rows, then I up rows), h = bf16(silu(Y[:, :I]) * Y[:, I:]), then
    prepare(h, n, m). Returns (Prepared of h or None, h or None); the results
    equal linear(split_k) -> silu_mul -> prepare bit for bit. With split_k,
    problems with too few tiles to fill the GPU split K as linear does
    (sharq_linear_silu_prepare_ws)."""
    torch = _torch()
    _check_prepared(prep)
    _need(w_gu.codes, torch.uint8, "w_gu.codes", 3)
    _need(w_gu.scales, torch.uint8, "w_gu.scales", 3)
    T, K = prep.bb_codes.shape[1], prep.K
    O = w_gu.codes.shape[1]
    if w_gu.K != K or O % 2:
        raise ValueError("w_gu must be [2I, K] with the activation's K")
    _check_stage_major(w_gu.codes, w_gu.scales, O, K, "w_gu")
    I = O // 2
    dev = prep.bb_codes.device
    kw = dict(dtype=torch.uint8, device=dev)
    h = torch.empty((T, I), dtype=torch.bfloat16, device=dev) if with_h else None
    hp = None
    if with_prepared:
        G = stages(I)
        hp = Prepared(torch.empty((G, T, 64), **kw), torch.empty((G, T, 4), **kw),
                      torch.empty((G, T, 64), **kw), torch.empty((G, T, 4), **kw),
                      torch.empty((T, I // 8), **kw) if with_mask else None, I)
    _fused_call(prep, w_gu, T, I, K, n, m, h, hp, split_k)
    return hp, h


def linear_silu_prepare_into(prep: Prepared, w_gu: MXFP4, out: Prepared, n: int = 2, m: int = 4,
                             split_k: bool = True) -> Prepared:
    """linear_silu_prepare writing prepare(h) into preallocated `out` (no h)."""
    _check_prepared(prep)
    _check_prepared(out)
    _check_mx(w_gu, "w_gu")
    T, K, I = prep.bb_codes.shape[1], prep.K, out.K
    if w_gu.K != K or tuple(w_gu.codes.shape) != (stages(K), 2 * I, 64) or out.bb_codes.shape[1] != T:
        raise ValueError("shapes of prep, w_gu and out do not match")
    _fused_call(prep, w_gu, T, I, K, n, m, None, out, split_k)
    return out


def _fused_call(prep, w_gu, T, I, K, n, m, h, hp, split_k):
    dev = prep.bb_codes.device
    args = (prep.bb_codes.data_ptr(), prep.bb_scales.data_ptr(), prep.res_codes.data_ptr(),
            prep.res_scales.data_ptr(), w_gu.codes.data_ptr(), w_gu.scales.data_ptr(), T, I, K, n, m, _ptr(h),
            _ptr(hp and hp.bb_codes), _ptr(hp and hp.bb_scales), _ptr(hp and hp.res_codes),
            _ptr(hp and hp.res_scales), _ptr(hp and hp.mask))
    _same_device(*_parts(prep), w_gu.codes, w_gu.scales, h, *(_parts(hp) if hp else ()))
    nbytes = _lib.call("sharq_linear_silu_prepare_workspace_bytes", T, I, K) if split_k else 0
    if nbytes > 0:
        ws = _scratch(dev, nbytes)
        _run("sharq_linear_silu_prepare_ws", dev, *args, ws.data_ptr(), ws.numel())
        return
    _run("sharq_linear_silu_prepare", dev, *args)


def linear_grouped_silu_prepare(prep: Prepared, w_gu: MXFP4, seg_offsets, a_rows=None, n: int = 2, m: int = 4,
                                with_h: bool = False, with_prepared: bool = True, with_mask: bool = True,
                                out: Prepared = None):
    """Grouped fused gate|up projection: linear_grouped against each expert's
    w_gu ([E, G, 2I, 64]: I gate rows, then I up rows), then silu_mul and
    prepare(h, n, m), in one kernel. Rows are the sorted pairs. Returns
    (Prepared of h or None, h or None), bit-identical to the three-step chain.
    `out` (a Prepared of [G_I, P, ...]) receives prepare(h) when given."""
    torch = _torch()
    _check_prepared(prep)
    E, _, O, _ = _check_mx(w_gu, "w_gu", 4)
    K = prep.K
    if w_gu.K != K or O % 2:
        raise ValueError("w_gu must be [E, 2I, K] with the activation's K")
    P = _check_plan(seg_offsets, E, a_rows, prep.bb_codes.shape[1])
    I = O // 2
    dev = prep.bb_codes.device
    kw = dict(dtype=torch.uint8, device=dev)
    h = torch.empty((P, I), dtype=torch.bfloat16, device=dev) if with_h else None
    hp = None
    if out is not None:
        _check_prepared(out)
        if out.K != I or out.bb_codes.shape[1] != P:
            raise ValueError("out must be a Prepared of [P, I]")
        hp = out
    elif with_prepared:
        G = stages(I)
        hp = Prepared(torch.empty((G, P, 64), **kw), torch.empty((G, P, 4), **kw),
                      torch.empty((G, P, 64), **kw), torch.empty((G, P, 4), **kw),
                      torch.empty((P, I // 8), **kw) if with_mask else None, I)
    _same_device(*_parts(prep), w_gu.codes, w_gu.scales, seg_offsets, a_rows, h, *(_parts(hp) if hp else ()))
    _run("sharq_linear_grouped_silu_prepare", dev, prep.bb_codes.data_ptr(), prep.bb_scales.data_ptr(),
         prep.res_codes.data_ptr(), prep.res_scales.data_ptr(), prep.bb_codes.shape[1], _ptr(a_rows),
         seg_offsets.data_ptr(), E, w_gu.codes.data_ptr(), w_gu.scales.data_ptr(), P, I, K, n, m, _ptr(h),
         _ptr(hp and hp.bb_codes), _ptr(hp and hp.bb_scales), _ptr(hp and hp.res_codes),
         _ptr(hp and hp.res_scales), _ptr(hp and hp.mask))
    return hp, h


class CompactBackbone(NamedTuple):
    """A compressed backbone: kept codes [T, K/4] (row-major), per-group rank
    fields [T, meta_row_bytes], the n:m pattern and K. The backbone's block
    scales stay in the Prepared it came from."""
    codes: "object"
    meta: "object"
    n: int
    m: int
    K: int


def compress_backbone(prep: Prepared, n: int = 2, m: int = 4, out: CompactBackbone = None) -> CompactBackbone:
    """The compressed form of prep's backbone (needs prep.mask)."""
    torch = _torch()
    _check_prepared(prep)
    if prep.mask is None:
        raise ValueError("compressing the backbone needs the mask")
    T, K = prep.bb_codes.shape[1], prep.K
    row = _lib.call("sharq_backbone_meta_row_bytes", K, n, m)
    _lib.check("sharq_backbone_meta_row_bytes", int(min(row, 0)))
    if out is None:
        dev = prep.bb_codes.device
        out = CompactBackbone(torch.empty((T, K // 4), dtype=torch.uint8, device=dev),
                              torch.empty((T, row), dtype=torch.uint8, device=dev), n, m, K)
    if (out.n, out.m, out.K) != (n, m, K):
        raise ValueError("out does not match the backbone")
    _check_matrix(out.codes, torch.uint8, T, K // 4, "out.codes", contiguous=True)
    _check_matrix(out.meta, torch.uint8, T, row, "out.meta", contiguous=True)
    _same_device(prep.bb_codes, prep.mask, out.codes, out.meta)
    _run("sharq_compress_backbone", prep.bb_codes.device, prep.bb_codes.data_ptr(), prep.mask.data_ptr(), T, K, n, m,
         out.codes.data_ptr(), out.meta.data_ptr())
    return out


def expand_backbone(cb: CompactBackbone, bb_codes=None, mask=None, with_mask: bool = True):
    """Dense stage-major backbone codes [G, T, 64] (and the mask [T, K/8])
    from a CompactBackbone. Returns (bb_codes, mask or None)."""
    torch = _torch()
    _need(cb.codes, torch.uint8, "codes", 2)
    _need(cb.meta, torch.uint8, "meta", 2)
    T, K = cb.codes.shape[0], cb.K
    row = _lib.call("sharq_backbone_meta_row_bytes", K, cb.n, cb.m)
    _lib.check("sharq_backbone_meta_row_bytes", int(min(row, 0)))
    _check_matrix(cb.codes, torch.uint8, T, K // 4, "codes", contiguous=True)
    _check_matrix(cb.meta, torch.uint8, T, row, "meta", contiguous=True)
    dev = cb.codes.device
    if bb_codes is None:
        bb_codes = torch.empty((stages(K), T, 64), dtype=torch.uint8, device=dev)
    if with_mask and mask is None:
        mask = torch.empty((T, K // 8), dtype=torch.uint8, device=dev)
    if not with_mask:
        mask = None
    _need(bb_codes, torch.uint8, "bb_codes", 3)
    if tuple(bb_codes.shape) != (stages(K), T, 64) or not bb_codes.is_contiguous():
        raise ValueError(f"bb_codes must be a contiguous [{stages(K)}, {T}, 64] tensor")
    if mask is not None:
        _check_matrix(mask, torch.uint8, T, K // 8, "mask", contiguous=True)
    _same_device(cb.codes, cb.meta, bb_codes, mask)
    _run("sharq_expand_backbone", dev, cb.codes.data_ptr(), cb.meta.data_ptr(), T, K, cb.n, cb.m,
         bb_codes.data_ptr(), _ptr(mask))
    return bb_codes, mask


def moe_combine(y, pair_index, weights, out=None, bf16: bool = False):
    """out[t] = sum_j weights[t, j] * y[pair_index[t, j]] (slots with -1 skipped),
    fp32 accumulation in slot order; fp32 [T, H] or, with bf16, bf16 [T, H].
    y is fp32 or bf16."""
    torch = _torch()
    rows_bf16 = isinstance(y, torch.Tensor) and y.dtype == torch.bfloat16
    _need(y, torch.bfloat16 if rows_bf16 else torch.float32, "y", 2)
    _need(pair_index, torch.int32, "pair_index", 2)
    _need(weights, torch.float32, "weights", 2)
    if not (y.is_contiguous() and pair_index.is_contiguous() and weights.is_contiguous()):
        raise ValueError("y, pair_index and weights must be contiguous")
    if pair_index.shape != weights.shape:
        raise ValueError("pair_index and weights must have the same [T, k] shape")
    T, k = pair_index.shape
    P, H = y.shape
    dt = torch.bfloat16 if bf16 else torch.float32
    if out is None:
        out = torch.empty((T, H), dtype=dt, device=y.device)
    _check_matrix(out, dt, T, H, "out", contiguous=True)
    _same_device(y, pair_index, weights, out)
    if rows_bf16:
        _run("sharq_moe_combine_bf16", y.device, y.data_ptr(), P, H, pair_index.data_ptr(), weights.data_ptr(), T, k,
             0 if bf16 else out.data_ptr(), out.data_ptr() if bf16 else 0)
        return out
    _run("sharq_moe_combine", y.device, y.data_ptr(), P, H, pair_index.data_ptr(), weights.data_ptr(), T, k,
         0 if bf16 else out.data_ptr(), out.data_ptr() if bf16 else 0)
    return out


def silu_mul(gu, out=None):
    """h = bf16(silu(gu[:, :I]) * gu[:, I:]) for a fused gate|up output gu fp32 [T, 2I]."""
    torch = _torch()
    _need(gu, torch.float32, "gu", 2)
    if not gu.is_contiguous():
        raise ValueError("gu must be contiguous")
    T, I2 = gu.shape
    I = I2 // 2
    if out is None:
        out = torch.empty((T, I), dtype=torch.bfloat16, device=gu.device)
    _check_matrix(out, torch.bfloat16, T, I, "out", contiguous=True)
    _same_device(gu, out)
    _run("sharq_silu_mul", gu.device, gu.data_ptr(), T, I, out.data_ptr())
    return out


# ---------------------------------------------------------------------------
# NVFP4: 16-entry E2M1 blocks with E4M3 block scales and an fp32 tensor scale
# ---------------------------------------------------------------------------


class NVPrepared(NamedTuple):
    """Outputs of the NVFP4 prepare: codes [G, T, 64] as in Prepared, E4M3
    block scales [G, T, 8] (byte j of a row's stage g covers K entries
    128 g + 16 j .. + 15), the mask, K and the activation's tensor scale."""
    bb_codes: "object"
    bb_scales: "object"
    res_codes: "object"
    res_scales: "object"
    mask: "object"
    K: int
    tensor_scale: float


class NVFP4(NamedTuple):
    """An NVFP4 tensor, stage-major: codes [G, R, 64], E4M3 scales [G, R, 8]."""
    codes: "object"
    scales: "object"
    K: int
    tensor_scale: float


def _check_nv(codes, scales, R, K, name):
    torch = _torch()
    _need(codes, torch.uint8, name + ".codes", 3)
    _need(scales, torch.uint8, name + ".scales", 3)
    G = stages(K)
    if tuple(codes.shape) != (G, R, 64) or tuple(scales.shape) != (G, R, 8):
        raise ValueError(f"{name}: expected codes [{G}, {R}, 64] and scales [{G}, {R}, 8], "
                         f"got {tuple(codes.shape)} and {tuple(scales.shape)}")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name}: codes and scales must be contiguous")


def prepare_nvfp4(x, tensor_scale: float, gamma=None, n: int = 2, m: int = 4, with_mask: bool = True,
                  out: Optional[NVPrepared] = None) -> NVPrepared:
    """The prepare operator with NVFP4 codes; tensor_scale is the activation's
    fp32 tensor scale (shared by backbone and residual)."""
    torch = _torch()
    _need(x, torch.bfloat16, "x", 2)
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous along K")
    T, K = x.shape
    if gamma is not None:
        _need(gamma, torch.bfloat16, "gamma", 1)
        if gamma.numel() != K:  # the kernels read K entries of gamma
            raise ValueError(f"gamma must hold K = {K} entries, got {gamma.numel()}")
        gamma = gamma.contiguous()
    if out is None:
        kw = dict(dtype=torch.uint8, device=x.device)
        G = stages(K)
        out = NVPrepared(torch.empty((G, T, 64), **kw), torch.empty((G, T, 8), **kw),
                         torch.empty((G, T, 64), **kw), torch.empty((G, T, 8), **kw),
                         torch.empty((T, K // 8), **kw) if with_mask else None, K, float(tensor_scale))
    else:
        if out.K != K:
            raise ValueError("out was allocated for another K")
        _check_nv(out.bb_codes, out.bb_scales, T, K, "out backbone")
        _check_nv(out.res_codes, out.res_scales, T, K, "out residual")
        if out.mask is not None:
            _check_matrix(out.mask, torch.uint8, T, K // 8, "out.mask", contiguous=True)
        out = out._replace(tensor_scale=float(tensor_scale))
    _same_device(x, gamma, *_parts(out))
    _run("sharq_prepare_nvfp4", x.device, x.data_ptr(), T, K, _ld(x), _ptr(gamma), n, m, float(tensor_scale),
         out.bb_codes.data_ptr(), out.bb_scales.data_ptr(), out.res_codes.data_ptr(),
         out.res_scales.data_ptr(), _ptr(out.mask))
    return out


def quantize_nvfp4(w, tensor_scale: float, out: Optional[NVFP4] = None) -> NVFP4:
    """NVFP4 of a bf16 [O, K] tensor with the given fp32 tensor scale."""
    torch = _torch()
    _need(w, torch.bfloat16, "w", 2)
    if w.stride(1) != 1:
        raise ValueError("w rows must be contiguous along K")
    O, K = w.shape
    if out is None:
        out = NVFP4(torch.empty((stages(K), O, 64), dtype=torch.uint8, device=w.device),
                    torch.empty((stages(K), O, 8), dtype=torch.uint8, device=w.device), K, float(tensor_scale))
    else:
        _check_nv(out.codes, out.scales, O, K, "out")
        out = out._replace(tensor_scale=float(tensor_scale))
    _same_device(w, out.codes, out.scales)
    _run("sharq_quantize_nvfp4", w.device, w.data_ptr(), O, K, _ld(w), float(tensor_scale),
         out.codes.data_ptr(), out.scales.data_ptr())
    return out


def linear_nvfp4(prep: NVPrepared, w: NVFP4, out=None):
    """Two-path GEMM on NVFP4 operands: Y = deq(A_s) W^T + deq(A_r) W^T, fp32 [T, O]."""
    torch = _torch()
    T, K = prep.bb_codes.shape[1], prep.K
    O = w.codes.shape[1]
    _check_nv(prep.bb_codes, prep.bb_scales, T, K, "backbone")
    _check_nv(prep.res_codes, prep.res_scales, T, K, "residual")
    _check_nv(w.codes, w.scales, O, K, "w")
    if w.K != K:
        raise ValueError("weight K does not match the activation K")
    if out is None:
        out = torch.empty((T, O), dtype=torch.float32, device=prep.bb_codes.device)
    _check_matrix(out, torch.float32, T, O, "out")
    _same_device(*_parts(prep), w.codes, w.scales, out)
    _run("sharq_linear_nvfp4", out.device, prep.bb_codes.data_ptr(), prep.bb_scales.data_ptr(),
         prep.res_codes.data_ptr(), prep.res_scales.data_ptr(), float(prep.tensor_scale),
         w.codes.data_ptr(), w.scales.data_ptr(), float(w.tensor_scale), T, O, K, out.data_ptr(),
         _ld(out))
    return out


# ---------------------------------------------------------------------------
# Layout conversion: canonical row-major block-FP4 <-> stage-major
# ---------------------------------------------------------------------------


def _pack(codes_rm, scales_rm, K, block, name):
    torch = _torch()
    _need(codes_rm, torch.uint8, name + " codes", 2)
    _need(scales_rm, torch.uint8, name + " scales", 2)
    R = codes_rm.shape[0]
    _check_matrix(codes_rm, torch.uint8, R, K // 2, name + " codes", contiguous=True)
    _check_matrix(scales_rm, torch.uint8, R, K // block, name + " scales", contiguous=True)
    G = stages(K)
    codes = torch.empty((G, R, 64), dtype=torch.uint8, device=codes_rm.device)
    scales = torch.empty((G, R, 128 // block), dtype=torch.uint8, device=codes_rm.device)
    _same_device(codes_rm, scales_rm)
    _run("sharq_pack_stage_major", codes_rm.device, codes_rm.data_ptr(), scales_rm.data_ptr(), R, K, block,
         codes.data_ptr(), scales.data_ptr())
    return codes, scales


def pack_mxfp4(codes_rm, scales_rm, K: int) -> MXFP4:
    """An MXFP4 tensor from the canonical row-major layout (codes [R, K/2],
    E8M0 scale bytes [R, K/32]), e.g. a weight quantised elsewhere."""
    codes, scales = _pack(codes_rm, scales_rm, K, 32, "MXFP4")
    return MXFP4(codes, scales, K)


def pack_nvfp4(codes_rm, scales_rm, K: int, tensor_scale: float) -> NVFP4:
    """An NVFP4 tensor from the canonical row-major layout (codes [R, K/2],
    E4M3 scale bytes [R, K/16]) and its fp32 tensor scale."""
    codes, scales = _pack(codes_rm, scales_rm, K, 16, "NVFP4")
    return NVFP4(codes, scales, K, float(tensor_scale))


def unpack_stage_major(codes, scales, K: int):
    """(codes [R, K/2], scales [R, K/block]) in the canonical row-major layout
    from stage-major codes [G, R, 64] and scales [G, R, 128/block] (block 32
    for MXFP4 scales [G, R, 4], 16 for NVFP4 scales [G, R, 8])."""
    torch = _torch()
    _need(codes, torch.uint8, "codes", 3)
    _need(scales, torch.uint8, "scales", 3)
    G, R, _ = codes.shape
    per = scales.shape[2]
    if per not in (4, 8) or tuple(codes.shape) != (stages(K), R, 64) or tuple(scales.shape) != (stages(K), R, per) \
            or not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("expected contiguous stage-major codes [G, R, 64] and scales [G, R, 4 or 8]")
    block = 128 // per
    codes_rm = torch.empty((R, K // 2), dtype=torch.uint8, device=codes.device)
    scales_rm = torch.empty((R, K // block), dtype=torch.uint8, device=codes.device)
    _same_device(codes, scales)
    _run("sharq_unpack_stage_major", codes.device, codes.data_ptr(), scales.data_ptr(), R, K, block,
         codes_rm.data_ptr(), scales_rm.data_ptr())
    return codes_rm, scales_rm


# ---------------------------------------------------------------------------
# Plain MXFP4 path: one activation operand, no decomposition
# ---------------------------------------------------------------------------


def _check_mx(t, name, ndim=3):
    """The shape of an MXFP4 tensor's codes; codes and scales are contiguous, stage-major and fit its K."""
    torch = _torch()
    codes, scales, K = t
    G = stages(K)
    if type(codes) is type(scales) is torch.Tensor:
        shape = codes.shape
        if (len(shape) == ndim and shape[-3] == G and shape[-1] == 64 and scales.shape == (*shape[:-1], 4)
                and codes.dtype is scales.dtype is torch.uint8 and codes.is_cuda and scales.is_cuda
                and codes.is_contiguous() and scales.is_contiguous()):
            return shape
    _need(codes, torch.uint8, name + ".codes", ndim)
    _need(scales, torch.uint8, name + ".scales", ndim)
    shape, sshape = codes.shape, scales.shape
    if shape[-3] != G or shape[-1] != 64 or sshape[:-1] != shape[:-1] or sshape[-1] != 4:
        raise ValueError(f"{name}: expected stage-major codes [.., {G}, R, 64] and scales [.., {G}, R, 4], "
                         f"got {tuple(shape)} and {tuple(sshape)}")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError(f"{name}: codes and scales must be contiguous")
    return shape


def _out_dtype(out, dtype):
    """The type of a product's output and its number in the ABI."""
    torch = _torch()
    if out is not None and dtype is not None and out.dtype != dtype:
        raise TypeError(f"out is {out.dtype}, dtype asks for {dtype}")
    dtype = out.dtype if out is not None else dtype or torch.float32
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"the output is float32 or bfloat16, not {dtype}")
    return dtype, 0 if dtype == torch.float32 else 1


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(name, *shape):
    """The library's answer for a shape (asking it takes a fifth of a small call)."""
    return _lib.call(name, *shape)


def linear_mxfp4(a: MXFP4, w: MXFP4, out=None, dtype=None, split_k: bool = True):
    """One plain MXFP4 product Y = deq(a) deq(w)^T, [T, O] of dtype float32
    (the default) or bfloat16 (the fp32 sum rounded once). With split_k, K is
    split over a workspace where the library expects that to be faster (single
    tokens, few output tiles); the result is deterministic either way."""
    torch = _torch()
    T, O, K = _check_mx(a, "a")[1], _check_mx(w, "w")[1], a.K
    if w.K != K:
        raise ValueError("weight K does not match the activation K")
    dtype, number = _out_dtype(out, dtype)
    dev = a.codes.device
    if out is None:
        out, ldy = torch.empty((T, O), dtype=dtype, device=dev), O
    else:
        _check_matrix(out, dtype, T, O, "out")
        ldy = _ld(out)
    _same_device(a.codes, a.scales, w.codes, w.scales, out)
    ws = _scratch(dev, _workspace_bytes("sharq_linear_mxfp4_workspace_bytes", T, O, K) if split_k else 0)
    _run("sharq_linear_mxfp4", dev, a.codes.data_ptr(), a.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(),
         T, O, K, out.data_ptr(), ldy, number, _ptr(ws), 0 if ws is None else ws.numel())
    return out


def _mx_like(rows, K, device):
    torch = _torch()
    return MXFP4(torch.empty((stages(K), rows, 64), dtype=torch.uint8, device=device),
                 torch.empty((stages(K), rows, 4), dtype=torch.uint8, device=device), K)


def linear_silu_mxfp4(a: MXFP4, w_gu: MXFP4, out: Optional[MXFP4] = None, split_k: bool = True) -> MXFP4:
    """Fused gate|up projection on the plain path: the product with w_gu (I
    gate rows, then I up rows), h = bf16(silu(gate) * up), MXFP4 of h. Equals
    linear_mxfp4(split_k) -> silu_mul -> quantize_mxfp4 bit for bit; neither
    the product nor h passes through memory (but for the fp32 partials of a
    split K)."""
    T, O, K = _check_mx(a, "a")[1], _check_mx(w_gu, "w_gu")[1], a.K
    if w_gu.K != K or O % 2:
        raise ValueError("w_gu must be [2I, K] with the activation's K")
    I = O // 2
    dev = a.codes.device
    if out is None:
        out = _mx_like(T, I, dev)
    else:
        _check_mx(out, "out")
        if out.K != I or out.codes.shape[1] != T:
            raise ValueError(f"out must be an MXFP4 tensor of [{T}, {I}]")
    _same_device(a.codes, a.scales, w_gu.codes, w_gu.scales, out.codes, out.scales)
    ws = _scratch(dev, _workspace_bytes("sharq_linear_silu_mxfp4_workspace_bytes", T, I, K) if split_k else 0)
    _run("sharq_linear_silu_mxfp4", dev, a.codes.data_ptr(), a.scales.data_ptr(), w_gu.codes.data_ptr(),
         w_gu.scales.data_ptr(), T, I, K, out.codes.data_ptr(), out.scales.data_ptr(), _ptr(ws),
         0 if ws is None else ws.numel())
    return out


def _check_plan(seg_offsets, E, a_rows, rows):
    """Output rows of a grouped call over `rows` activation rows: the segments and the gather lie side by side."""
    torch = _torch()
    _need(seg_offsets, torch.int32, "seg_offsets", 1)
    if seg_offsets.numel() != E + 1 or not seg_offsets.is_contiguous():
        raise ValueError("seg_offsets must be a contiguous [E + 1] tensor")
    if a_rows is None:
        return rows
    _need(a_rows, torch.int32, "a_rows", 1)
    if not a_rows.is_contiguous():
        raise ValueError("a_rows must be contiguous")
    return a_rows.numel()


def _check_grouped(a, w, seg_offsets, a_rows, name):
    """(T_src, E, rows of the weight, P) of a grouped call on the plain path."""
    T = _check_mx(a, "a")[1]
    E, _, O, _ = _check_mx(w, name, 4)
    if w.K != a.K:
        raise ValueError("weight K does not match the activation K")
    P = _check_plan(seg_offsets, E, a_rows, T)
    _same_device(a.codes, a.scales, w.codes, w.scales, seg_offsets, a_rows)
    return T, E, O, P


def linear_grouped_mxfp4(a: MXFP4, w: MXFP4, seg_offsets, a_rows=None, out=None, dtype=None):
    """linear_mxfp4 per expert segment: row p of the [P, O] result (float32 or
    bfloat16) is activation row a_rows[p] (row p without a_rows) times the
    weight of the expert e with seg_offsets[e] <= p < seg_offsets[e + 1].
    w.codes is [E, G, O, 64]. Rows behind the last segment are not written."""
    torch = _torch()
    T, E, O, P = _check_grouped(a, w, seg_offsets, a_rows, "w")
    dtype, number = _out_dtype(out, dtype)
    if out is None:
        out = torch.empty((P, O), dtype=dtype, device=a.codes.device)
    else:
        _check_matrix(out, dtype, P, O, "out", contiguous=True)
        _same_device(a.codes, out)
    _run("sharq_linear_grouped_mxfp4", a.codes.device, a.codes.data_ptr(), a.scales.data_ptr(), T, _ptr(a_rows),
         seg_offsets.data_ptr(), E, w.codes.data_ptr(), w.scales.data_ptr(), P, O, a.K, out.data_ptr(), number)
    return out


def linear_grouped_silu_mxfp4(a: MXFP4, w_gu: MXFP4, seg_offsets, a_rows=None,
                              out: Optional[MXFP4] = None) -> MXFP4:
    """linear_silu_mxfp4 per expert segment: MXFP4 of h [P, I] for expert
    weights w_gu.codes [E, G, 2I, 64]. Rows behind the last segment are not
    written."""
    T, E, O, P = _check_grouped(a, w_gu, seg_offsets, a_rows, "w_gu")
    if O % 2:
        raise ValueError("w_gu must be [E, 2I, K]")
    if out is None:
        out = _mx_like(P, O // 2, a.codes.device)
    else:
        _check_mx(out, "out")
        if out.K != O // 2 or out.codes.shape[1] != P:
            raise ValueError(f"out must be an MXFP4 tensor of [{P}, {O // 2}]")
        _same_device(a.codes, out.codes, out.scales)
    _run("sharq_linear_grouped_silu_mxfp4", a.codes.device, a.codes.data_ptr(), a.scales.data_ptr(), T, _ptr(a_rows),
         seg_offsets.data_ptr(), E, w_gu.codes.data_ptr(), w_gu.scales.data_ptr(), P, O // 2, a.K,
         out.codes.data_ptr(), out.scales.data_ptr())
    return out


# ---------------------------------------------------------------------------
# Expert routing
# ---------------------------------------------------------------------------


class Routing(NamedTuple):
    """Where each token goes: the chosen experts and their weights (best
    first), and the pairs (token, expert) sorted by expert, as the grouped
    calls and moe_combine read them."""
    expert: "object"       # i32 [T, k], -1 in an empty slot
    weight: "object"       # fp32 [T, k], 0 in an empty slot
    seg_offsets: "object"  # i32 [E + 1]
    a_rows: "object"       # i32 [T * k], -1 behind the last pair
    pair_index: "object"   # i32 [T, k], -1 in an empty slot


_SCORES = {"softmax": 0, "sigmoid": 1}
_GROUP_SCORES = {"max": 0, "sum2": 1}


def moe_route(logits, k: int, score: str = "softmax", bias=None, groups: int = 1, top_groups: Optional[int] = None,
              group_score: str = "max", renormalize: bool = True, scale: float = 1.0, num_tokens=None) -> Routing:
    """The k experts of each token from router logits [T, E] (float32, bfloat16
    or float16; rows may be strided), their weights and the dispatch plan.

    Experts are ordered by their logit, or with bias (fp32 [E]) by score +
    bias; equal ones go to the lower index, and an expert whose logit is -inf
    or NaN is never chosen (slots that stay empty hold -1 and weight 0). With
    groups > 1 only the top_groups best groups of consecutive experts take
    part, judged by their largest value ("max") or the sum of their two largest
    scores + bias ("sum2"). weight is the score without the bias, divided by
    the sum over the chosen with renormalize, times scale (held in float32, as
    the weights are). Rows from num_tokens (int32 [1] on the device) on are
    padding and choose nothing."""
    torch = _torch()
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    dtype = logits.dtype
    kind = 0 if dtype == torch.float32 else 1 if dtype == torch.bfloat16 else 2 if dtype == torch.float16 else None
    if kind is None:
        raise TypeError(f"logits must be float32, bfloat16 or float16, got {dtype}")
    _need(logits, dtype, "logits", 2)
    T, E = logits.shape
    if T and (logits.stride(1) != 1 and E > 1):
        raise ValueError("logits rows must be contiguous along the experts")
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if group_score not in _GROUP_SCORES:
        raise ValueError(f"group_score must be one of {sorted(_GROUP_SCORES)}, got {group_score!r}")
    if bias is not None:
        _need(bias, torch.float32, "bias", 1)
        if bias.numel() != E or not bias.is_contiguous():
            raise ValueError(f"bias must be a contiguous [{E}] tensor")
    if num_tokens is not None:
        _need(num_tokens, torch.int32, "num_tokens")
        if num_tokens.numel() != 1:
            raise ValueError("num_tokens must hold one value")
    _same_device(logits, bias, num_tokens)
    dev = logits.device
    # one allocation for the four [T, k] arrays (four take longer than a small call's kernel); a_rows first, 16-byte
    # aligned as linear_grouped asks for it
    a_rows, expert, pair_index, weight = torch.empty((4, T, k), dtype=torch.int32, device=dev).unbind(0)
    r = Routing(expert, weight.view(torch.float32), torch.empty(E + 1, dtype=torch.int32, device=dev),
                a_rows.view(-1), pair_index)
    ws = _scratch(dev, _workspace_bytes("sharq_moe_route_workspace_bytes", T, E)) if T > 1 else None
    _run("sharq_moe_route", dev, logits.data_ptr(), kind, T, E, _ld(logits), _ptr(bias), k,
         _SCORES[score], groups, groups if top_groups is None else top_groups, _GROUP_SCORES[group_score],
         int(renormalize), float(scale), _ptr(num_tokens), expert.data_ptr(), weight.data_ptr(),
         r.seg_offsets.data_ptr(), a_rows.data_ptr(), pair_index.data_ptr(), _ptr(ws), 0 if ws is None else ws.numel())
    return r
