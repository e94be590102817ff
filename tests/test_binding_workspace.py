"""The workspace of a split-K call belongs to that call: the binding keeps no
reference to it, so that no later call, and no later graph, writes memory that
an earlier graph still uses (CPU: the library calls are recorded, not made)."""

import gc
import weakref

import pytest
import torch

import activation_sparsity_fp4_amd as sq
from host_stub import record
from test_binding_devices import CALLS, pick

SPLIT = ["linear", "linear_silu_prepare", "linear_mxfp4", "linear_silu_mxfp4"]


@pytest.mark.parametrize("name", SPLIT)
def test_no_workspace_outlives_its_call(monkeypatch, name):
    calls = record(monkeypatch, sq, workspace_bytes=3 << 20)
    made = []
    empty = torch.empty

    def noted(*size, **kw):
        t = empty(*size, **kw)
        made.append((t.numel(), t.data_ptr(), weakref.ref(t)))
        return t

    monkeypatch.setattr(torch, "empty", noted)
    f, names = CALLS[name]
    held = f(*pick(names, 0))
    del held
    gc.collect()
    entry, args, _ = calls[0]
    # the last arguments: workspace, its bytes, stream
    work, nbytes = args[-3], args[-2]
    assert nbytes >= 3 << 20 and work in [p for n, p, _ in made if n >= 3 << 20], entry
    assert all(ref() is None for _, _, ref in made), f"{entry}: a tensor of the call is still held"
