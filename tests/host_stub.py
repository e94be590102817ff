"""Tensors that stand on the CPU and report a GPU, to follow what the binding
does with devices, streams and workspaces where no GPU is at hand. Nothing is
launched: the library calls of `record` only note how they were made."""

import contextlib

import torch


class OnGpu(torch.Tensor):
    """A CPU tensor that reports to lie on GPU `index`."""

    index = 0

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index

    def contiguous(self):
        return self if self.is_contiguous() else on_gpu(self.as_subclass(torch.Tensor).contiguous(), self.index)

    def __getitem__(self, item):
        return on_gpu(self.as_subclass(torch.Tensor)[item], self.index)


def on_gpu(t, index=0):
    t = t.as_subclass(OnGpu)
    t.index = index
    return t


class Calls(list):
    """(name, arguments, current device) of each library call that enqueues work."""


def record(monkeypatch, sq, workspace_bytes=0):
    """Let the binding run on OnGpu tensors with GPU 0 current; returns the list its calls are noted in."""
    calls = Calls()
    current = [0]
    real = torch.empty
    ask = sq._lib.call

    def call(name, *args):
        if name.endswith("_workspace_bytes"):
            return workspace_bytes
        if name.endswith("_meta_row_bytes"):
            return ask(name, *args)
        calls.append((name, args, current[0]))
        return 0

    def empty(*size, dtype=None, device=None):
        device = torch.device(device)
        return on_gpu(real(*size, dtype=dtype), device.index if device.type == "cuda" else 0)

    @contextlib.contextmanager
    def use(device):
        before, current[0] = current[0], torch.device(device).index
        try:
            yield
        finally:
            current[0] = before

    monkeypatch.setattr(sq._lib, "call", call)
    monkeypatch.setattr(sq, "_workspace_bytes", lambda name, *shape: workspace_bytes)
    monkeypatch.setattr(sq, "_stream", lambda device: 1000 + device.index)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "device", use)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    return calls
