"""What the binding of the expert relayouts allocates and refuses before any
kernel is launched.  No GPU: allocations and library calls are recorded."""
import pytest
import torch

import sequence_head_relayout_gb300 as vf

pytestmark = pytest.mark.usefixtures("lib_built")


class Recorder:
    """Stands in for torch.empty and for the launching library calls; host
    tensors pass for pinned ones."""

    def __init__(self, monkeypatch):
        self.made, self.calls = [], []
        empty = torch.empty

        def record(shape, dtype=None, device=None, pin_memory=False):
            self.made.append((tuple(shape), torch.device(device or "cpu").type, pin_memory))
            return empty(shape, dtype=dtype)

        monkeypatch.setattr(vf.torch, "empty", record)
        monkeypatch.setattr(vf, "_gpu_addressable", lambda t, what: None)
        monkeypatch.setattr(vf, "_stream", lambda stream, device: None)
        monkeypatch.setattr(vf, "_call", lambda fn, *args: self.calls.append(fn))


def test_plan_workspace_is_device_memory(monkeypatch):
    """The workspace is dropped when the call returns, while the kernels still use
    it: only the device allocator orders its next use behind them.  (Pinned host
    memory is free for anyone the moment the tensor goes.)"""
    seen = Recorder(monkeypatch)
    T, K, E = 10000, 2, 8
    plan = vf.expert_plan(torch.zeros(T, K, dtype=torch.int64), E)
    words = vf.lib().vf_expert_workspace(T, K, E) // 4
    assert words > 0 and seen.calls == ["vf_expert_plan"]
    outs = [tuple(t.shape) for t in plan[:4]]
    assert [m[0] for m in seen.made] == outs + [(words,)]
    assert all(m[1:] == ("cpu", True) for m in seen.made[:4])      # beside the indices
    assert seen.made[4][1:] == ("cuda", False)
