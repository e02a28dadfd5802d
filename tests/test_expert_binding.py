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


def _calls(x, packed, w):
    plan = vf.ExpertPlan(*(torch.zeros(s, dtype=torch.int32) for s in ((4, 2), (8,), (4,), (5,))))
    return {"expert_pack": lambda: vf.expert_pack(x, plan),
            "expert_pack_q": lambda: vf.expert_pack_q(x, plan),
            "expert_merge": lambda: vf.expert_merge(packed, plan, w),
            "expert_merge_q": lambda: vf.expert_merge_q(packed, plan, w)}


def test_gradients_are_never_lost_silently(monkeypatch):
    """A pack or a merge records no graph, so it refuses what autograd follows;
    detached, without grad mode and inside a Function the same calls run."""
    seen = Recorder(monkeypatch)
    monkeypatch.setattr(vf, "_expert_call", lambda fn, d, stream, like: seen.calls.append(fn))
    x = torch.zeros(4, 64, dtype=torch.bfloat16, requires_grad=True)
    y = torch.zeros(8, 64, dtype=torch.bfloat16, requires_grad=True)
    w = torch.zeros(4, 2, requires_grad=True)
    live = dict(_calls(x, y, None))
    live.update({k + " with weights": f for k, f in _calls(x, y.detach(), w).items()})
    for name, call in live.items():
        with pytest.raises(ValueError, match="requires a gradient.*detach.*as its gradient"):
            call()
            pytest.fail("%s was accepted" % name)
    assert not seen.calls and not any(m[1] == "cuda" for m in seen.made)
    for name, call in _calls(x.detach(), y.detach(), w.detach()).items():
        call()
    with torch.no_grad():
        for name, call in live.items():
            call()

    class Pack(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return _calls(x, None, None)["expert_pack"]()

        @staticmethod
        def backward(ctx, grad):
            return None

    Pack.apply(x)
    # the gradients' own calls take what a graph holds: nothing follows them
    plan = vf.ExpertPlan(*(torch.zeros(s, dtype=torch.int32) for s in ((4, 2), (8,), (4,), (5,))))
    vf.expert_merge_backward(x.detach(), y, plan, w)
    assert seen.calls == (["vf_expert_pack"] * 2 + ["vf_expert_merge"] * 2) * 3 + [
        "vf_expert_pack", "vf_expert_merge_backward"]


@pytest.mark.parametrize("T,K,E,align", [(1, 1, 4, 65537), (4096, 2, 4096, 1 << 18), (1, 1, 4, 0),
                                         (1, 1, 4, -3), (1, 1, 0, 1), (1, 1, 4097, 1),
                                         (0, 0, 4, 1), (0, 1, 4, 1 << 40)])
def test_plan_refuses_sizes_before_it_allocates(monkeypatch, T, K, E, align):
    experts = torch.zeros(T, K, dtype=torch.int64)
    seen = Recorder(monkeypatch)
    with pytest.raises(vf.VFError):
        vf.expert_plan(experts, E, align=align)
    assert not seen.made and not seen.calls
