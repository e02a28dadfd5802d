"""Oracle of the expert relayouts: plain CPU loops and float64 arithmetic over
the definitions of ``include/vf_relayout.h`` ("Expert relayouts"), sharing no
code with the library.

Tensors are CPU tensors.  ``merge`` and ``merge_backward`` return float64
results and, beside each, the sum of the magnitudes of its terms, from which a
test derives how far a float32 sum may be off.
"""
import torch

from . import loops

NAN_SCALE_BITS = 0x7FC00000


def plan(experts: torch.Tensor, E: int, align: int = 1):
    """(row_of, slot_of, counts, offsets) int32, slot by slot."""
    T, K = experts.shape
    chosen = [int(e) for e in experts.reshape(-1).tolist()]
    members = [[] for _ in range(E)]
    for i, e in enumerate(chosen):
        if 0 <= e < E:
            members[e].append(i)
    rows = T * K + min(E, T * K) * (align - 1)
    row_of, slot_of = [-1] * (T * K), [-1] * rows
    offsets, counts = [0], []
    for m in members:
        at = offsets[-1]
        for rank, i in enumerate(m):
            row_of[i] = at + rank
            slot_of[at + rank] = i
        counts.append(len(m))
        while at % align or at < offsets[-1] + len(m):
            at += 1
        offsets.append(at)
    i32 = torch.int32
    return (torch.tensor(row_of, dtype=i32).view(T, K), torch.tensor(slot_of, dtype=i32),
            torch.tensor(counts, dtype=i32), torch.tensor(offsets, dtype=i32))


def pack(tokens: torch.Tensor, slot_of: torch.Tensor, offsets: torch.Tensor, K: int,
         before: torch.Tensor) -> torch.Tensor:
    """``before`` with every row below offsets[E] written: a token's row, or
    zeros in a gap."""
    out = before.clone()
    for r in range(int(offsets[-1])):
        i = int(slot_of[r])
        out[r] = tokens[i // K] if i >= 0 else 0
    return out


def merge(packed: torch.Tensor, row_of: torch.Tensor, weights=None):
    """(sum [T,M], sum of magnitudes [T,M]) in float64."""
    T, K = row_of.shape
    out = torch.zeros((T, packed.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(out)
    for t in range(T):
        for k in range(K):
            r = int(row_of[t, k])
            if r >= 0:
                term = packed[r].double() * (1.0 if weights is None else float(weights[t, k]))
                out[t] += term
                mag[t] += term.abs()
    return out, mag


def merge_backward(grad: torch.Tensor, packed: torch.Tensor, row_of: torch.Tensor,
                   offsets: torch.Tensor, weights: torch.Tensor, before: torch.Tensor):
    """(grad_packed float64, with ``before``'s rows behind the last expert;
    grad_weights float64; sum of magnitudes of each grad_weights)."""
    T, K = row_of.shape
    gp = before.double().clone()
    gp[:int(offsets[-1])] = 0
    gw = torch.zeros((T, K), dtype=torch.float64)
    mag = torch.zeros_like(gw)
    for t in range(T):
        g = grad[t].double()
        for k in range(K):
            r = int(row_of[t, k])
            if r >= 0:
                gp[r] = g * float(weights[t, k])
                terms = g * packed[r].double()
                gw[t, k] = terms.sum()
                mag[t, k] = terms.abs().sum()
    return gp, gw, mag


def checkpoint(x: torch.Tensor, fmt: int, group: int):
    """(codes [n,M], scales [n,groups]) of bfloat16 rows: each group is a head
    row of the lossy transport's oracle (a short last group is padded with
    zeros, which change neither its largest magnitude nor its other codes)."""
    n, M = x.shape
    groups = -(-M // group)
    wide = torch.zeros((n, groups * group), dtype=x.dtype)
    wide[:, :M] = x
    codes, scales = loops.attn_split_q(wide.view(n, groups, group), 1, 1, fmt)
    return codes.view(n, groups * group)[:, :M].contiguous(), scales.view(n, groups)


def restore(codes: torch.Tensor, scales: torch.Tensor, fmt: int, group: int) -> torch.Tensor:
    """bfloat16 rows of a checkpoint, through the lossy transport's oracle."""
    n, M = codes.shape
    groups = scales.shape[1]
    wide = torch.zeros((n, groups * group), dtype=codes.dtype)
    wide[:, :M] = codes
    out = loops.head_merge_q(wide.reshape(-1), scales.reshape(-1), n, groups, group, 1, 1, fmt)
    return out.view(n, groups * group)[:, :M].contiguous().view(torch.bfloat16)


def values(codes: torch.Tensor, scales: torch.Tensor, fmt: int, group: int) -> torch.Tensor:
    """float64 values of a checkpoint: code times scale, NaN where the scale is
    not finite."""
    n, M = codes.shape
    if fmt == loops.INT8:
        code = codes.view(torch.int8).double()
    else:
        table = torch.tensor([loops.e4m3_decode(c) for c in range(256)], dtype=torch.float64)
        code = table[codes.view(torch.uint8).long()]
    s = scales.double().repeat_interleave(group, dim=1)[:, :M]
    return torch.where(torch.isfinite(s), code * s, torch.full_like(s, float("nan")))


def product(packed: torch.Tensor, weights: torch.Tensor, counts: torch.Tensor,
            offsets: torch.Tensor, before: torch.Tensor):
    """(packed rows times their experts' weights, with ``before``'s rows behind the
    last expert and zeros in the gaps; sum of the magnitudes of its terms)."""
    out = before.double().clone()
    mag = torch.zeros_like(out)
    out[:int(offsets[-1])] = 0
    for e in range(counts.numel()):
        at, n = int(offsets[e]), int(counts[e])
        x, w = packed[at:at + n].double(), weights[e].double()
        out[at:at + n] = x @ w.t()
        mag[at:at + n] = x.abs() @ w.abs().t()
    return out, mag


def weight_grad(grad: torch.Tensor, packed: torch.Tensor, counts: torch.Tensor,
                offsets: torch.Tensor):
    """(gradient of the product's weights, sum of the magnitudes of its terms)."""
    E = counts.numel()
    out = torch.zeros((E, grad.shape[1], packed.shape[1]), dtype=torch.float64)
    mag = torch.zeros_like(out)
    for e in range(E):
        at, n = int(offsets[e]), int(counts[e])
        g, x = grad[at:at + n].double(), packed[at:at + n].double()
        out[e] = g.t() @ x
        mag[e] = g.abs().t() @ x.abs()
    return out, mag
