"""Edges of the expert relayouts: gradients that are not finite, or whose
products with codes leave float32 unless the scale comes first, indices in pinned
host memory, skewed routings and the exchange between ranks.

Bounds as in ``tests/test_gpu_expert.py``.
"""
import pytest
import torch

import sequence_head_relayout_gb300 as vf
from oracle import experts as X

from .test_gpu_expert import (BF16, DEV, F16, F32, FMT, backward_bounds, gen, make_plan,
                              packed_for, rows_like, routing, sentinel, weights_for, within)

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("oracle_built")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    vf.lib()
    yield
    torch.cuda.synchronize()


# ---- dropped slots of gradients that are not finite -----------------------------

def dropped_routing(E):
    """Tokens with all slots dropped, some and none; both kinds of dropped index."""
    return torch.tensor([[-1, -1, E, -1, -1], [0, -1, 1, E + 2, 2], [-1, 3, -1, 0, -1],
                         [1, 2, 3, 0, 1], [-1, -1, -1, -1, -1], [2, -1, 2, 1, -1],
                         [-1, -1, -1, -1, 3]])


def not_finite(grad):
    """Infinities and NaN in tokens 0 to 3, at both ends of the row and all over."""
    M = grad.shape[1]
    grad[0] = float("nan")
    grad[1, M - 1] = float("inf")
    grad[2, 0] = -float("inf")
    grad[3, M // 2] = float("nan")
    return grad


def check_backward(call, grad, values, plan, w, dtype, extra):
    gp = sentinel((plan.slot_of.numel(), grad.shape[1]), dtype)
    want, gw_want, mag = X.merge_backward(grad.cpu(), values, plan.row_of.cpu(),
                                          plan.offsets.cpu(), w, gp.cpu())
    got, gw = call(gp)
    dropped = plan.row_of < 0
    assert (gw[dropped] == 0).all(), "a dropped slot's gradient is %s" % gw[dropped].tolist()
    b1, b2 = backward_bounds(want, grad, mag, dtype, grad.shape[1], extra=extra)
    within(got, want, b1)
    within(gw, gw_want, b2)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M", [1, 7, 34, 100, 264, 2048])
def test_dropped_slots_have_no_gradient(M, dtype):
    E = 4
    e = dropped_routing(E)
    for align in (1, 4):
        plan = make_plan(e, E, align)
        y = packed_for(plan, M, dtype, M)
        grad = not_finite(rows_like(e.shape[0], M, dtype, M + 1)).to(DEV)
        w = weights_for(*e.shape, M, e, E)
        check_backward(lambda gp: vf.expert_merge_backward(grad, y, plan, w.to(DEV),
                                                           grad_packed=gp),
                       grad, y.cpu(), plan, w, dtype, 0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("M", [1, 7, 34, 100, 264, 2048])
def test_dropped_slots_have_no_gradient_from_codes(M, fmt):
    E, group = 4, 64
    e = dropped_routing(E)
    plan = make_plan(e, E, 4)
    y = packed_for(plan, M, BF16, M)
    grad = not_finite(rows_like(e.shape[0], M, BF16, M + 1)).to(DEV)
    w = weights_for(*e.shape, M, e, E)
    _, codes, scales = vf.expert_merge_q(y, plan, w.to(DEV), fmt, group)
    kept = X.checkpoint(y.cpu(), FMT[fmt], group)
    check_backward(lambda gp: vf.expert_merge_backward_q(grad, codes, scales, plan, w.to(DEV), fmt,
                                                         group, grad_packed=gp),
                   grad, X.values(kept[0], kept[1], FMT[fmt], group), plan, w, BF16, 1)


# ---- gradients and scales at opposite ends of float32 ------------------------------

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("M", [33, 34, 100, 256, 1024, 1003])
@pytest.mark.parametrize("powers", [(118, -90), (122, -95), (-130, 100)])
def test_backward_takes_code_times_scale(M, fmt, powers):
    """Each row is its codes times its scales: with huge gradients of tiny rows a
    sum of gradient times code would leave float32, with tiny gradients of huge
    rows it would lose bits, where the products with the row do neither."""
    T, K, E, group = 9, 3, 5, 128
    e = torch.randint(0, E, (T, K), generator=gen(M))
    plan = make_plan(e, E)
    y = (rows_like(T * K, M, F32, M) * 2.0 ** powers[1]).to(BF16).to(DEV)
    grad = (rows_like(T, M, F32, M + 1) * 2.0 ** powers[0]).to(BF16).to(DEV)
    w = weights_for(T, K, M)
    _, codes, scales = vf.expert_merge_q(y, plan, w.to(DEV), fmt, group)
    kept = X.checkpoint(y.cpu(), FMT[fmt], group)
    values = X.values(kept[0], kept[1], FMT[fmt], group)
    _, want, mag = X.merge_backward(grad.cpu(), values, plan.row_of.cpu(), plan.offsets.cpu(), w,
                                    y.cpu())
    assert torch.isfinite(grad).all() and mag.max() < 2.0 ** 60 and mag.min() > 2.0 ** -60
    check_backward(lambda gp: vf.expert_merge_backward_q(grad, codes, scales, plan, w.to(DEV), fmt,
                                                         group, grad_packed=gp),
                   grad, values, plan, w, BF16, 1)


# ---- plans of pinned host indices ----------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_plans_of_pinned_indices(dtype):
    """Plans over many blocks, on two streams behind other work, with pinned memory
    of the workspace's size taken and overwritten while they run."""
    T, K, E, align = 5000, 4, 64, 8
    words = vf.lib().vf_expert_workspace(T, K, E) // 4
    assert words > 0
    routings = [routing(T, K, E, seed) for seed in range(4)]
    pinned = [e.to(dtype).pin_memory() for e in routings]
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    for s in streams:
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
    plans, others = [], []
    for i, e in enumerate(pinned):
        plans.append(vf.expert_plan(e, E, align=align, stream=streams[i % 2]))
        others.append(torch.empty(words, dtype=torch.int32, pin_memory=True).fill_(1 << 20))
    torch.cuda.synchronize()
    for e, plan in zip(routings, plans):
        for a, b in zip(plan, X.plan(e, E, align)):
            assert not a.is_cuda and torch.equal(a, b)
    assert all((o == 1 << 20).all() for o in others)
    on_current = vf.expert_plan(pinned[0], E, align=align)
    torch.cuda.synchronize()
    assert torch.equal(on_current.row_of, plans[0].row_of)


@pytest.mark.parametrize("T", [700, 5000])
def test_indices_that_change_during_the_plan(T):
    """Both forms of the plan while the host rewrites its indices, all slots moving
    between the first and the last expert: any plan may come out, but every row it
    names exists, and nothing outside its tensors is written."""
    K, E = 4, 64
    assert (vf.lib().vf_expert_workspace(T, K, E) > 0) == (T == 5000)
    e = torch.zeros(T, K, dtype=torch.int64).pin_memory()
    rows, guard = vf.expert_rows(T, K, E), 1 << 18
    i32 = dict(dtype=torch.int32, device=DEV)
    wide = [torch.full((n + 2 * guard,), 12345, **i32) for n in (T * K, rows)]
    row_of, slot_of = (b[guard:-guard] for b in wide)
    plan = vf.ExpertPlan(row_of.view(T, K), slot_of, torch.empty(E, **i32),
                         torch.empty(E + 1, **i32))
    stream, done = torch.cuda.Stream(DEV), torch.cuda.Event()
    torch.cuda.synchronize()
    for _ in range(20):
        for _ in range(10):
            vf.expert_plan(e, E, out=plan, stream=stream)
        done.record(stream)
        while not done.query():
            e.fill_(E - 1)
            e.fill_(0)
        assert ((row_of >= -1) & (row_of < rows)).all()
        for b in wide:
            assert (b[:guard] == 12345).all() and (b[-guard:] == 12345).all()
    vf.expert_plan(e, E, out=plan)
    for a, b in zip(plan, X.plan(e, E)):
        assert torch.equal(a.cpu(), b)


# ---- routings with most slots in a few experts ----------------------------------------

@pytest.mark.parametrize("how", ["one", "few", "falling"])
@pytest.mark.parametrize("T,K,E,align", [(150000, 8, 64, 128), (400001, 3, 256, 1),
                                         (70000, 4, 4096, 16)])
def test_skewed_plans_over_many_blocks(T, K, E, align, how):
    g = torch.Generator(device=DEV).manual_seed(T)
    if how == "one":
        e = torch.full((T, K), E - 1, device=DEV)
    elif how == "few":                       # nine of ten slots in two experts
        e = torch.randint(0, E, (T, K), generator=g, device=DEV)
        e[torch.rand(T, K, generator=g, device=DEV) < 0.9] = 1
        e[::3] = E - 2
    else:                                    # expert e about as often as 1 / (e + 1)
        u = torch.rand(T, K, generator=g, device=DEV, dtype=torch.float64)
        e = ((E + 1.0) ** u).long() - 1
    assert vf.lib().vf_expert_workspace(T, K, E) > 0
    plan = vf.expert_plan(e, E, align=align)
    flat = e.reshape(-1)
    counts = torch.bincount(flat, minlength=E)
    steps = (counts + align - 1) // align * align
    assert torch.equal(plan.counts.long(), counts)
    assert torch.equal(plan.offsets.long()[1:], steps.cumsum(0)) and int(plan.offsets[0]) == 0
    order = torch.argsort(flat, stable=True)
    at = torch.arange(T * K, device=DEV) - (counts.cumsum(0) - counts)[flat[order]]
    row = plan.offsets.long()[flat[order]] + at
    assert torch.equal(plan.row_of.reshape(-1)[order].long(), row)
    slots = torch.full_like(plan.slot_of, -1)
    slots[row] = order.int()
    assert torch.equal(plan.slot_of, slots)


# ---- the exchange between ranks ---------------------------------------------------------

@pytest.mark.parametrize("E", [12, 10])
def test_exchange_of_expert_rows(E):
    """Experts spread over P ranks, all of them emulated here one after the other.
    Source s packs by expert and sends destination p the rows offsets[p*E//P] ..
    offsets[(p+1)*E//P]; the receiver sorts the P segments by its own experts with a
    second plan (one slot per row) and merges them back into the order they came in;
    the source merges with its weights.  Rows are moved and scaled by powers of two,
    so the result is that of one rank with all experts, bit for bit."""
    P, T, K, M = 4, 60, 3, 72
    first = [p * E // P for p in range(P + 1)]
    scale = 2.0 ** (torch.arange(E) % 7 - 3)
    sent, plans, xs, ws = [], [], [], []
    for s in range(P):
        e = routing(T + s, K, E, 40 + s)
        xs.append(rows_like(T + s, M, BF16, 50 + s).to(DEV))
        ws.append(weights_for(T + s, K, 60 + s).to(DEV))
        plans.append(vf.expert_plan(e.to(DEV), E))
        sent.append(vf.expert_pack(xs[s], plans[s]))
    offsets = [p.offsets.tolist() for p in plans]          # split sizes: read back once

    def segment(s, p):
        return slice(offsets[s][first[p]], offsets[s][first[p + 1]])

    returned = [torch.empty_like(b) for b in sent]
    for p in range(P):
        recv = torch.cat([sent[s][segment(s, p)] for s in range(P)])
        experts = torch.cat([torch.repeat_interleave(
            torch.arange(first[p + 1] - first[p]),
            plans[s].counts[first[p]:first[p + 1]].long().cpu()) for s in range(P)])
        local = vf.expert_plan(experts.to(DEV)[:, None], first[p + 1] - first[p])
        rows = vf.expert_pack(recv, local)
        at = local.offsets.tolist()
        for i in range(first[p + 1] - first[p]):
            rows[at[i]:at[i + 1]] *= scale[first[p] + i].item()
        back = vf.expert_merge(rows, local)
        done = 0
        for s in range(P):
            n = offsets[s][first[p + 1]] - offsets[s][first[p]]
            returned[s][segment(s, p)] = back[done:done + n]
            done += n
    for s in range(P):
        whole = sent[s].clone()
        for i in range(E):
            whole[offsets[s][i]:offsets[s][i + 1]] *= scale[i].item()
        got = vf.expert_merge(returned[s], plans[s], ws[s])
        assert torch.equal(got, vf.expert_merge(whole, plans[s], ws[s]))
