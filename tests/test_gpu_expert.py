"""GPU tests of the expert relayouts against the CPU oracle.

Plans, packs, checkpoints and restored rows have one correct result and are
compared bit for bit.  Sums are compared with float64, within bounds derived
from the arithmetic that the header states (float32, one rounding at the end):

* a float32 sum of n products by fused multiply-adds is off by at most
  n u / (1 - n u) times the sum of the magnitudes, u = 2^-24, in any order;
* a rounding to the output type is off by at most half a unit, eps / 2
  relative, or half the smallest subnormal.
"""
import pytest
import torch

import sequence_head_relayout_gb300 as vf
from oracle import experts as X
from oracle import loops

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("oracle_built")]

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FMT = {"int8": loops.INT8, "e4m3": loops.E4M3}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    vf.lib()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rounding(x, dtype):
    """Bound of one rounding of values near x (float64) to dtype."""
    info = torch.finfo(dtype)
    return x.abs() * (info.eps / 2) + info.smallest_normal * info.eps / 2


def within(got, want, bound):
    """Same NaN and infinite places, and |got - want| <= bound elsewhere."""
    got = got.cpu().double()
    assert got.shape == want.shape
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    off = (got - want).abs()[fine] - bound[fine]
    assert off.numel() == 0 or off.max() <= 0, "off by %g over the bound" % off.max()


def routing(T, K, E, seed, how="mixed"):
    g = gen(seed)
    if how == "none":
        return torch.full((T, K), -1)
    if how == "one":
        return torch.full((T, K), E - 1)
    e = torch.randint(0, E, (T, K), generator=g)
    if how == "mixed":                       # a third dropped, by both kinds of index
        d = torch.rand(T, K, generator=g)
        e[d < 0.2] = -1
        e[d > 0.9] = E + 3
        if T > 2:
            e[T // 2] = -1                   # a token with no expert
    return e


def rows_like(n, M, dtype, seed):
    x = torch.randn(n, M, generator=gen(seed)) * 3
    return x.to(dtype)


def token_view(T, M, dtype, seed, layout, device=DEV):
    """A [T,M] view of the layout, filled with random values."""
    x = rows_like(T, M, dtype, seed).to(device)
    if layout == "contiguous":
        return x
    if layout == "padded8":
        v = torch.empty(T, M + 8, dtype=dtype, device=device)[:, :M]
    elif layout == "padded1":                # odd rows: no wide access possible
        v = torch.empty(T, M + 1, dtype=dtype, device=device)[:, 1:]
    elif layout == "transposed":
        v = torch.empty(M, T, dtype=dtype, device=device).t()
    else:                                    # every second column
        v = torch.empty(T, 2 * M, dtype=dtype, device=device)[:, ::2]
    v.copy_(x)
    return v


LAYOUTS = ["contiguous", "padded8", "padded1", "transposed", "strided"]


def make_plan(e, E, align=1, dtype=torch.int64):
    return vf.expert_plan(e.to(dtype).to(DEV), E, align=align)


# ---- the plan ----------------------------------------------------------------------

PLANS = [
    # T, K, E, align
    (1, 1, 1, 1), (1, 8, 256, 1), (1, 8, 256, 16), (5, 2, 3, 1), (16, 8, 128, 128),
    (33, 3, 7, 5), (1000, 8, 64, 128), (1024, 8, 256, 1), (1025, 8, 256, 8), (3001, 6, 512, 1),
    (20000, 2, 8, 64), (9, 2, 4096, 1), (9000, 3, 4096, 4), (17, 40, 64, 1), (4099, 4, 1000, 1),
]


@pytest.mark.parametrize("how", ["mixed", "all", "one", "none"])
@pytest.mark.parametrize("shape", PLANS)
def test_plan(shape, how):
    T, K, E, align = shape
    e = routing(T, K, E, T + K, how)
    want = X.plan(e, E, align)
    for dtype in (torch.int32, torch.int64):
        got = make_plan(e, E, align, dtype)
        for name, a, b in zip(vf.ExpertPlan._fields, got, want):
            assert torch.equal(a.cpu(), b), name


def test_plan_strided_and_reused():
    T, K, E = 700, 4, 20
    e = routing(T, K, E, 1)
    wide = torch.full((T, 3 * K), 5, device=DEV)
    wide[:, ::3] = e.to(DEV)
    cols = e.to(DEV).t().contiguous().t()
    want = X.plan(e, E, 2)
    out = vf.expert_plan(wide[:, ::3], E, align=2)
    for view in (cols, wide[:, ::3]):
        for t in out[:4]:
            t.fill_(-7)
        assert vf.expert_plan(view, E, align=2, out=out) is out
        for a, b in zip(out, want):
            assert torch.equal(a.cpu(), b)
    one = e[:, :1].to(DEV).expand(T, 3)                     # a broadcast routing
    for a, b in zip(vf.expert_plan(one, E), X.plan(one.cpu(), E)):
        assert torch.equal(a.cpu(), b)


def test_plan_extreme_indices():
    big = 2 ** 31
    e = torch.tensor([[0, big], [-big * 2, 1], [2 ** 62, big * 2 + 1], [-2 ** 63, 2 ** 63 - 1]])
    want = X.plan(e, 2)
    for a, b in zip(make_plan(e, 2), want):
        assert torch.equal(a.cpu(), b)
    assert want[2].tolist() == [1, 1]


def test_plan_of_no_tokens():
    p = vf.expert_plan(torch.empty(0, 3, dtype=torch.int64, device=DEV), 5, align=4)
    assert p.row_of.shape == (0, 3) and p.slot_of.numel() == 0
    assert p.counts.tolist() == [0] * 5 and p.offsets.tolist() == [0] * 6


def test_large_plan_is_a_stable_sort():
    T, K, E, align = 200000, 8, 256, 128
    e = torch.randint(-1, E, (T, K), device=DEV)
    p = vf.expert_plan(e, E, align=align)
    flat = e.reshape(-1)
    kept = (flat >= 0).nonzero()[:, 0]
    assert torch.equal(p.counts.long(), torch.bincount(flat[kept], minlength=E))
    steps = (p.counts.long() + align - 1) // align * align
    assert torch.equal(p.offsets.long()[1:], steps.cumsum(0)) and int(p.offsets[0]) == 0
    order = kept[torch.argsort(flat[kept], stable=True)]
    at = torch.arange(order.numel(), device=DEV)
    first = p.counts.long().cumsum(0) - p.counts.long()
    row = p.offsets.long()[flat[order]] + at - first[flat[order]]
    assert torch.equal(p.row_of.reshape(-1)[order].long(), row)
    assert torch.equal(p.slot_of[row].long(), order)
    assert int((p.row_of >= 0).sum()) == kept.numel() == int((p.slot_of >= 0).sum())


# ---- the pack -----------------------------------------------------------------------

WIDTHS = [1, 2, 7, 8, 33, 100, 256, 260, 264, 520, 1003, 2048]


def sentinel(shape, dtype):
    return torch.full(shape, 77.0, dtype=dtype, device=DEV)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M", WIDTHS)
def test_pack(M, dtype):
    for T, K, E, align, how in ((1, 2, 4, 1, "all"), (19, 3, 5, 4, "mixed"), (40, 1, 3, 1, "mixed"),
                                (6, 2, 9, 7, "none")):
        e = routing(T, K, E, M, how)
        plan = make_plan(e, E, align)
        for layout in LAYOUTS if T == 19 else LAYOUTS[:1]:
            x = token_view(T, M, dtype, M + T, layout)
            out = sentinel((plan.slot_of.numel(), M), dtype)
            before = out.cpu()
            assert vf.expert_pack(x, plan, out=out) is out
            want = X.pack(x.cpu(), plan.slot_of.cpu(), plan.offsets.cpu(), K, before)
            assert torch.equal(out.cpu().view(torch.uint8), want.view(torch.uint8)), layout


def test_pack_keeps_bit_patterns():
    x = torch.randint(-2 ** 15, 2 ** 15, (50, 72), dtype=torch.int16).view(BF16).to(DEV)
    plan = make_plan(routing(50, 2, 6, 3, "all"), 6)
    out = vf.expert_pack(x, plan)
    token = (plan.slot_of // 2).long()
    assert torch.equal(out.view(torch.int16), x.view(torch.int16)[token])


def test_pack_many_slots_per_token():
    T, K, E, M = 7, 70, 9, 40
    plan = make_plan(routing(T, K, E, 2), E, 8)
    x = token_view(T, M, BF16, 1, "contiguous")
    out = sentinel((plan.slot_of.numel(), M), BF16)
    want = X.pack(x.cpu(), plan.slot_of.cpu(), plan.offsets.cpu(), K, out.cpu())
    assert torch.equal(vf.expert_pack(x, plan, out=out).cpu(), want)


# ---- the merge and its gradients ------------------------------------------------------

def weights_for(T, K, seed, e=None, E=None):
    w = torch.softmax(torch.randn(T, K, generator=gen(seed)), 1) * 2
    if e is not None:                        # a dropped slot's weight is never used
        w[(e < 0) | (e >= E)] = float("nan")
    return w


def packed_for(plan, M, dtype, seed):
    y = rows_like(plan.slot_of.numel(), M, dtype, seed).to(DEV)
    y[plan.slot_of < 0] = float("nan")       # rows that no slot owns are never read
    return y


def merge_bound(want, mag, K, dtype):
    total = mag * (K * U / (1 - K * U))
    return total + rounding(want.abs() + total, dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M", WIDTHS)
def test_merge(M, dtype):
    for T, K, E, align, how in ((1, 2, 4, 1, "all"), (19, 3, 5, 4, "mixed"), (11, 8, 16, 1, "mixed"),
                                (6, 2, 9, 7, "none"), (5, 19, 4, 1, "all")):
        e = routing(T, K, E, M, how)
        plan = make_plan(e, E, align)
        y = packed_for(plan, M, dtype, M)
        for w in (None, weights_for(T, K, M, e, E)):
            want, mag = X.merge(y.cpu(), plan.row_of.cpu(), w)
            bound = merge_bound(want, mag, K, dtype)
            wd = None if w is None else w.to(DEV)
            within(vf.expert_merge(y, plan, wd), want, bound)
            if T == 19:
                for layout in LAYOUTS[1:]:
                    out = token_view(T, M, dtype, 1, layout)
                    assert vf.expert_merge(y, plan, wd, out=out) is out
                    within(out, want, bound)


def test_merge_writes_only_its_view():
    T, K, E, M = 12, 2, 4, 96
    plan = make_plan(routing(T, K, E, 5), E)
    y = packed_for(plan, M, BF16, 5)
    buf = sentinel((T + 2, M + 40), BF16)
    vf.expert_merge(y, plan, out=buf[1:-1, 8:8 + M])
    edge = buf.clone()
    edge[1:-1, 8:8 + M] = 77
    assert (edge == 77).all()


def test_merge_of_nothing_is_zero():
    plan = make_plan(torch.full((5, 2), -1), 3)
    y = torch.full((10, 64), float("nan"), dtype=BF16, device=DEV)
    w = torch.full((5, 2), float("inf"), device=DEV)
    assert (vf.expert_merge(y, plan, w) == 0).all()
    gp, gw = vf.expert_merge_backward(torch.ones(5, 64, dtype=BF16, device=DEV), y, plan, w,
                                      grad_packed=sentinel((10, 64), BF16))
    assert (gw == 0).all() and (gp == 77).all()


def test_merge_non_finite_rows():
    plan = make_plan(torch.tensor([[0, 1], [1, 0], [1, -1]]), 2)
    # rows: expert 0: slots 0, 3; expert 1: slots 1, 2, 4
    y = torch.ones(6, 64, dtype=F32, device=DEV)
    y[0, 3], y[2, 5], y[3, 9], y[5] = float("inf"), -float("inf"), float("nan"), float("nan")
    w = torch.tensor([[2.0, 0.0], [1.0, -1.0], [0.0, 1.0]])
    want, mag = X.merge(y.cpu(), plan.row_of.cpu(), w)
    assert torch.isinf(want).any() and torch.isnan(want).any()
    within(vf.expert_merge(y, plan, w.to(DEV)), want, merge_bound(want, mag, 2, F32))


def backward_bounds(gp, grad, gw_mag, dtype, M, extra=0):
    n = M + extra
    product = gp.abs() * U
    return product + rounding(gp.abs() + product, dtype), gw_mag * (n * U / (1 - n * U))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M", WIDTHS)
def test_merge_backward(M, dtype):
    for T, K, E, align, how in ((1, 2, 4, 1, "all"), (19, 3, 5, 4, "mixed"), (11, 8, 16, 1, "mixed"),
                                (6, 2, 9, 7, "none"), (5, 19, 4, 1, "all")):
        e = routing(T, K, E, M, how)
        plan = make_plan(e, E, align)
        y = packed_for(plan, M, dtype, M)
        w = weights_for(T, K, M, e, E)
        for layout in LAYOUTS if T == 19 else LAYOUTS[:1]:
            grad = token_view(T, M, dtype, M + 1, layout)
            gp = sentinel((plan.slot_of.numel(), M), dtype)
            want, gw_want, mag = X.merge_backward(grad.cpu(), y.cpu(), plan.row_of.cpu(),
                                                  plan.offsets.cpu(), w, gp.cpu())
            got, gw = vf.expert_merge_backward(grad, y, plan, w.to(DEV), grad_packed=gp)
            b1, b2 = backward_bounds(want, grad, mag, dtype, M)
            within(got, want, b1)
            within(gw, gw_want, b2)


def test_backward_of_a_broadcast_gradient_and_strided_weights():
    T, K, E, M = 23, 4, 6, 136
    plan = make_plan(routing(T, K, E, 9), E, 2)
    y = packed_for(plan, M, BF16, 3)
    w = torch.randn(K, T, generator=gen(1)).to(DEV).t()
    for grad in (torch.randn(M, generator=gen(2)).to(BF16).to(DEV).expand(T, M),
                 torch.randn(T, 1, generator=gen(2)).to(BF16).to(DEV).expand(T, M),
                 torch.ones((), dtype=BF16, device=DEV).expand(T, M)):
        gp = sentinel((plan.slot_of.numel(), M), BF16)
        want, gw_want, mag = X.merge_backward(grad.cpu(), y.cpu(), plan.row_of.cpu(),
                                              plan.offsets.cpu(), w.cpu(), gp.cpu())
        got, gw = vf.expert_merge_backward(grad, y, plan, w, grad_packed=gp)
        b1, b2 = backward_bounds(want, grad, mag, BF16, M)
        within(got, want, b1)
        within(gw, gw_want, b2)


def test_backward_without_columns():
    plan = make_plan(torch.tensor([[0, 1]]), 2)
    z = torch.empty(1, 0, dtype=BF16, device=DEV)
    gw = torch.full((1, 2), 7.0, device=DEV)
    vf.expert_merge_backward(z, torch.empty(2, 0, dtype=BF16, device=DEV), plan,
                             torch.ones(1, 2, device=DEV), grad_weights=gw)
    assert (gw == 0).all()
    assert vf.expert_merge(torch.empty(2, 0, dtype=BF16, device=DEV), plan).shape == (1, 0)
    assert vf.expert_pack(z, plan).shape == (2, 0)


def test_gradients_against_differences():
    """The merge is linear in the rows and in the weights, so a central
    difference is its directional derivative up to the roundings: each of the
    two float32 sums is off by its bound, and so is the gradient side."""
    T, K, E, M = 13, 3, 5, 72
    plan = make_plan(routing(T, K, E, 4), E)
    y = rows_like(plan.slot_of.numel(), M, F32, 1).to(DEV)
    w = weights_for(T, K, 2).to(DEV)
    grad = rows_like(T, M, F32, 3).to(DEV)
    gp = torch.zeros_like(y)
    gp, gw = vf.expert_merge_backward(grad, y, plan, w, grad_packed=gp)
    for target in ("rows", "weights"):
        d = torch.randn((y if target == "rows" else w).shape, generator=gen(8)).to(DEV)
        there = [vf.expert_merge(y + s * d if target == "rows" else y, plan,
                                 w + s * d if target == "weights" else w) for s in (1.0, -1.0)]
        diff = ((there[0].double() - there[1].double()) * grad.double()).sum() / 2
        want = ((gp if target == "rows" else gw).double() * d.double()).sum()
        # every term of either side is rounded at most M + K + 3 times (the sums,
        # w +- d or y +- d, the products); their magnitudes:
        mag = (X.merge((y.abs() + d.abs() if target == "rows" else y.abs()).cpu(),
                       plan.row_of.cpu(),
                       (w.abs() + d.abs() if target == "weights" else w.abs()).cpu())[0]
               * grad.abs().cpu().double()).sum()
        assert (diff - want).abs().item() <= 2 * (M + K + 3) * U * mag.item()


def test_pack_and_unweighted_merge_are_adjoint():
    T, K, E, M = 21, 4, 6, 80
    plan = make_plan(routing(T, K, E, 6), E, 4)
    x, y = rows_like(T, M, F32, 1).to(DEV), packed_for(plan, M, F32, 2)
    out = torch.zeros_like(y)
    left = (vf.expert_pack(x, plan, out=out).double() * torch.nan_to_num(y).double()).sum()
    merged = vf.expert_merge(y, plan)
    right = (x.double() * merged.double()).sum()
    mag = (x.cpu().double().abs() * X.merge(y.cpu().abs(), plan.row_of.cpu())[0]).sum()
    assert (left - right).abs().item() <= K * U / (1 - K * U) * mag.item() * (1 + U)


# ---- 8-bit checkpoints ------------------------------------------------------------------

def plant(x):
    """Groups of zeros, of tiny and huge values, and non-finite ones."""
    if x.shape[0] > 8:
        x[1] = 0
        x[2] *= 2.0 ** -100
        x[3] *= 2.0 ** 100
        x[4, :1] = float("inf")
        x[5, -1:] = float("nan")
        x[6] = -0.0
    return x


def same_kept(codes, scales, want, rows=None):
    wc, ws = want
    c, s = codes.cpu().view(torch.uint8), scales.cpu().view(torch.int32)
    wc, ws = wc.view(torch.uint8), ws.contiguous().view(torch.int32)
    if rows is not None:
        c, s, wc, ws = c[rows], s[rows], wc[rows], ws[rows]
    assert torch.equal(c, wc) and torch.equal(s, ws)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("M", [1, 7, 8, 33, 100, 256, 260, 520, 1003, 1024, 1280])
def test_pack_q_and_restore(M, group, fmt):
    for T, K, E, align, how in ((1, 2, 4, 1, "all"), (19, 3, 5, 4, "mixed")):
        plan = make_plan(routing(T, K, E, M, how), E, align)
        for layout in LAYOUTS if T == 19 and group in (32, 128) else LAYOUTS[:1]:
            x = token_view(T, M, BF16, M + T, layout)
            x.copy_(plant(x.clone()))
            n = plan.slot_of.numel()
            packed, codes, scales = vf.expert_pack_q(x, plan, fmt, group, out=sentinel((n, M), BF16))
            want = X.pack(x.cpu(), plan.slot_of.cpu(), plan.offsets.cpu(), K,
                          sentinel((n, M), BF16).cpu())
            assert torch.equal(packed.cpu().view(torch.int16), want.view(torch.int16))
            kept = X.checkpoint(x.cpu(), FMT[fmt], group)
            same_kept(codes, scales, kept)
            got = vf.expert_restore_q(codes, scales, plan, fmt, group, out=sentinel((n, M), BF16))
            rows = X.restore(kept[0], kept[1], FMT[fmt], group)
            want = X.pack(rows, plan.slot_of.cpu(), plan.offsets.cpu(), K,
                          sentinel((n, M), BF16).cpu())
            assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("M", [1, 7, 8, 33, 100, 256, 260, 520, 1003, 1024, 1280])
def test_merge_q_and_backward(M, group, fmt):
    for T, K, E, align, how in ((1, 2, 4, 1, "all"), (19, 3, 5, 4, "mixed"), (7, 11, 6, 1, "all")):
        e = routing(T, K, E, M, how)
        plan = make_plan(e, E, align)
        y = plant(rows_like(plan.slot_of.numel(), M, BF16, M)).to(DEV)
        y[plan.slot_of < 0] = float("nan")
        w = weights_for(T, K, M, e, E)
        out, codes, scales = vf.expert_merge_q(y, plan, w.to(DEV), fmt, group)
        want, mag = X.merge(y.cpu(), plan.row_of.cpu(), w)
        within(out, want, merge_bound(want, mag, K, BF16))
        kept = X.checkpoint(y.cpu(), FMT[fmt], group)
        same_kept(codes, scales, kept, plan.slot_of.cpu() >= 0)
        grad = token_view(T, M, BF16, M + 1, "padded1" if T == 19 else "contiguous")
        values = X.values(kept[0], kept[1], FMT[fmt], group)
        gp = sentinel((plan.slot_of.numel(), M), BF16)
        want, gw_want, mag = X.merge_backward(grad.cpu(), values, plan.row_of.cpu(),
                                              plan.offsets.cpu(), w, gp.cpu())
        got, gw = vf.expert_merge_backward_q(grad, codes, scales, plan, w.to(DEV), fmt, group,
                                             grad_packed=gp)
        b1, b2 = backward_bounds(want, grad, mag, BF16, M, extra=1)   # 1: code times scale
        within(got, want, b1)
        # 8 values of a group may reach 2^100 * 2^100 and overflow float32: infinite there
        top = torch.finfo(F32).max
        fits = torch.isnan(gw_want) | (mag < top / 2)
        within(torch.where(fits.to(DEV), gw, 0), torch.where(fits, gw_want, 0), b2)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("M", [100, 101, 256])
def test_checkpoints_from_elsewhere(M, fmt):
    """Any code and scale bits: scales of zero, infinity and NaN, every code (but
    E4M3's NaN, whose payload is unspecified)."""
    T, K, E, group = 30, 2, 4, 32
    plan = make_plan(routing(T, K, E, 1, "all"), E)
    n, groups = plan.slot_of.numel(), -(-M // group)
    g = gen(M)
    codes = torch.randint(0, 256, (n, M), generator=g).to(torch.uint8)
    if fmt == "e4m3":
        codes[(codes & 0x7F) == 0x7F] = 0
    scales = torch.randn(n, groups, generator=g).abs() * 2.0 ** torch.randint(
        -40, 40, (n, groups), generator=g)
    scales[::5], scales[1::7], scales[2::9] = 0, float("inf"), float("nan")
    code_type = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
    dc, ds = codes.view(code_type).to(DEV), scales.to(DEV)
    got = vf.expert_restore_q(dc[:T].contiguous(), ds[:T].contiguous(), plan, fmt, group)
    rows = X.restore(codes[:T], scales[:T], FMT[fmt], group)
    token = (plan.slot_of // K).long().cpu()
    assert torch.equal(got.cpu().view(torch.int16), rows[token].view(torch.int16))
    grad, w = rows_like(T, M, BF16, 2), weights_for(T, K, 3)
    values = X.values(codes, scales, FMT[fmt], group)
    before = torch.zeros(n, M, dtype=BF16)
    want, gw_want, mag = X.merge_backward(grad, values, plan.row_of.cpu(), plan.offsets.cpu(), w,
                                          before)
    gp, gw = vf.expert_merge_backward_q(grad.to(DEV), dc, ds, plan, w.to(DEV), fmt, group)
    b1, b2 = backward_bounds(want, grad, mag, BF16, M, extra=1)
    within(gp, want, b1)
    within(gw, gw_want, b2)


def test_merge_q_leaves_unowned_rows():
    plan = make_plan(torch.tensor([[0, -1], [1, 0]]), 2, 4)
    n, M = plan.slot_of.numel(), 96
    y = packed_for(plan, M, BF16, 1)
    codes = torch.full((n, M), 55, dtype=torch.int8, device=DEV)
    scales = torch.full((n, 1), 7.0, device=DEV)
    vf.expert_merge_q(y, plan, None, "int8", 128, codes=codes, scales=scales)
    unowned = plan.slot_of < 0
    assert (codes[unowned] == 55).all() and (scales[unowned] == 7).all()


def test_hostile_plans_stay_in_bounds():
    """Row numbers outside the packed side are dropped, offsets outside it zero
    nothing outside it (the buffers are parts of a larger one, checked around)."""
    T, K, E, M, n = 9, 2, 3, 64, 12
    row_of = torch.tensor([[0, 12], [-5, 3], [2 ** 31 - 1, 5], [-2 ** 31, 7], [1, 2], [4, 6],
                           [8, 9], [10, 11], [100, -1]], dtype=torch.int32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    plan = vf.ExpertPlan(row_of, torch.full((n,), -1, **i32),
                         torch.tensor([-9, 5, 2 ** 31 - 1], **i32),
                         torch.tensor([-2 ** 31, 7, 2 ** 31 - 1, 2 ** 31 - 1], **i32), 8)
    buf = sentinel((n + 8, M), F32)
    x = rows_like(T, M, F32, 1).to(DEV)
    vf.expert_pack(x, plan, out=buf[4:-4])
    assert (buf[:4] == 77).all() and (buf[-4:] == 77).all()
    y = rows_like(n, M, F32, 2).to(DEV)
    there = (row_of >= 0) & (row_of < n)
    want, mag = X.merge(y.cpu(), torch.where(there, row_of, -1).cpu())
    within(vf.expert_merge(y, plan), want, merge_bound(want, mag, K, F32))
    buf.fill_(77)
    _, gw = vf.expert_merge_backward(x, y, plan, torch.ones(T, K, device=DEV),
                                     grad_packed=buf[4:-4])
    assert (buf[:4] == 77).all() and (buf[-4:] == 77).all() and (gw[~there] == 0).all()
