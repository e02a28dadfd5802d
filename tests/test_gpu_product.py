"""GPU tests of the experts' products against the CPU oracle in float64.

Bounds: products of 16-bit values are exact in float32, and a sum of n of them in
any order, by additions that round or cut off (at most one unit in the last place,
2^-23 of the partial sum), is off by at most n 2^-23 times the sum of the
magnitudes; the rounding to the output type adds at most half a unit.
"""
import pytest
import torch

import sequence_head_relayout_gb300 as vf
from oracle import experts as X

from .test_gpu_expert import rounding, routing, within

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
CUT = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _lib():
    vf.lib()
    yield
    torch.cuda.synchronize()


def randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def rows_of(plan, M, dtype, seed):
    """Packed rows on the CPU, NaN where no slot goes."""
    x = randn((plan.slot_of.numel(), M), dtype, seed)
    x[plan.slot_of.cpu() < 0] = float("nan")
    return x


def weight_view(E, N, M, dtype, seed, layout):
    """(CPU values, a view of them on the GPU)."""
    w = randn((E, N, M), dtype, seed)
    if layout == "contiguous":
        v = torch.empty(E, N, M, dtype=dtype, device=DEV)
    elif layout == "transposed":
        v = torch.empty(E, M, N, dtype=dtype, device=DEV).transpose(1, 2)
    elif layout == "padded":                               # still 16-byte rows when M is
        v = torch.empty(E, N + 3, M + 8, dtype=dtype, device=DEV)[:, 2:2 + N, :M]
    elif layout == "odd":
        v = torch.empty(E, N, M + 1, dtype=dtype, device=DEV)[:, :, 1:]
    elif layout == "strided":
        v = torch.empty(E, N, 2 * M, dtype=dtype, device=DEV)[:, :, ::2]
    elif layout == "expert_last":
        v = torch.empty(N, M, E, dtype=dtype, device=DEV).permute(2, 0, 1)
    else:                                                  # one set of weights for all
        w = w[:1].expand(E, N, M)
        return w, w[:1].to(DEV).expand(E, N, M)
    v.copy_(w)
    return w, v


def check_product(plan, x, w_cpu, w, out=None):
    N, M = w.shape[1:]
    rows = x.shape[0]
    before = torch.full((rows, N), 3.0, dtype=x.dtype)
    if out is None:
        out = before.to(DEV)
    got = vf.expert_product(x.to(DEV), w, plan, out=out)
    assert got is out
    want, mag = X.product(x, w_cpu, plan.counts.cpu(), plan.offsets.cpu(), before)
    within(got, want, mag * (M * CUT) + rounding(want.abs() + mag * (M * CUT), x.dtype))
    used = int(plan.offsets[-1])
    assert torch.equal(got[used:].cpu(), before[used:])
    gap = plan.slot_of[:used].cpu() < 0
    assert (got[:used].cpu()[gap] == 0).all()
    return got


def check_weight_grad(plan, g, x, out_dtype):
    n = int(plan.counts.max()) if plan.counts.numel() else 0
    got = vf.expert_weight_grad(g.to(DEV), x.to(DEV), plan, dtype=out_dtype)
    assert got.dtype == out_dtype
    want, mag = X.weight_grad(g, x, plan.counts.cpu(), plan.offsets.cpu())
    err = mag * (max(n, 1) * CUT)
    within(got, want, err + rounding(want.abs() + err, out_dtype))
    return got


def make(T, K, E, align, how="mixed", seed=0):
    return vf.expert_plan(routing(T, K, E, seed + T, how).to(DEV), E, align=align)


SHAPES = [
    # T, K, E, align, N, M
    (1, 1, 1, 1, 1, 1), (1, 8, 16, 1, 128, 64), (1, 8, 16, 128, 256, 128), (3, 2, 4, 1, 8, 8),
    (16, 4, 8, 16, 136, 72), (33, 3, 7, 5, 65, 63), (40, 2, 3, 1, 127, 200),
    (64, 8, 5, 8, 264, 264), (100, 4, 130, 1, 72, 136), (257, 2, 3, 128, 384, 320),
    (300, 1, 2, 1, 129, 65), (700, 2, 3, 1, 256, 512), (1000, 2, 300, 4, 40, 96),
    (1500, 1, 1, 1, 520, 88), (5, 1, 4096, 1, 16, 24), (90, 2, 3, 1, 64, 320),
    (1600, 1, 2, 1, 128, 192), (2000, 1, 1, 8, 192, 328), (1, 2, 4, 1, 200, 4096),
    (20, 1, 2, 16, 130, 2500), (2, 1, 3, 1, 4096, 72), (60, 1, 2, 1, 513, 1030),
    (5000, 1, 1, 1, 72, 200), (6000, 1, 2, 8, 300, 130), (3000, 1, 3, 1, 256, 264),
    (14000, 1, 1, 1, 40, 100), (30000, 1, 2, 1, 130, 64), (9, 1, 2, 1, 1, 512),
    (9, 1, 2, 1, 512, 1), (50, 2, 4, 1, 24, 1000),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", SHAPES)
def test_product(shape, dtype):
    T, K, E, align, N, M = shape
    plan = make(T, K, E, align)
    w_cpu, w = weight_view(E, N, M, dtype, 1, "contiguous")
    check_product(plan, rows_of(plan, M, dtype, 2), w_cpu, w)


@pytest.mark.parametrize("shape", SHAPES)
def test_row_gradient(shape):
    """The same product with the weights' view transposed."""
    T, K, E, align, N, M = shape
    plan = make(T, K, E, align)
    w_cpu, w = weight_view(E, N, M, BF16, 1, "contiguous")
    check_product(plan, rows_of(plan, N, BF16, 2), w_cpu.transpose(1, 2), w.transpose(1, 2))


@pytest.mark.parametrize("out_dtype", [None, F32])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("shape", SHAPES)
def test_weight_grad(shape, dtype, out_dtype):
    T, K, E, align, N, M = shape
    plan = make(T, K, E, align)
    check_weight_grad(plan, rows_of(plan, N, dtype, 1), rows_of(plan, M, dtype, 2),
                      out_dtype or dtype)


@pytest.mark.parametrize("layout", ["transposed", "padded", "odd", "strided", "expert_last",
                                    "expanded"])
@pytest.mark.parametrize("T", [4, 90, 900])
def test_weight_layouts(layout, T):
    E, N, M = 3, 144, 72
    plan = make(T, 2, E, 1)
    x = rows_of(plan, M, BF16, 5)
    w_cpu, w = weight_view(E, N, M, BF16, 6, layout)
    check_product(plan, x, w_cpu, w)
    y = rows_of(plan, N, BF16, 7)
    check_product(plan, y, w_cpu.transpose(1, 2), w.transpose(1, 2))


@pytest.mark.parametrize("how", ["none", "one", "all"])
def test_skewed_routings(how):
    T, K, E = 300, 2, 9
    plan = make(T, K, E, 16, how)
    w_cpu, w = weight_view(E, 192, 128, BF16, 1, "contiguous")
    check_product(plan, rows_of(plan, 128, BF16, 2), w_cpu, w)
    got = check_weight_grad(plan, rows_of(plan, 192, BF16, 3), rows_of(plan, 128, BF16, 4), F32)
    assert (got[plan.counts.cpu() == 0] == 0).all()


def test_misaligned_buffers():
    """Buffers that start at any element: operands and outputs."""
    plan = make(200, 2, 3, 1)
    n, N, M = plan.slot_of.numel(), 96, 64
    x, g = rows_of(plan, M, BF16, 1), rows_of(plan, N, BF16, 2)
    w_cpu, w = weight_view(3, N, M, BF16, 3, "contiguous")
    for shift in (0, 1, 4):
        def at(t):
            flat = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)[shift:shift + t.numel()]
            return flat.view(t.shape).copy_(t)
        want, mag = X.product(x, w_cpu, plan.counts.cpu(), plan.offsets.cpu(), torch.zeros(n, N))
        got = vf.expert_product(at(x), at(w), plan, out=at(torch.zeros(n, N, dtype=BF16)))
        within(got, want, mag * (M * CUT) + rounding(want.abs() + mag * (M * CUT), BF16))
        for dtype in (BF16, F32):
            got = vf.expert_weight_grad(at(g), at(x), plan,
                                        out=at(torch.zeros(3, N, M, dtype=dtype)))
            want, mag = X.weight_grad(g, x, plan.counts.cpu(), plan.offsets.cpu())
            err = mag * (n * CUT)
            within(got, want, err + rounding(want.abs() + err, dtype))


def test_empty():
    plan = vf.expert_plan(torch.zeros((0, 2), dtype=torch.int64, device=DEV), 3)
    w = torch.ones((3, 8, 16), dtype=BF16, device=DEV)
    assert vf.expert_product(torch.empty((0, 16), dtype=BF16, device=DEV), w, plan).shape == (0, 8)
    got = vf.expert_weight_grad(torch.empty((0, 8), dtype=BF16, device=DEV),
                                torch.empty((0, 16), dtype=BF16, device=DEV), plan)
    assert got.shape == (3, 8, 16) and (got == 0).all()
    plan = make(10, 2, 3, 1, "all")
    rows = plan.slot_of.numel()
    none = torch.empty((rows, 0), dtype=BF16, device=DEV)
    got = vf.expert_product(none, w[:, :, :0], plan)         # sums of nothing
    assert got.shape == (rows, 8) and (got == 0).all()
    assert vf.expert_product(none, w[:, :0, :0], plan).shape == (rows, 0)
    assert vf.expert_weight_grad(none, none, plan).shape == (3, 0, 0)


def test_sums_that_tell():
    """Whole numbers whose sums are exact: every product in its place, bit for bit."""
    plan = make(500, 2, 5, 8)
    n, N, M = plan.slot_of.numel(), 264, 200
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-3, 4, (n, M), generator=g).to(BF16)
    w = torch.randint(-3, 4, (5, N, M), generator=g).to(BF16)
    y = torch.randint(-3, 4, (n, N), generator=g).to(BF16)
    x[plan.slot_of.cpu() < 0] = float("nan")
    y[plan.slot_of.cpu() < 0] = float("inf")
    want, _ = X.product(x, w, plan.counts.cpu(), plan.offsets.cpu(), torch.zeros(n, N))
    got = vf.expert_product(x.to(DEV), w.to(DEV), plan, out=torch.zeros(n, N, dtype=BF16,
                                                                        device=DEV))
    assert torch.equal(got.cpu(), want.to(BF16))
    want, _ = X.weight_grad(y, x, plan.counts.cpu(), plan.offsets.cpu())
    got = vf.expert_weight_grad(y.to(DEV), x.to(DEV), plan, dtype=F32)
    assert torch.equal(got.cpu(), want.float())


def test_infinities_and_nans_stay_in_their_rows():
    plan = make(64, 1, 2, 1, "all")
    n, N, M = plan.slot_of.numel(), 64, 64
    x, (w_cpu, w) = rows_of(plan, M, BF16, 1), weight_view(2, N, M, BF16, 2, "contiguous")
    x[3, 5], x[9, 0] = float("inf"), float("nan")
    got = check_product(plan, x, w_cpu, w)
    assert torch.isnan(got[9]).all() and not torch.isfinite(got[3]).any()
    assert torch.isfinite(got[4:9]).all()


def test_hostile_plans():
    """No content of a plan leads out of the buffers: guard bands stay."""
    E, N, M, rows = 6, 72, 40, 100
    x = randn((rows, M), BF16, 1).to(DEV)
    g = randn((rows, N), BF16, 2).to(DEV)
    w = randn((E, N, M), BF16, 3).to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    big = 2 ** 31 - 1
    for counts, offsets in [([big] * E, [0, 10, 20, 30, 40, 50, 60]),
                            ([5] * E, [-7, big, -big, 99, 100, 101, big]),
                            ([-1, 200, -big, 0, 3, 1], [0] * 7),
                            ([90, 90, 90, 90, 90, 90], [50] * 7)]:
        plan = vf.ExpertPlan(torch.zeros((rows, 1), **i32), torch.zeros((rows,), **i32),
                             torch.tensor(counts, **i32), torch.tensor(offsets, **i32), 4)
        band = torch.full((rows + 200, N), 7.0, dtype=BF16, device=DEV)
        vf.expert_product(x, w, plan, out=band[100:100 + rows])
        assert (band[:100] == 7).all() and (band[100 + rows:] == 7).all()
        band = torch.full((E + 2, N, M), 7.0, dtype=F32, device=DEV)
        vf.expert_weight_grad(g, x, plan, out=band[1:1 + E])
        assert (band[0] == 7).all() and (band[-1] == 7).all()


def test_equal_calls_give_equal_bits():
    plan = make(800, 2, 4, 1)
    x, g = rows_of(plan, 512, BF16, 1).to(DEV), rows_of(plan, 384, BF16, 2).to(DEV)
    w = randn((4, 384, 512), BF16, 3).to(DEV)
    used = int(plan.offsets[-1])
    first = vf.expert_product(x, w, plan)[:used].clone(), vf.expert_weight_grad(g, x, plan)
    for _ in range(3):
        assert torch.equal(vf.expert_product(x, w, plan)[:used], first[0])
        assert torch.equal(vf.expert_weight_grad(g, x, plan), first[1])


def test_refusals():
    plan = make(8, 2, 3, 1)
    n = plan.slot_of.numel()
    x = torch.zeros((n, 16), dtype=BF16, device=DEV)
    w = torch.zeros((3, 24, 16), dtype=BF16, device=DEV)
    g = torch.zeros((n, 24), dtype=BF16, device=DEV)
    for bad in [lambda: vf.expert_product(x.float(), w.float(), plan),
                lambda: vf.expert_product(x, w.half(), plan),
                lambda: vf.expert_product(x, w[:2], plan),
                lambda: vf.expert_product(x, w[:, :, :8], plan),
                lambda: vf.expert_product(x[:-1], w, plan),
                lambda: vf.expert_product(x[:, ::2], w[:, :, ::2], plan),
                lambda: vf.expert_product(x, w, plan, out=torch.zeros((n, 25), dtype=BF16,
                                                                      device=DEV)),
                lambda: vf.expert_product(x, w, plan, out=g.float()),
                lambda: vf.expert_product(x.cpu(), w, plan),
                lambda: vf.expert_product(x, w.cpu(), plan),
                lambda: vf.expert_product(x.cpu().pin_memory(), w, plan),
                lambda: vf.expert_product(x.clone().requires_grad_(), w, plan),
                lambda: vf.expert_product(x, w.clone().requires_grad_(), plan),
                lambda: vf.expert_weight_grad(g.half(), x, plan),
                lambda: vf.expert_weight_grad(g[:-1], x, plan),
                lambda: vf.expert_weight_grad(g, x, plan, dtype=F16),
                lambda: vf.expert_weight_grad(g, x, plan, out=torch.zeros((3, 24, 15), dtype=BF16,
                                                                          device=DEV))]:
        with pytest.raises((ValueError, TypeError)):
            bad()
    with pytest.raises(vf.VFError) as e:                     # a result over its operand
        vf.expert_product(x, w[:, :16], plan, out=x)
    assert e.value.status == -3
    with pytest.raises(vf.VFError) as e:
        pinned = vf.ExpertPlan(*(t.cpu().pin_memory() for t in plan[:4]))
        vf.expert_product(x, w, pinned)
    assert e.value.status == -1
