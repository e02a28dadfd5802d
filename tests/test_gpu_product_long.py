"""GPU tests of long sums in the experts' products: the forms of the weights' gradient
that take a sum in parts and those whose CTAs share one, segments of any length.

Whole numbers are compared bit for bit.  All operands are odd, so that no product is 0 and
a row that is left out or read twice changes every element of the result; all partial sums
stay below 2^24, so that float32 holds them exactly, whatever the order.
"""
import pytest
import torch

import sequence_head_relayout_gb300 as vf
from oracle import experts as X

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    vf.lib()
    yield
    torch.cuda.synchronize()


def plan_of(counts, align=1, seed=0):
    """A plan of one slot to a token with these counts, every 40th token's dropped."""
    e = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
    e = torch.cat([e, torch.full((len(e) // 40,), -1)])
    e = e[torch.randperm(len(e), generator=torch.Generator().manual_seed(seed))]
    plan = vf.expert_plan(e[:, None].to(DEV), len(counts), align=align)
    assert plan.counts.tolist() == list(counts)
    return plan


def odd(shape, dtype, seed, top=3):
    """Odd whole numbers from -top to top."""
    g = torch.Generator().manual_seed(seed)
    return (2 * torch.randint(0, top + 1, shape, generator=g) - top).to(dtype)


def odd_rows(plan, M, dtype, seed, top=3):
    x = odd((plan.slot_of.numel(), M), dtype, seed, top)
    x[plan.slot_of.cpu() < 0] = float("nan")
    return x


# The form that is chosen (by the tiles and the mean of the counts), counts, N, M, align
FORMS = [
    # pairs of CTAs; in float32 parts of 768 rows whose last has 1, 63, 64 and all rows
    ("pairs", [769, 2367, 832, 1536], 260, 1300, 1),
    ("pairs", [3000, 1, 0, 65], 392, 1288, 16),
    # single CTAs, tiles of 256 columns: nearly all rows at one expert of few on average
    ("single", [2400, 0, 1, 63, 64, 65, 100, 50], 260, 1300, 1),
    ("single", [0, 5, 2560, 90, 8, 0, 31, 32], 257, 1305, 8),
    # single CTAs, tiles of 128 columns
    ("few", [1601, 831], 130, 200, 1),
    ("few", [769, 2304, 0], 128, 192, 5),
    # two CTAs share a tile's rows, unevenly, or have none
    ("two", [4001, 2400], 130, 64, 1),
    ("two", [6208, 64], 72, 200, 4),
    # four CTAs do
    ("four", [14001, 12003], 130, 64, 1),
    ("four", [24000, 7], 72, 100, 128),
    ("four", [6200], 129, 257, 1),
    ("four", [0, 12500], 64, 128, 1),
]


def check_exact(counts, N, M, align, dtype, out_dtype):
    plan = plan_of(counts, align)
    g, x = odd_rows(plan, N, dtype, 1), odd_rows(plan, M, dtype, 2)
    want, mag = X.weight_grad(g, x, plan.counts.cpu(), plan.offsets.cpu())
    assert mag.max() < 2 ** 24
    assert want.abs().max() < torch.finfo(out_dtype).max
    got = vf.expert_weight_grad(g.to(DEV), x.to(DEV), plan, dtype=out_dtype)
    assert torch.equal(got.cpu(), want.to(out_dtype))


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, F32), (F16, F32), (BF16, BF16), (F16, F16)])
@pytest.mark.parametrize("form,counts,N,M,align", FORMS)
def test_weight_grad_of_whole_numbers(form, counts, N, M, align, dtype, out_dtype):
    check_exact(counts, N, M, align, dtype, out_dtype)


# Segments of one and of several parts of a 16-bit result (4,096 rows of fp16, 32,768 of
# bf16) that end 0, 1, 63 and 64 rows into one, in every form
LONG = [
    ("pairs", [4097, 33000, 20, 8255], 260, 1300, 1),
    ("single", [16449, 100, 2, 4160, 90, 4096] + [7] * 58, 64, 300, 8),
    ("few", [4160, 4097, 1], 257, 300, 1),
    ("two", [8321], 600, 1300, 4),
    ("four", [0, 32832, 20, 0, 300, 8193], 100, 100, 1),
    ("four", [140001], 72, 65, 1),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("form,counts,N,M,align", LONG)
def test_long_segments_of_whole_numbers(form, counts, N, M, align, dtype):
    check_exact(counts, N, M, align, dtype, dtype)


PART = {(F16, F16): 4096, (BF16, BF16): 32768, (F16, F32): 768}


def drift(n, part):
    """Bound of the relative error of a sum of n like terms of one sign in float32: those of
    a part are added by additions that round or cut off, term i at most one unit, 2^-23, of
    the i terms there are; the parts with rounding, half a unit each."""
    return (min(n, part) + 1) / 2 * 2.0 ** -23 + -(-n // part) * 2.0 ** -24


def half_units(want, dtype):
    """The relative error that one rounding may make."""
    exponent = torch.frexp(want).exponent.double() - 1
    return 2.0 ** exponent * torch.finfo(dtype).eps / 2 / want


@pytest.mark.parametrize("n,dtype,out_dtype", [(1 << 20, F16, F16), (60001, F16, F32)])
def test_weight_grad_does_not_drift(n, dtype, out_dtype):
    """What the additions cut off is always of one sign: with terms of one sign it adds up,
    but for the parts."""
    g = torch.Generator(device=DEV).manual_seed(1)
    a = (torch.rand((n, 72), generator=g, device=DEV) + 1).to(dtype)
    b = ((torch.rand((n, 64), generator=g, device=DEV) + 1) * 2.0 ** -8).to(dtype)
    plan = vf.expert_plan(torch.zeros((n, 1), dtype=torch.int64, device=DEV), 1)
    got = vf.expert_weight_grad(a, b, plan, dtype=out_dtype)[0].double()
    want = a.double().t() @ b.double()                     # float64: 2^-53 of n is nothing
    bound = drift(n, PART[dtype, out_dtype]) + half_units(want, out_dtype)
    assert ((got - want).abs() / want <= bound).all()


def test_operands_that_need_a_copy():
    """Odd features at any address: the same sums by way of the workspace."""
    plan = plan_of([2311, 1])
    g, x = odd_rows(plan, 131, BF16, 1), odd_rows(plan, 67, BF16, 2)
    want, _ = X.weight_grad(g, x, plan.counts.cpu(), plan.offsets.cpu())
    flat = torch.empty(g.numel() + 1, dtype=BF16, device=DEV)[1:].view(g.shape).copy_(g)
    assert torch.equal(vf.expert_weight_grad(flat, x.to(DEV), plan, dtype=F32).cpu(),
                       want.float())


# Rows of an expert, N, M, the weights' view transposed: forms of one CTA with tiles of 64
# and 128 rows, and of pairs with tiles of 128 and 256
PRODUCTS = [(20, 200, 4100, False), (20, 200, 4104, True), (90, 100, 2056, False),
            (90, 128, 2050, True), (100, 300, 4096, False), (100, 264, 4097, True),
            (300, 300, 2064, False), (300, 264, 2047, True)]


def check_product_exact(rows, N, M, transposed, dtype=F16, align=8):
    plan = plan_of([rows, 2 * rows, 1, 0], align)
    x = odd_rows(plan, M, dtype, 1)
    w = odd((4, M, N) if transposed else (4, N, M), dtype, 2)
    w_cpu, w = (w.transpose(1, 2), w.to(DEV).transpose(1, 2)) if transposed else (w, w.to(DEV))
    before = torch.full((x.shape[0], N), 3.0, dtype=dtype)
    want, mag = X.product(x, w_cpu, plan.counts.cpu(), plan.offsets.cpu(), before)
    assert mag[:int(plan.offsets[-1])].max() < 2 ** 24
    assert want.abs().max() < torch.finfo(dtype).max
    got = vf.expert_product(x.to(DEV), w, plan, out=before.to(DEV))
    assert torch.equal(got.cpu(), want.to(dtype))


@pytest.mark.parametrize("rows,N,M,transposed", PRODUCTS)
def test_product_of_whole_numbers(rows, N, M, transposed):
    check_product_exact(rows, N, M, transposed)


# Features of several parts (4,096 of fp16, 32,768 of bf16) that end 1 to 64 into one
@pytest.mark.parametrize("rows,N,M,transposed,dtype", [
    (20, 200, 8200, False, F16), (20, 136, 12289, True, F16), (90, 100, 8256, False, F16),
    (90, 128, 8192, True, F16), (100, 300, 8255, False, F16), (100, 264, 4160, True, F16),
    (300, 300, 12352, False, F16), (300, 264, 8193, True, F16),
    (20, 72, 32769, False, BF16), (20, 72, 65600, True, BF16), (100, 200, 32832, False, BF16),
    (300, 136, 33000, True, BF16)])
def test_product_of_many_whole_numbers(rows, N, M, transposed, dtype):
    check_product_exact(rows, N, M, transposed, dtype)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows", [6, 300])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_product_does_not_drift(rows, dtype, transposed):
    M, N = 1 << 20, 72
    g = torch.Generator(device=DEV).manual_seed(1)
    x = (torch.rand((rows, M), generator=g, device=DEV) + 1).to(dtype)
    w = torch.rand((1, M, N) if transposed else (1, N, M), generator=g, device=DEV)
    w = ((w + 1) * 2.0 ** -8).to(dtype)
    w = w.transpose(1, 2) if transposed else w
    plan = vf.expert_plan(torch.zeros((rows, 1), dtype=torch.int64, device=DEV), 1)
    got = vf.expert_product(x, w, plan).double()
    want = torch.zeros_like(got)
    for k in range(0, M, M // 8):
        mine = slice(k, k + M // 8)
        want += x[:, mine].double() @ w[0, :, mine].double().t()
    bound = drift(M, PART[dtype, dtype]) + half_units(want, dtype)
    assert ((got - want).abs() / want <= bound).all()


@pytest.mark.parametrize("M", [64, 8256])
def test_hostile_plans_of_many_rows(M):
    """Segments of several parts, cut to the buffer, and ends of experts far in front of
    them: guard bands stay."""
    E, N, rows = 4, 72, 9000
    i32 = dict(dtype=torch.int32, device=DEV)
    big = 2 ** 31 - 1
    x = odd((rows, M), F16, 1).to(DEV)
    w = odd((E, N, M), F16, 2).to(DEV)
    g = odd((rows, N), F16, 3).to(DEV)
    for counts, offsets in [([big] * E, [0, 10, 4100, 8999, 9000]),
                            ([9000, -1, 5000, 4097], [-5, big, 4500, 4903, big]),
                            ([8192, 8192, 1, big], [0, 808, 9000, 8999, -big])]:
        plan = vf.ExpertPlan(torch.zeros((rows, 1), **i32), torch.zeros((rows,), **i32),
                             torch.tensor(counts, **i32), torch.tensor(offsets, **i32), 4)
        band = torch.full((rows + 200, N), 7.0, dtype=F16, device=DEV)
        vf.expert_product(x, w, plan, out=band[100:100 + rows])
        assert (band[:100] == 7).all() and (band[100 + rows:] == 7).all()
        for cols in (64, 200):
            band = torch.full((E + 2, N, cols), 7.0, dtype=F16, device=DEV)
            few = x.repeat(1, 4)[:, :cols].contiguous()
            vf.expert_weight_grad(g, few, plan, out=band[1:1 + E])
            assert (band[0] == 7).all() and (band[-1] == 7).all()
            assert not (band[1:1 + E] == 7).all()
