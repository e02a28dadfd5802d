"""GPU tests of the gated activation and the root-mean-square norm against the CPU
oracle in float64.

Bounds, with u = 2^-24 (half a unit of float32) and the header's arithmetic:

* s = 1 / (1 + exp(-g)): the exponential is off by at most 2 + 1.173 |g| units of
  2^-23 (CUDA's bound of its fast form; 2 of the full one, which float32 takes),
  which moves 1 + exp(-g) by no more of itself; the sum rounds by u, half a unit,
  and the division by u (float32) or 2 units (CUDA's bound of the fast one), 2.5 units
  together; below 2^-126 it may be 0;
* a sum of M squares is off by at most M u of itself, its root and reciprocal by
  half of that and 4 u, each product by u;
* every result is rounded once to its type: half a unit.
"""
import pytest
import torch

import sequence_head_relayout_gb300 as vf
from oracle import experts as X
from oracle import layer as L
from oracle import loops

from .test_gpu_expert import FMT, LAYOUTS, rounding, routing, token_view, within
from .test_gpu_product import make, randn, rows_of

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("oracle_built")]

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    vf.lib()
    yield
    torch.cuda.synchronize()


def view_like(x, layout, pad=True):
    """The CPU rows x as a GPU view of the layout."""
    n, M = x.shape
    v = token_view(n, M, x.dtype, 0, layout)
    return v.copy_(x)


# ---- gated activation ----------------------------------------------------------------

def sigmoid_units(g, dtype):
    """Units of 2^-23 that s may be off by."""
    return 2 + 1 if dtype == F32 else 2 + 1.173 * g.double().abs() + 2.5


def limited(y, dtype):
    """What float64 values round to beyond the type's range: infinities, from half a
    unit over the largest value on."""
    info = torch.finfo(dtype)
    return torch.where(y.abs() > info.max * (1 + info.eps / 4), y * float("inf"), y)


def glu_bound(g, u, dtype):
    y = limited(L.glu(g, u), dtype)
    err = y.abs() * (sigmoid_units(g, dtype) + 2) * 2 * U
    err = err + (g.double() * u.double()).abs() * 2.0 ** -125
    return y, err + rounding(y.abs() + err, dtype)


def glu_backward_bounds(d, g, u, dtype):
    dg, du = (limited(t, dtype) for t in L.glu_backward(d, g, u))
    gd, s, k = g.double(), L.sigmoid(g.double()), sigmoid_units(g, dtype)
    dus = (d.double() * u.double()).abs()
    slope = (1 + gd.abs() * (1 - s)) * 4 + gd.abs() * (s * k + 2)
    e1 = dus * s * slope * 2 * U + dg.abs() * (k + 4) * 2 * U
    e1 = e1 + dus * (1 + gd.abs()) * 2.0 ** -125
    e2 = du.abs() * (k + 2) * 2 * U + (d.double() * gd).abs() * 2.0 ** -125
    return (dg, e1 + rounding(dg.abs() + e1, dtype)), (du, e2 + rounding(du.abs() + e2, dtype))


def masked(plan, want, bound, before):
    """The oracle's rows with zeros in the gaps and `before` behind the last expert."""
    slot, used = plan.slot_of.cpu(), int(plan.offsets[-1])
    want, bound = want.clone(), bound.clone()
    want[slot < 0], bound[slot < 0] = 0.0, 0.0
    want[used:] = before
    return want, bound


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 1), (1, 8, 16, 1, 64), (3, 2, 4, 16, 2047),
                                   (40, 2, 3, 5, 66), (64, 3, 9, 1, 520), (33, 2, 300, 8, 2048),
                                   (700, 2, 3, 128, 96), (5, 1, 2, 4, 9001)])
def test_glu(shape, dtype):
    T, K, E, align, F = shape
    plan = make(T, K, E, align)
    both = rows_of(plan, 2 * F, dtype, 1) * 4
    grad = rows_of(plan, F, dtype, 2)
    dev = both.to(DEV)
    gate, up = dev[:, :F], dev[:, F:]
    out = torch.full((both.shape[0], F), 3.0, dtype=dtype, device=DEV)
    assert vf.expert_glu(gate, up, plan, out=out) is out
    within(out, *masked(plan, *glu_bound(both[:, :F], both[:, F:], dtype), 3.0))
    buf = torch.full((both.shape[0], 2 * F), 3.0, dtype=dtype, device=DEV)
    dg, du = vf.expert_glu_backward(grad.to(DEV), gate, up, plan, grad_gate=buf[:, :F],
                                    grad_up=buf[:, F:])
    a, b = glu_backward_bounds(grad, both[:, :F], both[:, F:], dtype)
    within(dg, *masked(plan, *a, 3.0))
    within(du, *masked(plan, *b, 3.0))
    fresh = vf.expert_glu_backward(grad.to(DEV), gate, up, plan)
    used = int(plan.offsets[-1])
    assert torch.equal(fresh[0][:used], dg[:used]) and torch.equal(fresh[1][:used], du[:used])
    assert fresh[1].data_ptr() - fresh[0].data_ptr() == F * fresh[0].element_size()
    assert fresh[0].stride() == (2 * F, 1)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("F", [64, 33])
def test_glu_layouts(layout, F):
    plan = make(30, 2, 3, 4)
    g, u, d = (rows_of(plan, F, BF16, i) for i in range(3))
    gv, uv, dv = (view_like(t, layout) for t in (g, u, d))
    out = view_like(torch.full_like(g, 3.0), layout)
    vf.expert_glu(gv, uv, plan, out=out)
    within(out, *masked(plan, *glu_bound(g, u, BF16), 3.0))
    outs = [view_like(torch.full_like(g, 3.0), layout) for _ in range(2)]
    vf.expert_glu_backward(dv, gv, uv, plan, grad_gate=outs[0], grad_up=outs[1])
    for got, want in zip(outs, glu_backward_bounds(d, g, u, BF16)):
        within(got, *masked(plan, *want, 3.0))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_glu_range(dtype):
    """Gates from where s is 0 to where it is 1, the type's largest and smallest."""
    info = torch.finfo(dtype)
    g = torch.cat([torch.linspace(-120, 120, 4001), torch.tensor([
        info.max, -info.max, info.tiny, -info.tiny, 0.0, -0.0, 1e-30, -88.5, -87.2, 89.0])])
    g = g.to(dtype)[:, None]
    n = g.shape[0]
    plan = vf.expert_plan(torch.zeros((n, 1), dtype=torch.int64, device=DEV), 1)
    u, d = torch.full_like(g, 0.5), torch.full_like(g, 2.0)
    got = vf.expert_glu(g.to(DEV), u.to(DEV), plan)
    within(got, *glu_bound(g, u, dtype))
    for got, want in zip(vf.expert_glu_backward(d.to(DEV), g.to(DEV), u.to(DEV), plan),
                         glu_backward_bounds(d, g, u, dtype)):
        within(got, *want)
    x = torch.tensor([float("nan"), float("inf")], dtype=dtype)[:, None].to(DEV)
    two = vf.expert_plan(torch.zeros((2, 1), dtype=torch.int64, device=DEV), 1)
    got = vf.expert_glu(x, torch.ones_like(x), two).cpu()
    assert torch.isnan(got[0]).all() and torch.isposinf(got[1]).all()


def test_glu_differences():
    """The gradients against central differences of the oracle's activation."""
    plan = make(20, 1, 2, 1, "all")
    g, u, d = (rows_of(plan, 40, F32, i) for i in range(3))
    dg, du = vf.expert_glu_backward(d.to(DEV), g.to(DEV), u.to(DEV), plan)
    h = 1e-5
    for got, f in ((dg, lambda e: L.glu(g.double() + e, u)),
                   (du, lambda e: L.glu(g, u.double() + e))):
        want = d.double() * (f(h) - f(-h)) / (2 * h)
        # h^2 / 6 times the third derivative, at most 1 here, and float64's 2^-52 / h
        assert (got.cpu().double() - want).abs().max() < 1e-5


def test_glu_hostile_plan():
    rows, F = 50, 24
    i32 = dict(dtype=torch.int32, device=DEV)
    x = randn((rows, F), BF16, 1).to(DEV)
    for last in (-5, 2 ** 31 - 1, 51):
        plan = vf.ExpertPlan(torch.zeros((rows, 1), **i32),
                             torch.full((rows,), 2 ** 31 - 1, **i32), torch.zeros((2,), **i32),
                             torch.tensor([0, 0, last], **i32))
        band = torch.full((rows + 20, F), 7.0, dtype=BF16, device=DEV)
        vf.expert_glu(x, x, plan, out=band[10:10 + rows])
        assert (band[:10] == 7).all() and (band[10 + rows:] == 7).all()
        assert (last > 0) == bool((band[10:10 + rows] != 7).any())


# ---- norm ------------------------------------------------------------------------------

def norm_bound(h, w, eps, dtype):
    y = L.norm(h, w, eps)
    err = y.abs() * (h.shape[1] / 2 + 8) * U
    return y, err + rounding(y.abs() + err, dtype)


def check_norm(x, w, eps=1e-6, residual=None, xv=None, rv=None, out=None, total=None):
    dtype = x.dtype
    xv = x.to(DEV) if xv is None else xv
    if residual is None:
        got = vf.rms_norm(xv, w.to(DEV), eps, out=out)
        h = x
    else:
        rv = residual.to(DEV) if rv is None else rv
        got, sums = vf.rms_norm(xv, w.to(DEV), eps, residual=rv, out=out, total=total)
        h = L.total(x, residual)
        assert torch.equal(sums.cpu(), h)
    within(got, *norm_bound(h, w, eps, dtype))


SIZES = [(1, 1), (1, 4096), (2, 8), (3, 63), (5, 2047), (7, 64), (9, 264), (33, 1000), (40, 2048),
         (700, 96), (3, 5001), (2, 20000), (2, 40000), (1, 70001), (640, 520), (641, 3584)]


@pytest.mark.parametrize("weight", ["same", "fp32"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,M", SIZES)
def test_norm(T, M, dtype, weight):
    x, r = randn((T, M), dtype, 1) * 3, randn((T, M), dtype, 2)
    w = randn((M,), F32 if weight == "fp32" else dtype, 3)
    check_norm(x, w)
    check_norm(x, w, residual=r)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("M", [64, 33, 264])
def test_norm_layouts(layout, M):
    x, r, w = randn((37, M), BF16, 1), randn((37, M), BF16, 2), randn((M,), BF16, 3)
    xv, rv = view_like(x, layout), view_like(r, layout)
    outs = [view_like(torch.zeros_like(x), layout) for _ in range(2)]
    check_norm(x, w, xv=xv, out=outs[0])
    check_norm(x, w, residual=r, xv=xv, rv=rv, out=outs[0], total=outs[1])
    # views of different kinds in one call, and rows that repeat
    check_norm(x, w, residual=r, xv=xv, rv=r.to(DEV))
    check_norm(x[:1].expand(37, M), w, xv=xv[:1].expand(37, M))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_norm_special_rows(dtype):
    """Zeros (eps alone below the root), one huge element, NaN and infinities: each
    row by itself."""
    M = 128
    x = randn((6, M), dtype, 1)
    x[1] = 0
    x[2], x[2, 7] = 0, 100.0
    x[3, 5], x[4, 6] = float("nan"), float("inf")
    w = torch.ones(M, dtype=dtype)
    got = vf.rms_norm(x.to(DEV), w.to(DEV), 1e-5).cpu()
    want, bound = norm_bound(x, w, 1e-5, dtype)
    for t in (0, 1, 2, 5):
        within(got[t], want[t], bound[t])
    assert torch.isnan(got[3]).all()
    # 1 / inf is 0: the infinite element is 0 * inf, the others 0
    assert torch.isnan(got[4, 6]) and (got[4, :6] == 0).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("T,M", [(1, 1), (2, 33), (3, 256), (5, 264), (1, 4096), (40, 1000),
                                 (641, 3584), (3, 20000), (2, 40000), (7, 1001), (700, 1420),
                                 (9, 36)])
def test_norm_q(T, M, group, fmt):
    x, r = randn((T, M), BF16, 1) * 3, randn((T, M), BF16, 2)
    w = randn((M,), BF16, 3)
    codes, scales, total = vf.rms_norm_q(x.to(DEV), w.to(DEV), 1e-6, fmt, group,
                                         residual=r.to(DEV))
    h = L.total(x, r)
    assert torch.equal(total.cpu(), h)
    y = L.norm(h, w, 1e-6)
    rel = (M / 2 + 8) * U                          # of the float32 values
    top = 127.0 if fmt == "int8" else 448.0
    groups = -(-M // group)
    wide = torch.zeros((T, groups * group), dtype=torch.float64)
    wide[:, :M] = y
    amax = wide.view(T, groups, group).abs().amax(dim=2)
    assert scales.shape == (T, groups)
    assert ((scales.cpu().double() - amax / top).abs() <= amax / top * (rel + U)).all()
    q = y * (top / amax).repeat_interleave(group, dim=1)[:, :M]
    got = X.values(codes.cpu().view(torch.int8 if fmt == "int8" else torch.uint8),
                   torch.ones_like(scales.cpu()), FMT[fmt], group)
    off = q.abs() * (2 * rel + 2 * U)              # y, amax, the quotient and the product
    half = 0.5 if fmt == "int8" else torch.maximum(q.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10))
    assert ((got - q).abs() <= half + off * 1.07).all()
    again = vf.rms_norm_q(x.to(DEV), w.to(DEV), 1e-6, fmt, group, residual=r.to(DEV))
    assert all(torch.equal(a, b) for a, b in zip(again, (codes, scales, total)))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("M,pad", [(256, 0), (512, 8), (256, 1), (64, 0)])
def test_norm_q_bits(M, pad, fmt):
    """Rows of +-2 have an exact root, so that the values are the weight's and the
    codes and scales those of the transport's oracle, lost groups included."""
    T = 50
    sign = torch.randint(0, 2, (T, M), generator=torch.Generator().manual_seed(1)) * 4.0 - 2.0
    w = randn((M,), BF16, 2)
    w[3] = 2.0 ** -110
    w[32:64] = 2.0 ** -100                         # a group below the format's floor
    x = torch.empty((T, M + pad), dtype=BF16, device=DEV)[:, pad:].copy_(sign)
    y = (sign / 2).to(BF16) * w
    for group in (32, 64):
        codes, scales = vf.rms_norm_q(x, w.to(DEV), 0.0, fmt, group)
        wc, ws = X.checkpoint(y, FMT[fmt], group)
        assert torch.equal(codes.cpu().view(torch.uint8), wc.view(torch.uint8))
        assert torch.equal(scales.cpu(), ws)
    w[40], w[1] = float("inf"), float("nan")
    codes, scales = vf.rms_norm_q(x, w.to(DEV), 0.0, fmt, 32)
    assert torch.isnan(scales[:, :2]).all() and torch.isfinite(scales[:, 2:]).all()
    assert (codes[:, :64].view(torch.uint8) == 0).all()


def backward_check(x, g, w, more=None, eps=1e-6, views=None):
    T, M = x.shape
    xv, gv, mv = views or (x.to(DEV), g.to(DEV), None if more is None else more.to(DEV))
    dx, dw = vf.rms_norm_backward(gv, xv, w.to(DEV), eps, grad_total=mv)
    want, want_w, mag, mag_w = L.norm_backward(g, x, w, eps, more)
    err = mag * (2 * M + 20) * U
    within(dx, want, err + rounding(want.abs() + err, x.dtype))
    assert dw.dtype == F32
    within(dw, want_w, mag_w * (T + M / 2 + 16) * U + 2.0 ** -149)
    return dx, dw


@pytest.mark.parametrize("weight", ["same", "fp32"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,M", SIZES + [(1300, 40)])
def test_norm_backward(T, M, dtype, weight):
    x, g, m = randn((T, M), dtype, 1) * 3, randn((T, M), dtype, 2), randn((T, M), dtype, 4)
    w = randn((M,), F32 if weight == "fp32" else dtype, 3)
    first = backward_check(x, g, w)
    again = vf.rms_norm_backward(g.to(DEV), x.to(DEV), w.to(DEV))
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    backward_check(x, g, w, more=m)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("M", [64, 33])
def test_norm_backward_layouts(layout, M):
    x, g, m = (randn((37, M), BF16, i) for i in range(3))
    w = randn((M,), BF16, 3)
    backward_check(x, g, w, more=m, views=tuple(view_like(t, layout) for t in (x, g, m)))


def check_codes(codes, scales, y, fmt, group):
    """Against the float64 values y, with the bounds of test_norm_q."""
    T, M = y.shape
    rel, groups = (M / 2 + 8) * U, -(-M // group)
    top = 127.0 if fmt == "int8" else 448.0
    wide = torch.zeros((T, groups * group), dtype=torch.float64)
    wide[:, :M] = y
    amax = wide.view(T, groups, group).abs().amax(dim=2)
    assert ((scales.cpu().double() - amax / top).abs() <= amax / top * (rel + U)).all()
    q = y * (top / amax).repeat_interleave(group, dim=1)[:, :M]
    got = X.values(codes.cpu().view(torch.int8 if fmt == "int8" else torch.uint8),
                   torch.ones_like(scales.cpu()), FMT[fmt], group)
    off = q.abs() * (2 * rel + 2 * U)              # y, amax, the quotient and the product
    half = 0.5 if fmt == "int8" else torch.maximum(q.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10))
    assert ((got - q).abs() <= half + off * 1.07).all()


class Placed:
    """Rows at any address: the values in a buffer that holds `fill` around them, `base`
    elements behind an aligned address, rows `pitch` apart."""

    def __init__(self, x, base, pitch, fill):
        T, M = x.shape
        self.at = base + (torch.arange(T) * pitch)[:, None] + torch.arange(M)
        self.flat = torch.full((base + T * pitch + 40,), fill, dtype=x.dtype, device=DEV)
        self.view = self.flat.as_strided((T, M), (pitch, 1), base).copy_(x)
        self.fill = fill

    def untouched(self):
        flat = self.flat.cpu()
        flat[self.at.reshape(-1)] = self.fill
        return torch.equal(flat, torch.full_like(flat, self.fill))


# (T, M, base, pitch - M): odd lengths, rows that start anywhere, one to many warps to a
# row, rows of one element and a few, several rounds of a block, the longest in registers
# and longer ones; the last have one more unit than a multiple of 64
PLACES = [(5, 1, 0, 0), (9, 3, 0, 0), (7, 3, 5, 4), (33, 7, 0, 0), (40, 9, 1, 2),
          (20, 33, 0, 0), (21, 97, 3, 1), (17, 255, 0, 0), (11, 257, 7, 0), (9, 777, 0, 0),
          (8, 1421, 0, 2), (2600, 101, 0, 0), (10001, 37, 0, 0), (5003, 21, 3, 2),
          (3, 2047, 0, 0), (2, 2047, 2, 3), (1, 4095, 3, 0), (2, 8191, 0, 0), (2, 9001, 1, 0),
          (1, 32761, 0, 0), (2, 32763, 0, 0), (19, 510, 0, 1), (14, 1022, 4, 5),
          (9, 513, 0, 0), (9, 1031, 2, 1)]


@pytest.mark.parametrize("weight", ["same", "fp32"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,M,base,gap", PLACES)
def test_norm_at_any_address(T, M, base, gap, dtype, weight):
    """What lies around the rows is neither read into a result nor written."""
    x, r, g, m = (randn((T, M), dtype, i) for i in range(4))
    w = randn((M,), F32 if weight == "fp32" else dtype, 5)
    nan, pitch = float("nan"), M + gap
    place = [Placed(t, base, pitch, nan) for t in (x, r, g, m)]
    zero = torch.zeros_like(x)
    outs = [Placed(zero, base, pitch, 7.0) for _ in range(3)]
    out, total, dx = (o.view for o in outs)
    xv, rv, gv, mv = (p.view for p in place)
    # a residual at an address of its own too
    for other in (rv, Placed(r, base + 1, pitch + 2, nan).view):
        check_norm(x, w, residual=r, xv=xv, rv=other, out=out, total=total)
    check_norm(x, w, xv=xv, out=out)
    want, want_w, mag, mag_w = L.norm_backward(g, x, w, 1e-6, m)
    err = mag * (2 * M + 20) * U
    for first in (True, False):
        got, dw = vf.rms_norm_backward(gv, xv, w.to(DEV), grad_total=mv, grad_x=dx)
        within(got, want, err + rounding(want.abs() + err, dtype))
        within(dw, want_w, mag_w * (T + M / 2 + 16) * U + 2.0 ** -149)
        if first:
            kept = got.clone(), dw
    assert torch.equal(got, kept[0]) and torch.equal(dw, kept[1])
    want, want_w, mag, mag_w = L.norm_backward(g, x, w, 1e-6)
    err = mag * (2 * M + 20) * U
    got, dw = vf.rms_norm_backward(gv, xv, w.to(DEV), grad_x=dx)
    within(got, want, err + rounding(want.abs() + err, dtype))
    within(dw, want_w, mag_w * (T + M / 2 + 16) * U + 2.0 ** -149)
    assert all(o.untouched() for o in outs)
    # a weight that starts anywhere
    w1 = torch.full((M + 1,), nan, dtype=w.dtype, device=DEV)[1:].copy_(w)
    a, b = vf.rms_norm(xv, w1), vf.rms_norm(x.to(DEV), w.to(DEV))
    bound = norm_bound(x, w, 1e-6, dtype)[1]
    assert ((a - b).cpu().double().abs() <= 2 * bound).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("F,base,gap,align", [(191, 0, 0, 1), (193, 0, 0, 8), (255, 1, 0, 1),
                                              (257, 3, 2, 5), (513, 0, 1, 1), (1421, 5, 0, 4),
                                              (2047, 0, 0, 1), (2049, 2, 3, 1), (8191, 7, 1, 1)])
def test_glu_at_any_address(F, base, gap, align, dtype):
    """What lies around the rows is neither read into a result nor written."""
    plan = make(23, 2, 5, align)
    g, u, d = (rows_of(plan, F, dtype, i) for i in range(3))
    nan = float("nan")
    gp, up, dp = (Placed(t, base + i, F + gap + i, nan) for i, t in enumerate((g, u, d)))
    outs = [Placed(torch.full_like(g, 3.0), base + 2 * i, F + gap + 1, 7.0) for i in range(3)]
    out, dg, du = (o.view for o in outs)
    bounds = glu_backward_bounds(d, g, u, dtype)
    vf.expert_glu(gp.view, up.view, plan, out=out)
    within(out, *masked(plan, *glu_bound(g, u, dtype), 3.0))
    vf.expert_glu_backward(dp.view, gp.view, up.view, plan, grad_gate=dg, grad_up=du)
    for got, want in zip((dg, du), bounds):
        within(got, *masked(plan, *want, 3.0))
    assert all(o.untouched() for o in outs)
    # the halves of one buffer, and a gate whose rows repeat
    both = Placed(torch.full((g.shape[0], 2 * F), 3.0, dtype=dtype), base, 2 * F + gap, 7.0)
    vf.expert_glu_backward(dp.view, gp.view, up.view, plan, grad_gate=both.view[:, :F],
                           grad_up=both.view[:, F:])
    for got, want in zip((both.view[:, :F], both.view[:, F:]), bounds):
        within(got, *masked(plan, *want, 3.0))
    assert both.untouched()
    first = int((plan.slot_of >= 0).int().argmax())
    one = g[first:first + 1].expand_as(g)
    got = vf.expert_glu(gp.view[first:first + 1].expand_as(g), up.view, plan, out=out)
    within(got, *masked(plan, *glu_bound(one, u, dtype), 3.0))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_at_any_address_special_rows(dtype):
    """A row of NaN or infinities stays by itself where rows share their pieces."""
    for M in (97, 1421):
        x, w = randn((9, M), dtype, 1), randn((M,), dtype, 2)
        x[2], x[5], x[7] = float("nan"), float("inf"), 0.0
        clean = [0, 1, 3, 4, 6, 7, 8]
        out = vf.rms_norm(x.to(DEV), w.to(DEV), 1e-5).cpu()
        want, bound = norm_bound(x, w, 1e-5, dtype)
        within(out[clean], want[clean], bound[clean])
        assert torch.isnan(out[2]).all() and torch.isnan(out[5]).all()
        g = randn((9, M), dtype, 3)
        dx = vf.rms_norm_backward(g.to(DEV), x.to(DEV), w.to(DEV), 1e-5)[0].cpu()
        want, _, mag, _ = L.norm_backward(g, x, w, 1e-5)
        err = mag * (2 * M + 20) * U
        within(dx[clean], want[clean], (err + rounding(want.abs() + err, dtype))[clean])
        assert torch.isnan(dx[2]).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("T,M,base,gap", PLACES)
def test_norm_q_at_any_address(T, M, base, gap, fmt):
    """Codes, scales and totals, wherever the rows and the codes lie."""
    x, r, w = randn((T, M), BF16, 1) * 3, randn((T, M), BF16, 2), randn((M,), BF16, 3)
    nan, pitch = float("nan"), M + gap
    px, pr = Placed(x, base, pitch, nan), Placed(r, base + 1, pitch + 1, nan)
    total = Placed(torch.zeros_like(x), base + 2, pitch + 1, 7.0)
    h = L.total(x, r)
    for group, off in ((32, 0), (256, 0), (64, 1), (128, 6)):
        flat = torch.full((off + T * M + 20,), 3, dtype=torch.int8, device=DEV)
        codes = flat[off:off + T * M].view(T, M)
        if fmt == "e4m3":
            codes = codes.view(torch.float8_e4m3fn)
        _, scales = vf.rms_norm_q(px.view, w.to(DEV), 1e-6, fmt, group, codes=codes)
        check_codes(codes, scales, L.norm(x, w, 1e-6), fmt, group)
        vf.rms_norm_q(px.view, w.to(DEV), 1e-6, fmt, group, residual=pr.view, codes=codes,
                      scales=scales, total=total.view)
        check_codes(codes, scales, L.norm(h, w, 1e-6), fmt, group)
        assert torch.equal(total.view.cpu(), h) and total.untouched()
        assert (flat[:off] == 3).all() and (flat[off + T * M:] == 3).all()


def test_norm_differences():
    x, g, w = (randn(s, F32, i) for i, s in enumerate([(4, 48), (4, 48), (48,)]))
    dx, dw = vf.rms_norm_backward(g.to(DEV), x.to(DEV), w.to(DEV), 1e-3)
    h = 1e-5

    def f(x, w):
        return (L.norm(x, w, 1e-3) * g.double()).sum()
    for got, t, call in ((dx, x.double(), lambda t: f(t, w)), (dw, w.double(), lambda t: f(x, t))):
        want = torch.empty(t.numel(), dtype=torch.float64)
        for i in range(t.numel()):
            e = torch.zeros(t.numel(), dtype=torch.float64)
            e[i] = h
            want[i] = (call(t + e.view(t.shape)) - call(t - e.view(t.shape))) / (2 * h)
        # float32's error of sums of some 48 terms of size 1; the difference's is 1e-9
        assert (got.cpu().double().reshape(-1) - want).abs().max() < 48 * 2.0 ** -19


def test_no_rows():
    w = torch.ones(16, dtype=BF16, device=DEV)
    x = torch.empty((0, 16), dtype=BF16, device=DEV)
    assert vf.rms_norm(x, w).shape == (0, 16)
    assert [t.shape for t in vf.rms_norm(x, w, residual=x)] == [(0, 16)] * 2
    assert vf.rms_norm_q(x, w)[1].shape == (0, 1)
    dx, dw = vf.rms_norm_backward(x, x, w, grad_weight=torch.ones(16, device=DEV))
    assert dx.shape == (0, 16) and (dw == 0).all()
    none = torch.empty((5, 0), dtype=BF16, device=DEV)
    assert vf.rms_norm(none, w[:0]).shape == (5, 0)
    assert vf.rms_norm_backward(none, none, w[:0])[1].shape == (0,)
    plan = vf.expert_plan(torch.zeros((0, 2), dtype=torch.int64, device=DEV), 3)
    assert vf.expert_glu(x, x, plan).shape == (0, 16)


def test_layer_refusals():
    plan = make(8, 2, 3, 1)
    n = plan.slot_of.numel()
    x, w = torch.ones((8, 16), dtype=BF16, device=DEV), torch.ones(16, dtype=BF16, device=DEV)
    g = torch.ones((n, 16), dtype=BF16, device=DEV)
    for bad in [lambda: vf.rms_norm(x, w[:8]), lambda: vf.rms_norm(x, w.half()),
                lambda: vf.rms_norm(x[0], w), lambda: vf.rms_norm(x.int(), w),
                lambda: vf.rms_norm(x, w, residual=x[:4]), lambda: vf.rms_norm(x, w, total=x),
                lambda: vf.rms_norm(x, w, residual=x.float()), lambda: vf.rms_norm(x.cpu(), w),
                lambda: vf.rms_norm(x, w, out=g), lambda: vf.rms_norm(x, w.repeat(2)[::2]),
                lambda: vf.rms_norm(x.clone().requires_grad_(), w),
                lambda: vf.rms_norm(x, w.clone().requires_grad_()),
                lambda: vf.rms_norm(x, w, residual=x.clone().requires_grad_()),
                lambda: vf.rms_norm_q(x.half(), w.half()), lambda: vf.rms_norm_q(x, w, group=48),
                lambda: vf.rms_norm_q(x, w, fmt="e5m2"),
                lambda: vf.rms_norm_q(x.clone().requires_grad_(), w),
                lambda: vf.rms_norm_backward(x[:4], x, w),
                lambda: vf.rms_norm_backward(x, x, w, grad_total=x.float()),
                lambda: vf.rms_norm_backward(x, x, w, grad_weight=w),
                lambda: vf.expert_glu(g, g[:, :8], plan), lambda: vf.expert_glu(x, x, plan),
                lambda: vf.expert_glu(g, g.float(), plan), lambda: vf.expert_glu(g, g.cpu(), plan),
                lambda: vf.expert_glu(g, g, plan, out=x),
                lambda: vf.expert_glu(g.clone().requires_grad_(), g, plan),
                lambda: vf.expert_glu(g, g.clone().requires_grad_(), plan),
                lambda: vf.expert_glu_backward(x, g, g, plan)]:
        with pytest.raises((ValueError, TypeError)):
            bad()
    both = torch.ones((n, 24), dtype=BF16, device=DEV)
    for status, bad in [(-3, lambda: vf.rms_norm(x, w, out=x)),
                        (-3, lambda: vf.rms_norm(x, w, residual=w.expand(8, 16), total=x)),
                        (-1, lambda: vf.rms_norm(x, w, out=w.expand(8, 16))),
                        (-1, lambda: vf.rms_norm(x, w, eps=-1.0)),
                        (-1, lambda: vf.rms_norm(x, w, eps=float("nan"))),
                        (-3, lambda: vf.expert_glu(g, g, plan, out=g)),
                        (-3, lambda: vf.expert_glu_backward(g, g, g, plan,
                                                            grad_gate=both[:, :16],
                                                            grad_up=both[:, 8:])),
                        (-3, lambda: vf.expert_glu_backward(g, both[:, :16], g, plan,
                                                            grad_gate=both[:, :16])),
                        (-1, lambda: vf.expert_glu(g, g, plan, out=w.expand(n, 16)))]:
        with pytest.raises(vf.VFError) as e:
            bad()
        assert e.value.status == status
