"""GPU tests of calls that a layer's row-wise operators meet at their edges: single rows of
views, and gates so negative that their sigmoid leaves float32's normal range.
"""
import pytest
import torch

import sequence_head_relayout_gb300 as vf
from oracle import layer as L

from .test_gpu_expert import rounding, within

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    vf.lib()
    yield
    torch.cuda.synchronize()


def randn(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,pad", [(512, 1), (512, 2), (512, 4), (512, 0), (1024, 1), (1024, 2),
                                   (2048, 2), (3000, 1), (3000, 2), (3000, 6), (9001, 1)])
def test_a_row_by_itself(M, pad, dtype):
    """The first row of a view has the same bits with and without others behind it."""
    T = 48
    x, r, g = (randn((T, M + pad), dtype, i)[:, :M] for i in range(3))
    w = randn((M,), dtype, 4)
    for t in range(0, T, 3):
        one, two = slice(t, t + 1), slice(t, t + 2)
        pair = [vf.rms_norm(x[s], w, residual=r[s]) for s in (one, two)]
        assert torch.equal(pair[0][0][0], pair[1][0][0])
        assert torch.equal(vf.rms_norm(x[one], w)[0], vf.rms_norm(x[two], w)[0])
        pair = [vf.rms_norm_backward(g[s], x[s], w, grad_total=r[s])[0] for s in (one, two)]
        assert torch.equal(pair[0][0], pair[1][0])
        if dtype == BF16:
            pair = [vf.rms_norm_q(x[s], w) for s in (one, two)]
            assert torch.equal(pair[0][1][0], pair[1][1][0])       # the scales: float32


def test_a_row_without_a_stride():
    """Rows of size 1 keep whatever stride they got: [M, 1] transposed has stride 1."""
    M = 4096
    x, w = randn((M, 1), F32, 1), randn((M,), F32, 2)
    assert x.t().stride() == (1, 1)
    assert torch.equal(vf.rms_norm(x.t(), w), vf.rms_norm(x.t().contiguous(), w))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_glu_of_large_negative_gates(dtype):
    """s = exp(g) there, below float32's normal range, but what it is multiplied with can
    bring the results far above it.  The exponential is off by at most 2 + 1.173 |g| units
    of 2^-23 (CUDA's bound of its fast form, that of the full one is smaller), the quotient
    by 2.5, each product by half a unit; what is below 2^-126 is held to 2^-149: s, and
    g s."""
    g = torch.linspace(-103, -80, 500).to(dtype)[:, None]
    u = torch.full_like(g, 2.0 ** 100)
    d = torch.full_like(g, 2.0)
    plan = vf.expert_plan(torch.zeros((g.shape[0], 1), dtype=torch.int64, device=DEV), 1)

    def bound(want, units, factor):
        # (the units are of a value that may itself be below 2^-126)
        err = want.abs() * units * 2.0 ** -23 + factor * (g.double().abs() + 3) * 2.0 ** -149
        return want, err + rounding(want.abs() + err, dtype)

    units = 2 + 1.173 * g.double().abs() + 2.5
    want = L.glu(g, u)
    assert want.abs().max() > 2.0 ** -10
    within(vf.expert_glu(g.to(DEV), u.to(DEV), plan), *bound(want, units + 2, u.double()))
    dg, du = L.glu_backward(d, g, u)
    got = vf.expert_glu_backward(d.to(DEV), g.to(DEV), u.to(DEV), plan)
    # s (1 + g (1 - s)) d u: 1 - s is 1, the bracket rounds twice
    within(got[0], *bound(dg, units + 5, d.double() * u.double()))
    within(got[1], *bound(du, units + 2, d.double()))
