"""GPU tests of calls that a layer's row-wise operators meet at their edges: single rows of
views, and gates so negative that their sigmoid leaves float32's normal range.
"""
import pytest
import torch

import sequence_head_relayout_gb300 as vf

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
