"""Pins of the expert relayouts' oracle: a routing worked by hand, identities
that hold whatever the layout, and the checkpoint's error bounds."""
import pytest
import torch

from oracle import experts as X
from oracle import loops

pytestmark = pytest.mark.usefixtures("oracle_built")


def test_plan_worked_by_hand():
    # tokens 0..3, two choices each, three experts; token 2 is padding and
    # token 3's second choice was dropped
    e = torch.tensor([[2, 0], [0, 2], [-1, -1], [2, 7]])
    row_of, slot_of, counts, offsets = X.plan(e, 3)
    assert counts.tolist() == [2, 0, 3]
    assert offsets.tolist() == [0, 2, 2, 5]
    assert row_of.tolist() == [[2, 0], [1, 3], [-1, -1], [4, -1]]
    assert slot_of.tolist() == [1, 2, 0, 3, 6, -1, -1, -1]
    row_of, slot_of, counts, offsets = X.plan(e, 3, align=4)
    assert offsets.tolist() == [0, 4, 4, 8]
    assert row_of.tolist() == [[4, 0], [1, 5], [-1, -1], [6, -1]]
    assert slot_of.tolist() == [1, 2, -1, -1, 0, 3, 6] + [-1] * 10    # 8 + 3 * 3 rows


def test_rows_worked_by_hand():
    e = torch.tensor([[1, 0], [1, -1]])
    row_of, slot_of, counts, offsets = X.plan(e, 2, align=2)
    x = torch.tensor([[1.0, 2.0, 3.0], [4.0, 5.0, 6.0]])
    before = torch.full((slot_of.numel(), 3), 9.0)
    p = X.pack(x, slot_of, offsets, 2, before)
    assert p.tolist() == [[1, 2, 3], [0, 0, 0], [1, 2, 3], [4, 5, 6], [9, 9, 9], [9, 9, 9]]
    y = torch.arange(18.0).view(6, 3)
    w = torch.tensor([[0.5, 2.0], [3.0, float("nan")]])
    out, mag = X.merge(y, row_of, w)
    # token 0: 0.5 * row 2 + 2 * row 0; token 1: 3 * row 3
    assert out.tolist() == [[3.0, 5.5, 8.0], [27.0, 30.0, 33.0]] and torch.equal(mag, out)
    gp, gw, _ = X.merge_backward(x, y, row_of, offsets, w, before)
    assert gp.tolist() == [[2, 4, 6], [0, 0, 0], [0.5, 1, 1.5], [12, 15, 18], [9, 9, 9],
                           [9, 9, 9]]
    # <x0, row 2> = 6 + 14 + 24, <x0, row 0> = 0 + 2 + 6, <x1, row 3> = 36 + 50 + 66
    assert gw.tolist() == [[44, 8], [152, 0]]


def test_adjoint_and_sorted_identities():
    g = torch.Generator().manual_seed(3)
    T, K, E, M = 37, 3, 5, 4
    e = torch.randint(-1, E + 1, (T, K), generator=g)
    row_of, slot_of, counts, offsets = X.plan(e, E, 3)
    # rows of an expert hold its slots in order, and nothing is lost
    for x in range(E):
        s = slot_of[offsets[x]:offsets[x] + counts[x]]
        assert (e.reshape(-1)[s.long()] == x).all() and (s[1:] > s[:-1]).all()
    assert int(counts.sum()) == int(((e >= 0) & (e < E)).sum())
    # <pack(x), y> = <x, merge(y)>: each is the other's adjoint
    x = torch.randn(T, M, generator=g, dtype=torch.float64)
    y = torch.randn(slot_of.numel(), M, generator=g, dtype=torch.float64)
    y[slot_of < 0] = 0
    p = X.pack(x, slot_of, offsets, K, torch.zeros_like(y))
    assert torch.allclose((p * y).sum(), (x * X.merge(y, row_of)[0]).sum(), rtol=1e-12)


@pytest.mark.parametrize("fmt", [loops.INT8, loops.E4M3])
def test_checkpoint_error_bounds(fmt):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(20, 300, generator=g).to(torch.bfloat16)
    codes, scales = X.checkpoint(x, fmt, 128)
    assert codes.shape == (20, 300) and scales.shape == (20, 3)
    v = X.values(codes, scales, fmt, 128)
    amax = torch.stack([x[:, c:c + 128].abs().amax(1).double() for c in (0, 128, 256)], 1)
    amax = amax.repeat_interleave(128, 1)[:, :300]
    # INT8: half a step of amax/127, E4M3: 2^-4 of the value and half a step of
    # 2^-9 * amax / 448 where it is subnormal; 2^-21 covers the float32 steps
    half = amax / 254 if fmt == loops.INT8 else x.double().abs() / 16 + amax / 448 / 1024
    assert ((v - x.double()).abs() <= half * (1 + 2.0 ** -12) + amax * 2.0 ** -21).all()
    # the restored rows are these values rounded to bfloat16
    r = X.restore(codes, scales, fmt, 128)
    assert torch.equal(r, v.float().to(torch.bfloat16))
