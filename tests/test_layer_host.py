"""Host side of the experts' products, the gated activation and the norm without a
GPU: descriptors, workspace sizes, and every argument refused before the library
touches CUDA.  Fake pointer values are safe: nothing is dereferenced or launched; a
call that passes every host check reaches the CUDA pointer query, which fails here
with VF_ERR_CUDA."""
import os
import subprocess

import pytest
import torch

import sequence_head_relayout_gb300 as vf

OK, ARG, OVERFLOW, ALIAS, CUDA, CAPACITY = 0, -1, -2, -3, -4, -5
PASSES = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers pass the checks")
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L(lib_built):
    return vf.lib()


def address(i):
    return (i + 1) << 40


PRODUCT = dict(type=0, out_type=0, E=4, N=24, M=16, rows=8, slots=8, align=1,
               counts=address(0), offsets=address(1), packed=address(2), weights=address(3),
               s0=24 * 16, s1=16, s2=1, grad=address(4), out=address(5), grad_weights=address(6),
               workspace=0)
GLU = dict(type=0, E=4, rows=8, F=16, slot_of=address(0), offsets=address(1),
           gate=address(2), gate0=32, gate1=1, up=address(2) + 32, up0=32, up1=1,
           out=address(3), out0=16, out1=1, grad=address(4), grad0=16, grad1=1,
           grad_gate=address(5), gg0=32, gg1=1, grad_up=address(5) + 32, gu0=32, gu1=1)
NORM = dict(type=0, weight_type=0, format=0, eps=1e-6, T=8, M=64, group=64,
            x=address(0), x0=64, x1=1, weight=address(1), residual=0, r0=64, r1=1,
            total=address(2), t0=64, t1=1, out=address(3), o0=64, o1=1, codes=address(4),
            scales=address(5), grad=address(6), g0=64, g1=1, grad_total=0, m0=64, m1=1,
            grad_x=address(7), d0=64, d1=1, grad_weight=address(8), workspace=address(9))
STRUCTS = {"product": (vf._PRODUCT_DESC, PRODUCT), "glu": (vf._GLU_DESC, GLU),
           "norm": (vf._NORM_DESC, NORM)}


def desc(which, **kw):
    packed, fields = STRUCTS[which]
    assert set(kw) <= set(fields)
    values = list({**fields, **kw}.values())
    if which == "product":
        return packed.pack(*values[:-1]) + vf._POINTER.pack(values[-1])
    return packed.pack(*values)


def call(L, fn, **kw):
    which = "product" if "product" in fn or "weight_grad" in fn else \
        "glu" if "glu" in fn else "norm"
    return getattr(L, fn)(desc(which, **kw), None)


def test_descriptors_have_the_sizes_of_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include "vf_relayout.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu '
                   '%zu", sizeof(vf_product_desc), sizeof(vf_glu_desc), sizeof(vf_norm_desc)); }')
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), "-o", exe, str(src)], check=True)
    sizes = [int(n) for n in subprocess.run([exe], capture_output=True, check=True).stdout.split()]
    assert sizes == [len(desc(n)) for n in ("product", "glu", "norm")]


PRODUCTS = ("vf_expert_product", "vf_expert_weight_grad")


@pytest.mark.parametrize("fn", PRODUCTS)
def test_product_refusals(L, fn):
    assert getattr(L, fn)(None, None) == ARG
    for bad in (dict(type=2), dict(type=3), dict(type=-1), dict(E=0), dict(E=4097), dict(N=-1),
                dict(M=-1), dict(N=(1 << 20) + 1), dict(M=(1 << 20) + 1), dict(rows=-1),
                dict(rows=1 << 31), dict(slots=-1), dict(slots=(1 << 30) + 1), dict(align=0),
                dict(align=65537), dict(counts=0), dict(offsets=0), dict(packed=0),
                dict(counts=address(0) + 2), dict(offsets=address(1) + 1),
                dict(packed=address(2) + 1)):
        assert call(L, fn, **bad) == ARG, bad
    if fn == "vf_expert_product":
        for bad in (dict(weights=0), dict(out=0), dict(out=address(5) + 1),
                    dict(weights=address(3) + 1), dict(s0=-1), dict(s2=-8)):
            assert call(L, fn, **bad) == ARG, bad
        assert call(L, fn, s1=1 << 62) == OVERFLOW
        for over in (dict(out=address(2)), dict(out=address(3) + 64), dict(out=address(0)),
                     dict(out=address(1) - 8)):
            assert call(L, fn, **over) == ALIAS, over
    else:
        for bad in (dict(grad=0), dict(grad_weights=0), dict(out_type=1), dict(out_type=3),
                    dict(out_type=2, grad_weights=address(6) + 2)):
            assert call(L, fn, **bad) == ARG, bad
        for over in (dict(grad_weights=address(4)), dict(grad_weights=address(2) - 32),
                     dict(grad_weights=address(0))):
            assert call(L, fn, **over) == ALIAS, over


@PASSES
def test_product_accepts(L):
    assert call(L, "vf_expert_product") == CUDA
    assert call(L, "vf_expert_product", type=1, align=128, grad=0, grad_weights=0) == CUDA
    assert call(L, "vf_expert_product", s1=1, s2=24) == CUDA          # the view transposed
    assert call(L, "vf_expert_product", M=0, packed=0, weights=0) == CUDA
    assert call(L, "vf_expert_product", N=1, s1=3) == CUDA            # a stride that is not used
    assert call(L, "vf_expert_weight_grad", out_type=2, weights=0, out=0) == CUDA
    assert call(L, "vf_expert_weight_grad", rows=0, packed=0, grad=0) == CUDA


def test_nothing_to_do(L):
    assert call(L, "vf_expert_product", rows=0, out=0) == OK
    assert call(L, "vf_expert_product", N=0, out=0) == OK
    assert call(L, "vf_expert_weight_grad", N=0, grad_weights=0) == OK
    assert call(L, "vf_expert_weight_grad", M=0, grad_weights=0) == OK
    assert call(L, "vf_expert_glu", rows=0) == OK
    assert call(L, "vf_expert_glu_backward", F=0) == OK
    assert call(L, "vf_rms_norm", T=0) == OK
    assert call(L, "vf_rms_norm", M=0) == OK
    assert call(L, "vf_rms_norm_backward", M=0) == OK


def test_product_workspace(L):
    def size(fn="vf_expert_product", **kw):
        return getattr(L, fn + "_workspace")(desc("product", **kw))
    w, x = 4 * 24 * 16 * 2, 8 * 16 * 2
    assert size() == 0 and size(s1=1, s2=24) == 0 and size(M=0) == 0
    assert size(weights=address(3) + 2) == w and size(packed=address(2) + 2) == x
    assert size(weights=address(3) + 2, packed=address(2) + 2) == w + x
    assert size(s2=2, s1=32, s0=24 * 32) == w                  # no unit stride
    assert size(s0=0) == w                                     # one set for all experts
    assert size(M=15, s1=16) == 8 * 16 * 2                     # rows of 15, padded to 16
    assert size(M=15, s1=15, s0=24 * 15) == w + 8 * 16 * 2
    assert size(s1=1, s2=23, N=23, s0=23 * 16) == 4 * 16 * 24 * 2
    assert size(E=1, s0=7) == 0                                # a stride that is not used
    assert size(E=0) == ARG and size(s0=-8) == ARG
    fn = "vf_expert_weight_grad"
    assert size(fn) == 0 and size(fn, N=23) == 8 * 24 * 2 and size(fn, M=9) == 8 * 16 * 2
    assert size(fn, grad=address(4) + 8) == 8 * 24 * 2
    for fn, kw in (("vf_expert_product", dict(packed=address(2) + 2)),
                   ("vf_expert_weight_grad", dict(M=9))):
        assert call(L, fn, **kw) == CAPACITY
        assert call(L, fn, workspace=address(20) + 8, **kw) == ARG
        assert call(L, fn, workspace=address(0), **kw) == ALIAS
    assert call(L, "vf_expert_product", packed=address(2) + 2, workspace=address(5)) == ALIAS


@PASSES
def test_product_takes_a_workspace(L):
    for fn, kw in (("vf_expert_product", dict(packed=address(2) + 2)),
                   ("vf_expert_weight_grad", dict(M=9))):
        assert call(L, fn, workspace=address(20), **kw) == CUDA


def test_glu_refusals(L):
    for fn in ("vf_expert_glu", "vf_expert_glu_backward"):
        assert getattr(L, fn)(None, None) == ARG
        for bad in (dict(type=3), dict(type=-1), dict(E=0), dict(E=4097), dict(rows=-1),
                    dict(rows=1 << 31), dict(F=-1), dict(F=(1 << 30) + 1), dict(slot_of=0),
                    dict(offsets=0), dict(gate=0), dict(up=0), dict(gate=address(2) + 1),
                    dict(slot_of=address(0) + 2), dict(gate0=-1), dict(up1=-1)):
            assert call(L, fn, **bad) == ARG, bad
        assert call(L, fn, gate0=1 << 62) == OVERFLOW
    for bad in (dict(out=0), dict(out0=0), dict(out0=8), dict(out=address(3) + 1)):
        assert call(L, "vf_expert_glu", **bad) == ARG, bad
    for over in (dict(out=address(2) + 64), dict(out=address(0)), dict(out=address(1) - 16)):
        assert call(L, "vf_expert_glu", **over) == ALIAS, over
    fn = "vf_expert_glu_backward"
    for bad in (dict(grad=0), dict(grad_gate=0), dict(grad_up=0), dict(gg0=8), dict(gu0=0)):
        assert call(L, fn, **bad) == ARG, bad
    for over in (dict(grad_gate=address(4)), dict(grad_up=address(2)),
                 dict(grad_up=address(5) + 16),              # columns 8 .. 23 of gate's 0 .. 15
                 dict(grad_up=address(5)), dict(grad_up=address(5) + 32 + 16),
                 dict(gg0=24, gu0=24), dict(gu0=48), dict(gg1=2, gg0=64)):
        assert call(L, fn, **over) == ALIAS, over


@PASSES
def test_glu_accepts(L):
    assert call(L, "vf_expert_glu", grad=0, grad_gate=0, grad_up=0) == CUDA
    assert call(L, "vf_expert_glu", gate1=0, up0=0) == CUDA           # broadcast operands
    assert call(L, "vf_expert_glu_backward", out=0) == CUDA
    assert call(L, "vf_expert_glu_backward", grad_gate=address(5) + 32, grad_up=address(5)) == CUDA
    assert call(L, "vf_expert_glu_backward", grad_up=address(8), gu0=16) == CUDA
    assert call(L, "vf_expert_glu_backward", grad_up=address(5) + 64 + 32) == CUDA   # a row on


def test_norm_refusals(L):
    for fn in ("vf_rms_norm", "vf_rms_norm_backward"):
        assert getattr(L, fn)(None, None) == ARG
        for bad in (dict(type=3), dict(type=-1), dict(weight_type=1), dict(weight_type=3),
                    dict(T=-1), dict(T=(1 << 30) + 1), dict(M=-1), dict(M=(1 << 24) + 1),
                    dict(eps=-1e-6), dict(eps=NAN), dict(eps=INF), dict(x=0), dict(weight=0),
                    dict(x=address(0) + 1), dict(x0=-1), dict(weight=address(1) + 1)):
            assert call(L, fn, **bad) == ARG, bad
        assert call(L, fn, x0=1 << 62) == OVERFLOW
    fn = "vf_rms_norm"
    res = dict(residual=address(10))
    for bad in (dict(out=0), dict(o0=0), dict(o0=32),
                dict(total=0, **res), dict(t0=0, **res), dict(residual=address(10) + 1),
                dict(format=3), dict(format=-1), dict(format=1, group=48), dict(format=1, group=0),
                dict(format=1, type=1, weight_type=1), dict(format=2, type=2, weight_type=2),
                dict(format=1, codes=0), dict(format=1, scales=0),
                dict(format=1, scales=address(5) + 2)):
        assert call(L, fn, **bad) == ARG, bad
    for over in (dict(out=address(0)), dict(out=address(1) - 16), dict(total=address(0), **res),
                 dict(total=address(10), **res), dict(total=address(3), **res),
                 dict(format=1, codes=address(0)), dict(format=1, codes=address(5)),
                 dict(format=1, scales=address(1))):
        assert call(L, fn, **over) == ALIAS, over
    fn = "vf_rms_norm_backward"
    for bad in (dict(grad=0), dict(grad_x=0), dict(d0=0), dict(grad_weight=0), dict(workspace=0),
                dict(grad_weight=address(8) + 2), dict(workspace=address(9) + 8),
                dict(grad_total=address(10) + 1)):
        assert call(L, fn, **bad) == ARG, bad
    for over in (dict(grad_x=address(0)), dict(grad_x=address(6)), dict(grad_weight=address(1)),
                 dict(workspace=address(8)), dict(workspace=address(7)),
                 dict(grad_total=address(7))):
        assert call(L, fn, **over) == ALIAS, over


@PASSES
def test_norm_accepts(L):
    assert call(L, "vf_rms_norm", total=0) == CUDA
    assert call(L, "vf_rms_norm", residual=address(10)) == CUDA
    assert call(L, "vf_rms_norm", residual=address(0)) == CUDA        # x twice
    assert call(L, "vf_rms_norm", x0=0, x1=0) == CUDA
    assert call(L, "vf_rms_norm", format=2, out=0, group=32) == CUDA
    assert call(L, "vf_rms_norm", eps=0.0, weight_type=2) == CUDA
    assert call(L, "vf_rms_norm_backward", out=0, total=0) == CUDA
    assert call(L, "vf_rms_norm_backward", grad_total=address(6)) == CUDA
    assert call(L, "vf_rms_norm_backward", T=0, x=0, grad=0, grad_x=0, weight=0,
                workspace=0) == CUDA


def test_norm_workspace(L):
    assert L.vf_rms_norm_workspace(0, 64) == 0 and L.vf_rms_norm_workspace(1, 64) == 256
    assert L.vf_rms_norm_workspace(1 << 20, 64) <= 1 << 20
    for bad in ((-1, 64), (1, -1), ((1 << 30) + 1, 1), (1, (1 << 24) + 1)):
        assert L.vf_rms_norm_workspace(*bad) == ARG
