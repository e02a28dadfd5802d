"""Host side of the expert relayouts without a GPU: sizes, and every argument
refused before the library touches CUDA.  Fake pointer values are safe: nothing
is dereferenced or launched; a call that passes every host check reaches the
CUDA pointer query, which fails here with VF_ERR_CUDA."""
import ctypes

import pytest
import torch

import sequence_head_relayout_gb300 as vf

I64 = ctypes.c_int64
OK, ARG, OVERFLOW, ALIAS, CUDA = 0, -1, -2, -3, -4
# no device here: a call that passes every host check ends at the pointer query
PASSES = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers pass the checks")
A = {name: (i + 1) << 40 for i, name in enumerate(
    ("experts", "row_of", "slot_of", "counts", "offsets", "work", "tokens", "packed", "weights",
     "codes", "scales", "grad_packed", "grad_weights"))}
CALLS = ("vf_expert_pack", "vf_expert_restore", "vf_expert_merge", "vf_expert_merge_backward")


@pytest.fixture(scope="module")
def L(lib_built):
    return vf.lib()


def _i64(*xs):
    return (I64 * len(xs))(*xs)


def test_rows(L):
    assert vf.expert_rows(0, 2, 8, 16) == 0
    assert vf.expert_rows(1, 2, 8, 16) == 2 + 2 * 15          # two experts at the most
    assert vf.expert_rows(100, 2, 8, 16) == 200 + 8 * 15
    assert vf.expert_rows(1 << 27, 8, 4096, 1) == 1 << 30
    for bad in ((-1, 2, 8, 1), (1, 0, 8, 1), (1, 2, 0, 1), (1, 2, 8, 0), (1, 2, 4097, 1),
                ((1 << 30) + 1, 1, 8, 1), (1 << 28, 8, 8, 1), (1 << 30, 1, 4096, 1 << 20),
                (1, 2, 8, 65537), (1, 2, 8, 1 << 31)):
        assert L.vf_expert_rows(*bad) == ARG, bad
        with pytest.raises(vf.VFError):
            vf.expert_rows(*bad)
    assert L.vf_expert_workspace(1, 8, 256) == 0
    assert L.vf_expert_workspace(1 << 20, 8, 256) > 0
    assert L.vf_expert_workspace(1, 8, 0) == ARG


def _plan(L, experts=A["experts"], nbytes=8, strides=(8, 1), T=1 << 16, K=8, E=64, align=1,
          row_of=A["row_of"], slot_of=A["slot_of"], counts=A["counts"], offsets=A["offsets"],
          work=A["work"]):
    return L.vf_expert_plan(experts, nbytes, None if strides is None else _i64(*strides), T, K, E,
                            align, row_of, slot_of, counts, offsets, work, None)


def test_plan_refusals(L):
    assert _plan(L, nbytes=2) == ARG
    assert _plan(L, strides=None) == ARG
    assert _plan(L, strides=(-1, 1)) == ARG
    assert _plan(L, T=-1) == ARG
    assert _plan(L, E=0) == ARG
    assert _plan(L, align=0) == ARG
    assert _plan(L, strides=(1 << 62, 1)) == OVERFLOW
    for name in ("experts", "row_of", "slot_of", "counts", "offsets", "work"):
        assert _plan(L, **{name: None}) == ARG, name
        assert _plan(L, **{name: A[name] + 2}) == ARG, name    # not aligned to its items
    assert _plan(L, row_of=A["experts"] + 64) == ALIAS         # written over what is read
    assert _plan(L, slot_of=A["row_of"] + 64) == ALIAS         # two written ranges
    assert _plan(L, counts=A["offsets"] + 64 * 4) == ALIAS
    assert _plan(L, work=A["slot_of"]) == ALIAS


@PASSES
def test_plan_accepts(L):
    assert _plan(L) == CUDA
    assert _plan(L, nbytes=4, experts=A["experts"] + 4) == CUDA
    assert _plan(L, T=4, work=None) == CUDA                    # one block: no workspace
    assert _plan(L, strides=(0, 0)) == CUDA                    # a broadcast routing
    assert _plan(L, counts=A["offsets"] + 65 * 4) == CUDA
    assert _plan(L, T=0, experts=None, row_of=None, slot_of=None) == CUDA


def _desc(**kw):
    d = vf._ExpertDesc(type=0, format=0, T=4, K=2, M=64, E=4, rows=8, align=1, group=64)
    for name in ("row_of", "counts", "offsets", "tokens", "packed", "weights", "codes", "scales",
                 "grad_packed", "grad_weights"):
        setattr(d, name, A[name])
    d.token_strides[0], d.token_strides[1] = 64, 1
    d.weight_strides[0], d.weight_strides[1] = 2, 1
    if "strides" in kw:
        d.token_strides[0], d.token_strides[1] = kw.pop("strides")
    if "weight_strides" in kw:
        d.weight_strides[0], d.weight_strides[1] = kw.pop("weight_strides")
    for name, v in kw.items():
        setattr(d, name, v)
    return d


def _call(L, fn, **kw):
    if fn == "vf_expert_restore":
        kw.setdefault("format", 1)
    return getattr(L, fn)(ctypes.byref(_desc(**kw)), None)


@pytest.mark.parametrize("fn", CALLS)
def test_row_call_refusals(L, fn):
    assert getattr(L, fn)(None, None) == ARG
    for bad in (dict(type=3), dict(type=-1), dict(T=-1), dict(K=0), dict(M=-1), dict(E=0),
                dict(rows=-1), dict(rows=1 << 31), dict(align=0), dict(align=65537), dict(format=3), dict(format=-1),
                dict(format=1, group=48), dict(format=2, group=0), dict(format=1, type=1),
                dict(format=1, type=2), dict(row_of=None), dict(row_of=A["row_of"] + 2),
                dict(T=1 << 30, K=2), dict(M=1 << 31)):
        assert _call(L, fn, **bad) == ARG, bad
    # ranges of 2^61 bytes fit no address space: refused, by overlap if nothing else
    assert _call(L, fn, rows=(1 << 31) - 1, M=1 << 30, T=1 << 20) in (ARG, OVERFLOW, ALIAS, CUDA)
    # a plan with gaps reads counts and offsets wherever rows are written
    if fn != "vf_expert_merge":
        assert _call(L, fn, align=8, counts=None) == ARG
        assert _call(L, fn, align=8, offsets=A["offsets"] + 1) == ARG


def test_restore_needs_a_format(L):
    assert _call(L, "vf_expert_restore", format=0) == ARG


def test_row_call_pointers(L):
    for fn, fmt, used in (
            ("vf_expert_pack", 0, ("tokens", "packed")),
            ("vf_expert_pack", 1, ("tokens", "packed", "codes", "scales")),
            ("vf_expert_restore", 2, ("packed", "codes", "scales")),
            ("vf_expert_merge", 0, ("tokens", "packed")),
            ("vf_expert_merge", 2, ("tokens", "packed", "codes", "scales")),
            ("vf_expert_merge_backward", 0, ("tokens", "packed", "weights", "grad_packed",
                                             "grad_weights")),
            ("vf_expert_merge_backward", 1, ("tokens", "codes", "scales", "weights",
                                             "grad_packed", "grad_weights"))):
        for name in used:
            assert _call(L, fn, format=fmt, **{name: None}) == ARG, (fn, name)
            if name != "codes":
                assert _call(L, fn, format=fmt, **{name: A[name] + 1}) == ARG, (fn, name)


def test_row_call_strides(L):
    for fn in ("vf_expert_pack", "vf_expert_merge", "vf_expert_merge_backward"):
        assert _call(L, fn, strides=(-64, 1)) == ARG
        assert _call(L, fn, strides=(1 << 62, 1)) == OVERFLOW
        assert _call(L, fn, weight_strides=(2, -1)) == (ARG if fn != "vf_expert_pack" else
                                                        _call(L, fn))
    # only the merge writes its token view: it must not overlap itself
    assert _call(L, "vf_expert_merge", strides=(0, 1)) == ARG
    assert _call(L, "vf_expert_merge", strides=(63, 1)) == ARG
    assert _call(L, "vf_expert_merge", strides=(1, 1)) == ARG


def test_row_call_aliasing(L):
    t, p = A["tokens"], A["packed"]
    for fn in ("vf_expert_pack", "vf_expert_merge"):
        assert _call(L, fn, packed=t + 4 * 64 * 2 - 2) == ALIAS
        assert _call(L, fn, format=1, codes=t + 1) == ALIAS
        assert _call(L, fn, format=1, codes=p + 1) == ALIAS
        assert _call(L, fn, format=1, scales=A["codes"] + 4) == ALIAS
    assert _call(L, "vf_expert_pack", row_of=p) == ALIAS
    assert _call(L, "vf_expert_merge", weights=t + 8) == ALIAS
    assert _call(L, "vf_expert_restore", packed=A["codes"] - 2) == ALIAS
    assert _call(L, "vf_expert_merge_backward", grad_packed=p) == ALIAS
    assert _call(L, "vf_expert_merge_backward", grad_packed=t) == ALIAS
    assert _call(L, "vf_expert_merge_backward", grad_weights=A["weights"]) == ALIAS
    assert _call(L, "vf_expert_merge_backward", grad_weights=A["grad_packed"]) == ALIAS


@PASSES
def test_row_call_accepts(L):
    for fn in CALLS:
        assert _call(L, fn) == CUDA
        assert _call(L, fn, format=2) == CUDA
        assert _call(L, fn, align=8) == CUDA
        # nothing to move: no pointer is looked at
        assert _call(L, fn, T=0, tokens=None, packed=None, row_of=None) == OK
    assert _call(L, "vf_expert_pack", M=0, tokens=None, packed=None) == OK
    assert _call(L, "vf_expert_pack", strides=(0, 0)) == CUDA         # a broadcast row
    assert _call(L, "vf_expert_merge", weights=None) == CUDA
    assert _call(L, "vf_expert_merge", codes=A["codes"] + 1, format=1) == CUDA
    assert _call(L, "vf_expert_merge_backward", packed=None, format=1) == CUDA
    # the weights of M = 0 columns still have their (zero) gradients
    assert _call(L, "vf_expert_merge_backward", M=0, tokens=None, packed=None,
                 grad_packed=None) == CUDA


def test_binding_refusals(L):
    plan = vf.ExpertPlan(*(torch.zeros(s, dtype=torch.int32) for s in ((4, 2), (8,), (4,), (5,))))
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        vf.expert_plan(torch.zeros(4, 2, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="CUDA"):
        vf.expert_pack(x, plan)
    with pytest.raises(TypeError):
        vf.expert_pack(None, plan)
    with pytest.raises(ValueError, match="bfloat16"):
        vf.expert_pack_q(x.half(), plan)
    with pytest.raises(ValueError, match="bfloat16"):
        vf.expert_merge_q(x.float(), plan)
    with pytest.raises(ValueError, match="bfloat16"):
        vf.expert_merge_backward_q(x.half(), None, None, plan, None)
    with pytest.raises(ValueError, match="fmt"):
        vf.expert_restore_q(x, None, plan, fmt="fp4")


def test_descriptor_layout_matches_the_header(tmp_path):
    """The ctypes descriptor against the C compiler's view of the header."""
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = [f[0] for f in vf._ExpertDesc._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "vf_relayout.h"\n'
                   "int main(void) {\n" +
                   "".join('printf("%%zu ", offsetof(vf_expert_desc, %s));\n' % n for n in names) +
                   'printf("%zu\\n", sizeof(vf_expert_desc));\nreturn 0;\n}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    "-o", str(exe), str(src)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [getattr(vf._ExpertDesc, n).offset for n in names] + \
        [ctypes.sizeof(vf._ExpertDesc)]


@pytest.mark.parametrize("fn", CALLS)
def test_row_calls_limit_the_slots_of_a_token(L, fn):
    """A token's slots are taken in turn: 2^30 of one token would run for minutes."""
    for fmt in (0, 1):
        if fn != "vf_expert_restore" or fmt:
            for T, K in ((1, 65537), (1, 1 << 30), (0, 65537)):
                assert _call(L, fn, format=fmt, T=T, K=K) == ARG, (T, K)
            most = _call(L, fn, format=fmt, T=1, K=65536, weight_strides=(65536, 1))
            assert most == (ARG if torch.cuda.is_available() else CUDA)  # fake pointers
    # a plan sorts slots, however they are spread over tokens
    assert vf.expert_rows(1, 1 << 30, 8) == 1 << 30


def test_row_calls_and_ranges_that_wrap(L):
    """The exact status of ranges that end past the address space, of huge ones that
    cover the others, and of a view that covers itself."""
    end = 1 << 64
    for fn, name, size in (("vf_expert_pack", "packed", 8 * 64 * 2),
                           ("vf_expert_pack", "tokens", 4 * 64 * 2),
                           ("vf_expert_restore", "packed", 8 * 64 * 2),
                           ("vf_expert_restore", "codes", 4 * 64),
                           ("vf_expert_merge", "packed", 8 * 64 * 2),
                           ("vf_expert_merge", "weights", 4 * 2 * 4),
                           ("vf_expert_merge_backward", "grad_packed", 8 * 64 * 2),
                           ("vf_expert_merge_backward", "grad_weights", 4 * 2 * 4),
                           ("vf_expert_merge_backward", "row_of", 4 * 2 * 4)):
        assert _call(L, fn, **{name: end - size}) == OVERFLOW, (fn, name)
        assert _call(L, fn, **{name: end - 4 if size > 4 else end - 2}) == OVERFLOW, (fn, name)
    assert _plan(L, T=4, work=None, row_of=end - 4 * 8 * 4) == OVERFLOW
    assert _plan(L, T=4, work=None, strides=(1 << 61, 1)) == OVERFLOW
    huge = dict(rows=(1 << 31) - 1, M=1 << 30, T=1 << 20)
    # of the pack's ranges packed lies highest here: nothing is above it to be covered
    assert _call(L, "vf_expert_pack", **huge) == (ARG if torch.cuda.is_available() else CUDA)
    assert _call(L, "vf_expert_pack", row_of=A["grad_weights"], **huge) == ALIAS
    assert _call(L, "vf_expert_restore", **huge) == ALIAS
    assert _call(L, "vf_expert_merge", **huge) == ARG              # rows of 2^30, 64 apart
    assert _call(L, "vf_expert_merge_backward", **huge) == ALIAS


def test_pack_does_not_look_at_weights(L):
    reached = ARG if torch.cuda.is_available() else CUDA           # fake pointers
    assert _call(L, "vf_expert_pack", weight_strides=(2, -1), weights=1) == reached
    assert _call(L, "vf_expert_restore", weight_strides=(2, -1), weights=1) == reached
    assert _call(L, "vf_expert_merge", weight_strides=(2, -1)) == ARG
    assert _call(L, "vf_expert_merge_backward", weight_strides=(2, -1)) == ARG
