"""The norm, the experts' products and the gated activation as they are used: a
mixture-of-experts layer with its backward pass, captured graphs, other streams,
several host threads, offsets past 2^31, and random cases against float64.

In the layer every call is held to its own oracle, given the tensors that the calls
before it have left, with the bounds of ``tests/test_gpu_layer.py`` and
``tests/test_gpu_product.py``.
"""
import random
import threading

import pytest
import torch

import sequence_head_relayout_gb300 as vf
from oracle import experts as X
from oracle import layer as L

from .test_gpu_expert import rounding, within
from .test_gpu_expert_flow import gen, randn, routing
from .test_gpu_layer import (U, backward_check, check_norm, glu_backward_bounds, glu_bound,
                             masked, norm_bound)
from .test_gpu_product import CUT, check_product, check_weight_grad

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("oracle_built")]

DEV = torch.device("cuda:0")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    vf.lib()
    yield
    torch.cuda.synchronize()


def inputs(T, K, E, M, F, seed, dtype=BF16):
    """x, residual, norm weight, experts, routing weights, W1 [E,2F,M], W2 [E,M,F], the
    gradients of the layer's result and of the residual stream."""
    return (randn((T, M), seed, dtype), randn((T, M), seed + 1, dtype),
            randn((M,), seed + 2, dtype), routing(T, K, E, seed + 3),
            torch.rand(T, K, generator=gen(seed + 4), device=DEV),
            randn((E, 2 * F, M), seed + 5, dtype) * M ** -0.5,
            randn((E, M, F), seed + 6, dtype) * F ** -0.5,
            randn((T, M), seed + 7, dtype), randn((T, M), seed + 8, dtype))


def layer(x, res, wn, e, w, W1, W2, gout, gres, align=16, stream=None):
    """Forward and backward pass; every tensor of it by name."""
    E, F = W1.shape[0], W2.shape[2]
    kw = dict(stream=stream)
    s = {}
    s["plan"] = plan = vf.expert_plan(e, E, align=align, **kw)
    s["y"], s["h"] = vf.rms_norm(x, wn, residual=res, **kw)
    s["rows"] = vf.expert_pack(s["y"], plan, **kw)
    s["both"] = vf.expert_product(s["rows"], W1, plan, **kw)
    s["act"] = vf.expert_glu(s["both"][:, :F], s["both"][:, F:], plan, **kw)
    s["down"] = vf.expert_product(s["act"], W2, plan, **kw)
    s["out"] = vf.expert_merge(s["down"], plan, w, **kw)
    s["gdown"], s["gw"] = vf.expert_merge_backward(gout, s["down"], plan, w, **kw)
    s["gW2"] = vf.expert_weight_grad(s["gdown"], s["act"], plan, dtype=F32, **kw)
    s["gact"] = vf.expert_product(s["gdown"], W2.transpose(1, 2), plan, **kw)
    gg, _ = vf.expert_glu_backward(s["gact"], s["both"][:, :F], s["both"][:, F:], plan, **kw)
    s["gboth"] = gg.as_strided((gg.shape[0], 2 * F), (2 * F, 1))     # both halves
    s["gW1"] = vf.expert_weight_grad(s["gboth"], s["rows"], plan, **kw)
    s["grows"] = vf.expert_product(s["gboth"], W1.transpose(1, 2), plan, **kw)
    s["gy"] = vf.expert_merge(s["grows"], plan, **kw)
    s["gx"], s["gwn"] = vf.rms_norm_backward(s["gy"], s["h"], wn, grad_total=gres, **kw)
    return s


def same(a, b):
    """Bitwise, but for the rows behind the last expert, which are not written."""
    used = int(a["plan"].offsets[-1])
    rows = a["plan"].slot_of.numel()
    for name in a:
        u, v = a[name], b[name]
        if name == "plan":
            assert all(torch.equal(p, q) for p, q in zip(u[:4], v[:4]))
            continue
        if u.shape[0] == rows and u.dim() == 2:
            u, v = u[:used], v[:used]
        assert torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8)), name


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,K,E,M,F,align", [(150, 3, 7, 96, 72, 16), (1, 2, 8, 64, 128, 1),
                                             (700, 2, 3, 264, 130, 1), (40, 4, 30, 65, 33, 5)])
def test_layer(T, K, E, M, F, align, dtype):
    ins = inputs(T, K, E, M, F, 1, dtype)
    s = layer(*ins, align=align)
    x, res, wn, e, w, W1, W2, gout, gres = (t.cpu() for t in ins)
    plan, c = s["plan"], {k: v.cpu() for k, v in s.items() if k != "plan"}
    counts, offsets = plan.counts.cpu(), plan.offsets.cpu()
    used, slot = int(offsets[-1]), plan.slot_of.cpu()

    def product(name, rows, weights):
        want, mag = X.product(c[rows], weights, counts, offsets, c[name])
        err = mag * (c[rows].shape[1] * CUT)
        within(c[name][:used], want[:used], (err + rounding(want.abs() + err, dtype))[:used])

    def weights(name, grad, rows):
        want, mag = X.weight_grad(c[grad], c[rows], counts, offsets)
        err = mag * (max(1, int(counts.max())) * CUT)
        within(c[name], want, err + rounding(want.abs() + err, c[name].dtype))

    assert torch.equal(c["h"], L.total(x, res))
    within(c["y"], *norm_bound(c["h"], wn, 1e-6, dtype))
    token = slot[:used].clamp(min=0) // K
    assert torch.equal(c["rows"][:used][slot[:used] >= 0], c["y"][token][slot[:used] >= 0])
    product("both", "rows", W1)
    a = masked(plan, *glu_bound(c["both"][:, :F], c["both"][:, F:], dtype), 0.0)
    within(c["act"][:used], *(t[:used] for t in a))
    product("down", "act", W2)
    out, mag = X.merge(c["down"], plan.row_of.cpu(), w)
    err = mag * K * U
    within(c["out"], out, err + rounding(out.abs() + err, dtype))
    weights("gW2", "gdown", "act")
    product("gact", "gdown", W2.transpose(1, 2))
    for half, got in zip(glu_backward_bounds(c["gact"], c["both"][:, :F], c["both"][:, F:], dtype),
                         (c["gboth"][:, :F], c["gboth"][:, F:])):
        a = masked(plan, *half, 0.0)
        within(got[:used], *(t[:used] for t in a))
    weights("gW1", "gboth", "rows")
    product("grows", "gboth", W1.transpose(1, 2))
    gx, gwn, mag, mag_w = L.norm_backward(c["gy"], c["h"], wn, 1e-6, gres)
    err = mag * (2 * M + 20) * U
    within(c["gx"], gx, err + rounding(gx.abs() + err, dtype))
    within(c["gwn"], gwn, mag_w * (T + M / 2 + 16) * U + 2.0 ** -149)
    same(s, layer(*ins, align=align))


def test_codes_of_the_norm_go_to_the_experts():
    """rms_norm_q -> expert_restore_q: the normed rows by way of 8 bits, packed."""
    T, K, E, M = 90, 2, 5, 264
    x, res, wn, e = inputs(T, K, E, M, 8, 3)[:4]
    plan = vf.expert_plan(e, E, align=4)
    for fmt in ("int8", "e4m3"):
        codes, scales, h = vf.rms_norm_q(x, wn, fmt=fmt, group=64, residual=res)
        rows = vf.expert_restore_q(codes, scales, plan, fmt, 64)
        value = codes.float() * scales.repeat_interleave(64, 1)[:, :M]
        owned = plan.slot_of >= 0
        token = (plan.slot_of[owned] // K).long()
        assert torch.equal(rows[owned], value[token].to(BF16))


def test_captured_layers_with_a_graph_each():
    """Two layers captured, replayed at once on two streams with new inputs: as the
    eager layer, bit for bit.  The second has operands that are copied first."""
    sizes = [(600, 2, 6, 128, 192), (300, 3, 9, 99, 75)]
    ins, graphs, outs, streams = [], [], [], []
    for i, z in enumerate(sizes):
        ins.append(inputs(*z, 20 * i))
        layer(*ins[i])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer(*ins[i]))
        graphs.append(g)
        streams.append(torch.cuda.Stream(DEV))
    for trial in range(3):
        for i, z in enumerate(sizes):
            for old, new in zip(ins[i], inputs(*z, 1000 * (trial + 1) + 20 * i)):
                old.copy_(new)
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            same(outs[i], layer(*ins[i]))


def test_layer_on_another_stream():
    """Each call on a stream given by `stream`, behind work of that stream that has not
    run yet; nothing on the current stream orders them."""
    for z in ((500, 2, 6, 128, 64), (200, 2, 6, 67, 35)):
        final = inputs(*z, 7)
        want = layer(*final)
        late = [torch.zeros_like(t) for t in final]
        side = torch.cuda.Stream(DEV)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            for a, b in zip(late, final):
                a.copy_(b)
        got = layer(*late, stream=side)
        side.synchronize()
        same(want, got)


def test_layers_in_host_threads():
    sizes = [(200, 2, 6, 128, 64), (900, 1, 2, 64, 256), (3, 4, 30, 72, 40), (60, 2, 4, 33, 31)]
    ins = [inputs(*z, 100 * i) for i, z in enumerate(sizes)]
    want = [layer(*i) for i in ins]
    torch.cuda.synchronize()
    got, errors = [None] * len(ins), []

    def work(i):
        try:
            s = torch.cuda.Stream(DEV)
            with torch.cuda.stream(s):
                for _ in range(8):
                    got[i] = layer(*ins[i])
            s.synchronize()
        except Exception as ex:                       # reported by the main thread
            errors.append(ex)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(ins))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(want, got):
        same(a, b)


# ---- offsets past 2^31 -----------------------------------------------------------------

def test_products_past_31_bits():
    T, K, E, M, N = 36000, 8, 16, 8192, 64              # 288,000 rows, 2.36e9 elements
    plan = vf.expert_plan(routing(T, K, E, 1, dropped=0.0), E)
    n = plan.slot_of.numel()
    assert n * M > 2 ** 31
    x = torch.empty((n, M), dtype=BF16, device=DEV).normal_(generator=gen(2))
    w = randn((E, N, M), 3, BF16)
    far = torch.arange(n - 500, n, device=DEV)
    e = E - 1
    assert int(plan.offsets[e]) < n - 500
    out = vf.expert_product(x, w, plan)
    want, mag = (a.double() @ b.double().t() for a, b in ((x[far], w[e]),
                                                          (x[far].abs(), w[e].abs())))
    err = mag * (M * CUT)
    within(out[far], want.cpu(), (err + rounding(want.abs() + err, BF16)).cpu())
    # rows of M outputs: the result's offsets pass 2^31 too
    y = randn((n, N), 4, BF16)
    wide = vf.expert_product(y, w.transpose(1, 2), plan)
    want, mag = (a.double() @ b.double() for a, b in ((y[far], w[e]), (y[far].abs(), w[e].abs())))
    err = mag * (N * CUT)
    within(wide[far], want.cpu(), (err + rounding(want.abs() + err, BF16)).cpu())
    s = slice(int(plan.offsets[e]), n)
    for dtype in (BF16, F32):
        got = vf.expert_weight_grad(y, x, plan, dtype=dtype)[e]
        want, mag = (a.double().t() @ b.double() for a, b in ((y[s], x[s]),
                                                              (y[s].abs(), x[s].abs())))
        err = mag * (int(plan.counts[e]) * CUT)
        within(got, want.cpu(), (err + rounding(want.abs() + err, dtype)).cpu())
    # an odd view of the same rows: its copy's offsets pass 2^31
    odd = x.view(-1)[1:1 + n * (M - 1)].view(n, M - 1)
    got = vf.expert_product(odd, w[:, :, 1:], plan)
    want, mag = (a.double() @ b.double().t() for a, b in (
        (odd[far], w[e, :, 1:]), (odd[far].abs(), w[e, :, 1:].abs())))
    err = mag * (M * CUT)
    within(got[far], want.cpu(), (err + rounding(want.abs() + err, BF16)).cpu())


def test_weights_past_31_bits():
    E, N, M = 600, 1024, 4096                            # 2.5e9 elements
    e = torch.tensor([[E - 1], [0], [E - 2], [E - 1]], device=DEV)
    plan = vf.expert_plan(e, E)
    w = torch.zeros((E, N, M), dtype=BF16, device=DEV)
    w[-2:].normal_(generator=gen(1))
    x = randn((4, M), 2, BF16)
    got = vf.expert_product(x, w, plan)
    assert (got[0] == 0).all()
    for row, ex in ((1, E - 2), (2, E - 1), (3, E - 1)):
        want, mag = (w[ex].double() @ x[row].double(), w[ex].double().abs() @ x[row].double().abs())
        err = mag * (M * CUT)
        within(got[row], want.cpu(), (err + rounding(want.abs() + err, BF16)).cpu())
    g = randn((4, N), 3, BF16)
    dw = vf.expert_weight_grad(g, x, plan, out=w)
    assert (dw[1:-2] == 0).all()
    want = g[2:].double().t() @ x[2:].double()
    mag = g[2:].double().abs().t() @ x[2:].double().abs()
    within(dw[-1], want.cpu(), (mag * 2 * CUT + rounding(want.abs() + mag * 2 * CUT, BF16)).cpu())


def test_rows_past_31_bits():
    T, M = 300000, 8192                                  # 2.46e9 elements
    x = torch.empty((T, M), dtype=BF16, device=DEV).normal_(generator=gen(1))
    wn = randn((M,), 2, BF16)
    far = slice(T - 40, T)
    out = vf.rms_norm(x, wn)
    within(out[far], *norm_bound(x[far].cpu(), wn.cpu(), 1e-6, BF16))
    gx, gw = vf.rms_norm_backward(out, x, wn)
    want, _, mag, _ = L.norm_backward(out[far].cpu(), x[far].cpu(), wn.cpu(), 1e-6)
    err = mag * (2 * M + 20) * U
    within(gx[far], want, err + rounding(want.abs() + err, BF16))
    plan = vf.expert_plan(torch.zeros((T, 1), dtype=torch.int32, device=DEV), 1)
    act = vf.expert_glu(x, out, plan, out=gx)
    within(act[far], *glu_bound(x[far].cpu(), out[far].cpu(), BF16))
    codes, scales = vf.rms_norm_q(x, wn)
    few = vf.rms_norm_q(x[far], wn)
    assert torch.equal(codes[far].view(torch.uint8), few[0].view(torch.uint8))
    assert torch.equal(scales[far], few[1])
    # a view whose rows lie far apart
    base = torch.empty(40000 * 60000, dtype=BF16, device=DEV)
    view = base.as_strided((40000, 64), (60000, 1))
    view.copy_(x[:40000, :64])
    near = x[:40000, :64].contiguous()
    assert torch.equal(vf.rms_norm(view, wn[:64]), vf.rms_norm(near, wn[:64]))


# ---- random cases ------------------------------------------------------------------------

@pytest.mark.parametrize("seed", range(24))
def test_random_cases(seed):
    r = random.Random(seed)
    K = r.choice([1, 2, 3, 8])
    E = max(K, r.choice([1, 2, 5, 17, 64, 200]))
    T = int(10 ** r.uniform(0, 3.2))
    N, M = (r.choice([r.randint(1, 300), 8 * r.randint(1, 40), 64 * r.randint(1, 6)])
            for _ in range(2))
    dtype = r.choice([BF16, F16])
    plan = vf.expert_plan(routing(T, K, E, seed, dropped=r.choice([0.0, 0.2, 0.9])), E,
                          align=r.choice([1, 1, 8, 128]))
    n = plan.slot_of.numel()
    x, g = randn((n, M), seed, dtype), randn((n, N), seed + 1, dtype)
    x[plan.slot_of < 0], g[plan.slot_of < 0] = float("nan"), float("inf")
    w = randn((E, N, M), seed + 2, dtype)
    check_product(plan, x.cpu(), w.cpu(), w)
    check_product(plan, g.cpu(), w.cpu().transpose(1, 2), w.transpose(1, 2))
    check_weight_grad(plan, g.cpu(), x.cpu(), r.choice([dtype, F32]))
    t = randn((T, M), seed + 3, r.choice([BF16, F16, F32]))
    wn = randn((M,), seed + 4, r.choice([t.dtype, F32]))
    check_norm(t.cpu(), wn.cpu(), residual=torch.flip(t, [0]).cpu())
    backward_check(t.cpu(), torch.flip(t, [1]).cpu(), wn.cpu(), more=t.cpu() * 2)
