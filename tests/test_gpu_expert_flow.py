"""The expert relayouts as they are used: a whole mixture-of-experts layer and
its backward pass, captured graphs, other streams, several host threads, sizes
whose offsets pass 2^31, and random cases of every call against float64.

Bounds as in ``tests/test_gpu_expert.py``: a float32 sum of n products is off by
at most n u / (1 - n u) times the sum of the magnitudes, u = 2^-24, one rounding
to a type by at most half a unit of it.
"""
import threading

import pytest
import torch

import sequence_head_relayout_gb300 as vf

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    vf.lib()
    yield
    torch.cuda.synchronize()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def routing(T, K, E, seed, dropped=0.1):
    g = gen(seed)
    e = torch.topk(torch.rand(T, E, generator=g, device=DEV), K, dim=1).indices
    e[torch.rand(T, K, generator=g, device=DEV) < dropped] = -1
    return e


def randn(shape, seed, dtype=torch.float32):
    return torch.randn(shape, generator=gen(seed), device=DEV).to(dtype)


def gamma(n):
    return n * U / (1 - n * U)


def within(got, want, bound, what=""):
    off = (got.double() - want).abs() - bound
    assert off.numel() == 0 or off.max().item() <= 0, "%s off by %g over the bound" % (
        what, off.max().item())


# ---- a whole layer --------------------------------------------------------------

@pytest.mark.parametrize("align", [1, 16])
def test_layer_forward_and_backward(align):
    """Linear experts: out[t] = sum_k w[t,k] x[t] A_e.  Forward and all four
    gradients against float64 autograd of the definition, which knows no rows."""
    T, K, E, M, N = 150, 3, 7, 96, 72
    e = routing(T, K, E, 1)
    x, A, w = randn((T, M), 2), randn((E, M, N), 3), torch.rand(T, K, generator=gen(4), device=DEV)
    grad = randn((T, N), 5)

    plan = vf.expert_plan(e, E, align=align)
    rows = plan.slot_of.numel()
    first, count = plan.offsets.tolist(), plan.counts.tolist()
    segment = [slice(first[i], first[i] + count[i]) for i in range(E)]
    px = vf.expert_pack(x, plan)
    py = torch.zeros(rows, N, device=DEV)
    for i, s in enumerate(segment):
        py[s] = px[s] @ A[i]
    out = vf.expert_merge(py, plan, w)
    gy, gw = vf.expert_merge_backward(grad, py, plan, w)
    gA = torch.stack([px[s].t() @ gy[s] for s in segment])
    if align > 1:                            # whole aligned segments: gap rows are zeros
        whole = [slice(first[i], first[i + 1]) for i in range(E)]
        for i, s in enumerate(whole):
            assert (px[s][count[i]:] == 0).all() and (gy[s][count[i]:] == 0).all()
    gpx = torch.zeros(rows, M, device=DEV)
    for i, s in enumerate(segment):
        gpx[s] = gy[s] @ A[i].t()
    gx = vf.expert_merge(gpx, plan)

    def dense(x, A, w, grad):
        there = ((e >= 0) & (e < E)).double()
        y = torch.einsum("tm,tkmn->tkn", x, A[e.clamp(min=0)])
        return ((w * there)[:, :, None] * y).sum(1)

    leaves = [v.double().requires_grad_() for v in (x, A, w)]
    want = dense(*leaves, grad)
    wants = [want] + list(torch.autograd.grad(want, leaves, grad.double()))
    # the same in magnitudes: every product's and sum's terms
    mags = [v.double().abs().requires_grad_() for v in (x, A, w)]
    mag = dense(*mags, grad)
    bounds = [mag] + list(torch.autograd.grad(mag, mags, grad.double().abs()))
    # roundings on the way of a term: its dot products, the sum over K, the weight
    steps = [M + K + 2, N + K + 3, T + K + 3, M + N + 3]
    for name, got, want, b, n in zip(("out", "x", "A", "w"), (out, gx, gA, gw), wants, bounds,
                                     steps):
        within(got, want.detach(), gamma(n) * b.detach(), name)


def small_step(e, x, grad, w, E, fmt, align, out=None):
    """plan -> pack with a checkpoint -> merge with a checkpoint -> backward from
    the codes -> the rows restored; every tensor of it."""
    plan = vf.expert_plan(e, E, align=align)
    packed, c1, s1 = vf.expert_pack_q(x, plan, fmt, 64)
    y = vf.expert_restore_q(c1, s1, plan, fmt, 64)
    merged, c2, s2 = vf.expert_merge_q(y, plan, w, fmt, 64)
    gp, gw = vf.expert_merge_backward_q(grad, c2, s2, plan, w, fmt, 64)
    gx = vf.expert_merge(gp, plan)
    owned = plan.slot_of >= 0
    return plan, packed, c1, s1, y, merged, c2, s2, gp, gw, gx, owned


def same(a, b):
    """Bitwise, but for packed rows that no slot owns (not all are written)."""
    owned = a[-1]
    assert torch.equal(owned, b[-1])
    for u, v in zip(a[0], b[0]):
        assert u == v if isinstance(u, int) else torch.equal(u, v)
    for i, (u, v) in enumerate(zip(a[1:-1], b[1:-1])):
        if u.shape[0] == owned.shape[0]:
            u, v = u[owned], v[owned]
        assert torch.equal(u.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8)), i


@pytest.mark.parametrize("fmt,E", [("int8", 48), ("e4m3", 48), ("int8", 600)])
def test_captured_steps_with_a_graph_each(fmt, E):
    """Two steps captured (each plan over many blocks, with a workspace; at E = 600
    with more than 48 KB of shared memory), replayed at once on two streams with new
    inputs: as the eager step, bit for bit."""
    T, K, M = 2500, 4, 264
    ins, graphs, outs, streams = [], [], [], []
    for i in range(2):
        ins.append((routing(T, K, E, i), randn((T, M), 10 + i, torch.bfloat16),
                    randn((T, M), 20 + i, torch.bfloat16),
                    torch.rand(T, K, generator=gen(30 + i), device=DEV)))
        small_step(*ins[i], E, fmt, 8)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(small_step(*ins[i], E, fmt, 8))
        graphs.append(g)
        streams.append(torch.cuda.Stream(DEV))
    for trial in range(3):
        for i in range(2):
            ins[i][0].copy_(routing(T, K, E, 100 * trial + i, dropped=0.3 * trial))
            ins[i][1].copy_(randn((T, M), 200 * trial + i))
        torch.cuda.synchronize()
        for _ in range(3):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            same(outs[i], small_step(*ins[i], E, fmt, 8))


def test_results_do_not_depend_on_the_run():
    e, x, g = routing(5000, 8, 64, 3), randn((5000, 520), 4, torch.bfloat16), \
        randn((5000, 520), 5, torch.bfloat16)
    w = torch.rand(5000, 8, generator=gen(6), device=DEV)
    one = small_step(e, x, g, w, 64, "e4m3", 4)
    for _ in range(3):
        same(one, small_step(e, x, g, w, 64, "e4m3", 4))


def test_other_streams():
    """Each call on a stream given by `stream`, behind work of that stream that
    has not run yet; nothing on the current stream orders them."""
    T, K, E, M = 3000, 4, 32, 256
    e0, x0, g0 = routing(T, K, E, 1), randn((T, M), 2, torch.bfloat16), \
        randn((T, M), 3, torch.bfloat16)
    w = torch.rand(T, K, generator=gen(4), device=DEV)
    want = small_step(e0, x0, g0, w, E, "int8", 4)
    side = torch.cuda.Stream(DEV)
    e, x = torch.zeros_like(e0), torch.zeros_like(x0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        e.copy_(e0)
        x.copy_(x0)
    kw = dict(stream=side)
    plan = vf.expert_plan(e, E, align=4, **kw)
    packed, c1, s1 = vf.expert_pack_q(x, plan, "int8", 64, **kw)
    y = vf.expert_restore_q(c1, s1, plan, "int8", 64, **kw)
    merged, c2, s2 = vf.expert_merge_q(y, plan, w, "int8", 64, **kw)
    gp, gw = vf.expert_merge_backward_q(g0, c2, s2, plan, w, "int8", 64, **kw)
    gx = vf.expert_merge(gp, plan, **kw)
    plain = vf.expert_pack(x, plan, **kw)
    gp2, gw2 = vf.expert_merge_backward(g0, y, plan, w, **kw)
    side.synchronize()
    got = (plan, packed, c1, s1, y, merged, c2, s2, gp, gw, gx, plan.slot_of >= 0)
    same(got, want)
    owned = plan.slot_of >= 0
    assert torch.equal(plain[owned], packed[owned]) and torch.equal(gp2[owned], gp[owned])


def test_host_threads():
    T, K, E, M = 1500, 3, 24, 200
    cases = [(routing(T, K, E, i), randn((T, M), i, torch.bfloat16),
              randn((T, M), 50 + i, torch.bfloat16),
              torch.rand(T, K, generator=gen(i), device=DEV)) for i in range(6)]
    want = [small_step(*c, E, "e4m3", 2) for c in cases]
    torch.cuda.synchronize()
    got, errors = [None] * 6, []

    def work(i):
        try:
            s = torch.cuda.Stream(DEV)
            with torch.cuda.stream(s):
                for _ in range(5):
                    got[i] = small_step(*cases[i], E, "e4m3", 2)
            s.synchronize()
        except Exception as ex:                       # reported by the main thread
            errors.append(ex)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, want):
        same(a, b)


def test_host_threads_with_plans_of_all_sizes():
    """Plans whose kernels need different amounts of shared memory, at the same time:
    none lowers what another has asked for."""
    sizes = [(3000, 4, 4096), (4000, 4, 900), (2000, 8, 600), (2500, 4, 2048), (60, 8, 4096),
             (9000, 2, 1024)]
    cases = [routing(T, K, E, i) for i, (T, K, E) in enumerate(sizes)]
    want = [[t.clone() for t in vf.expert_plan(e, s[2])[:4]] for e, s in zip(cases, sizes)]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(i):
        try:
            s = torch.cuda.Stream(DEV)
            with torch.cuda.stream(s):
                for _ in range(200):
                    got = vf.expert_plan(cases[i], sizes[i][2])
                s.synchronize()
                wrong.extend(i for a, b in zip(got, want[i]) if not torch.equal(a, b))
        except Exception as ex:                       # reported by the main thread
            errors.append(ex)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    assert not wrong, wrong


def test_pinned_host_rows():
    e = routing(40, 2, 5, 1)
    plan = vf.expert_plan(e, 5)
    x = randn((40, 64), 2, torch.bfloat16)
    px = x.cpu().pin_memory()
    owned = plan.slot_of >= 0
    want = vf.expert_pack(x, plan)
    got = vf.expert_pack(px, plan)
    torch.cuda.synchronize()
    assert not got.is_cuda and torch.equal(got[owned.cpu()], want[owned].cpu())
    back = vf.expert_merge(got, plan)
    torch.cuda.synchronize()
    assert torch.equal(back, vf.expert_merge(want, plan).cpu())


# ---- offsets past 2^31 ------------------------------------------------------------

def test_offsets_past_31_bits():
    T, K, E, M = 36000, 8, 16, 8192                    # 288,000 rows, 2.36e9 elements
    e = routing(T, K, E, 1, dropped=0.0)
    plan = vf.expert_plan(e, E)
    assert plan.slot_of.numel() * M > 2 ** 31
    x = torch.empty(T, M, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(2))
    packed, codes, scales = vf.expert_pack_q(x, plan, "int8")
    far = torch.arange(plan.slot_of.numel() - 3000, plan.slot_of.numel(), device=DEV)
    token = (plan.slot_of[far] // K).long()
    assert torch.equal(packed[far], x[token])
    back = vf.expert_restore_q(codes, scales, plan, "int8")
    v = codes[token].float() * scales[token].repeat_interleave(128, 1)
    assert torch.equal(back[far], v.to(torch.bfloat16))
    del back
    w = torch.rand(T, K, generator=gen(3), device=DEV)
    out, c2, s2 = vf.expert_merge_q(packed, plan, w, "e4m3")
    assert c2.numel() > 2 ** 31
    some = token.unique()[:500]
    # all K rows of a token are its own row: its sum is x times the weights' sum
    want = x[some].double() * w[some].double().sum(1, keepdim=True)
    mag = x[some].double().abs() * w[some].double().sum(1, keepdim=True)
    within(out[some], want, gamma(K) * mag + (want.abs() + gamma(K) * mag) * 2.0 ** -8)
    values = c2[far].float() * s2[far].repeat_interleave(128, 1)
    # E4M3: half a step is 2^-4 of the value, or 2^-10 of the group's top over 448
    top = packed[far].float().view(len(far), -1, 128).abs().amax(2).repeat_interleave(128, 1)
    near = packed[far].float().abs() / 16 + top / 448 / 1024 + top * 2.0 ** -20
    assert ((values - packed[far].float()).abs() <= near).all()
    gp, gw = vf.expert_merge_backward_q(x, c2, s2, plan, w, "e4m3")
    k = (plan.slot_of[far] % K).long()
    want = w[token, k].double()[:, None] * x[token].double()
    within(gp[far], want, want.abs() * (U + 2.0 ** -8 * (1 + U)) + 2.0 ** -133)
    want = (x[token].double() * values.double()).sum(1)
    within(gw[token, k], want, gamma(M + 1) * (x[token].double() * values.double()).abs().sum(1))
    gp2, gw2 = vf.expert_merge_backward(x, packed, plan, w, grad_packed=gp)
    want = (x[token].double() ** 2).sum(1)
    within(gw2[token, k], want, gamma(M) * want)
    plain = vf.expert_merge(packed, plan)
    want = x[some].double() * K
    within(plain[some], want, want.abs() * (gamma(K) + 2.0 ** -8 * (1 + gamma(K))))


def test_token_view_past_31_bits():
    T, M, stride = 40000, 64, 60000                    # 2.4e9 elements from end to end
    base = torch.zeros(T * stride, dtype=torch.bfloat16, device=DEV)
    view = base.as_strided((T, M), (stride, 1))
    x = randn((T, M), 1, torch.bfloat16)
    view.copy_(x)
    plan = vf.expert_plan(routing(T, 2, 8, 2, dropped=0.0), 8)
    assert torch.equal(vf.expert_pack(view, plan), vf.expert_pack(x, plan))
    packed = vf.expert_pack(x, plan)
    view.zero_()
    vf.expert_merge(packed, plan, out=view)
    assert torch.equal(view, vf.expert_merge(packed, plan))


@pytest.mark.parametrize("E", [3, 4096])
def test_most_slots(E):
    """T*K = 2^30, the limit: the plan is checked in full (each slot has its row, in
    slot order within its expert), the rows of a pack and a merge at places."""
    T, K, M = 1 << 27, 8, 8
    e = torch.randint(0, E, (T, K), generator=gen(E), device=DEV, dtype=torch.int32)
    plan = vf.expert_plan(e, E)
    counts = torch.bincount(e.view(-1), minlength=E)
    assert torch.equal(plan.counts.long(), counts)
    assert torch.equal(plan.offsets.long()[1:], counts.cumsum(0))
    step = 1 << 26
    for i in range(0, T * K, step):
        rows = plan.row_of.view(-1)[i:i + step].long()
        assert torch.equal(plan.slot_of[rows],
                           torch.arange(i, i + step, device=DEV, dtype=torch.int32))
        chosen = e.view(-1)[i:i + step].long()
        assert ((rows >= plan.offsets[chosen]) & (rows < plan.offsets[chosen + 1])).all()
        slots = plan.slot_of[i:i + step]
        falls = (slots[1:] < slots[:-1]).nonzero()[:, 0] + i + 1
        assert torch.isin(falls, plan.offsets.long()).all()
    x = torch.empty(T, M, dtype=torch.bfloat16, device=DEV).normal_(generator=gen(1))
    packed = vf.expert_pack(x, plan)
    some = torch.randint(0, T * K, (1 << 20,), generator=gen(2), device=DEV)
    some[:1000] = torch.arange(T * K - 1000, T * K, device=DEV)
    assert torch.equal(packed[some], x[(plan.slot_of[some] // K).long()])
    merged = vf.expert_merge(packed, plan)
    t = (some // K)
    want = x[t].double() * K                               # eight times the same value: exact
    within(merged[t], want, want.abs() * 2.0 ** -8)


# ---- random cases -------------------------------------------------------------------

def reference(plan, K):
    rows = plan.slot_of.numel()
    owned = plan.slot_of >= 0
    slot = plan.slot_of.clamp(min=0).long()
    return rows, owned, slot // K, slot % K


@pytest.mark.parametrize("seed", range(30))
def test_random_cases(seed):
    g = torch.Generator().manual_seed(1000 + seed)

    def pick(*xs):
        return xs[int(torch.randint(0, len(xs), (1,), generator=g))]

    def upto(n):
        return int(torch.randint(1, n + 1, (1,), generator=g))

    K = pick(1, 2, 3, 4, 6, 8, 13)
    E = max(K, upto(pick(4, 40, 600)))
    T, M, align = upto(pick(3, 70, 3000)), pick(upto(50), upto(1200), 8 * upto(150), 4 * upto(90)), \
        pick(1, 1, 4, 128)
    dtype = pick(*DTYPES)
    e = routing(T, K, E, seed, dropped=pick(0.0, 0.2, 1.0))
    pad = pick(0, 0, 8, 3)

    def view(s):
        v = torch.empty(T, M + pad, dtype=dtype, device=DEV)[:, :M]
        return v.copy_(randn((T, M), s, dtype))

    plan = vf.expert_plan(e, E, align=align)
    rows, owned, token, k = reference(plan, K)
    there = (plan.row_of >= 0)
    used = int(plan.offsets[-1])
    x, grad, w = view(seed), view(seed + 1), torch.rand(T, K, generator=gen(seed), device=DEV)
    eps = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * eps

    packed = vf.expert_pack(x, plan, out=torch.full((rows, M), 7.0, dtype=dtype, device=DEV))
    assert torch.equal(packed[owned], x[token[owned]])
    assert (packed[:used][~owned[:used]] == 0).all() and (packed[used:] == 7).all()

    y = randn((rows, M), seed + 2, dtype)
    y[~owned] = float("nan")
    yd = torch.nan_to_num(y.double())[plan.row_of.clamp(min=0).long()] * there[:, :, None]
    for weights in (None, w):
        terms = yd * (1.0 if weights is None else weights.double()[:, :, None])
        want, mag = terms.sum(1), terms.abs().sum(1)
        out = vf.expert_merge(y, plan, weights, out=view(0))
        s = gamma(K) * mag
        within(out, want, s + (want.abs() + s) * eps + tiny, "merge")

    gp, gw = vf.expert_merge_backward(grad, y, plan, w, grad_packed=torch.full(
        (rows, M), 7.0, dtype=dtype, device=DEV))
    want = w.double()[token, k][:, None] * grad.double()[token]
    within(gp[owned], want[owned], want[owned].abs() * (U + eps * (1 + U)) + tiny, "rows")
    assert (gp[:used][~owned[:used]] == 0).all() and (gp[used:] == 7).all()
    terms = grad.double()[:, None, :] * yd
    within(gw, terms.sum(2), gamma(M) * terms.abs().sum(2), "weights")


# ---- refusals that need device tensors ------------------------------------------------

def test_binding_checks_shapes_and_types():
    plan = vf.expert_plan(routing(6, 2, 4, 1, dropped=0.0), 4)
    x = randn((6, 32), 1, torch.bfloat16)
    packed = vf.expert_pack(x, plan)
    w = torch.ones(6, 2, device=DEV)
    bad = [
        lambda: vf.expert_plan(torch.zeros(6, 2, device=DEV), 4),              # float indices
        lambda: vf.expert_plan(torch.zeros(6, dtype=torch.int64, device=DEV), 4),
        lambda: vf.expert_plan(torch.zeros(5, 2, dtype=torch.int64, device=DEV), 4, out=plan),
        lambda: vf.expert_plan(torch.zeros(6, 2, dtype=torch.int64, device=DEV), 4, align=2,
                               out=plan),
        lambda: vf.expert_pack(x[:5], plan),
        lambda: vf.expert_pack(x.double(), plan),
        lambda: vf.expert_pack(x[0], plan),
        lambda: vf.expert_pack(x, plan, out=packed[:, :16]),
        lambda: vf.expert_pack(x, plan, out=packed.float()),
        lambda: vf.expert_pack(x, plan._replace(row_of=plan.row_of.long())),
        lambda: vf.expert_pack(x, plan._replace(offsets=plan.offsets[:4])),
        lambda: vf.expert_pack(x, plan._replace(row_of=plan.row_of.t())),
        lambda: vf.expert_merge(packed[:-1], plan),
        lambda: vf.expert_merge(packed.t().contiguous().t(), plan),            # rows not contiguous
        lambda: vf.expert_merge(packed, plan, w.half()),
        lambda: vf.expert_merge(packed, plan, w[:, :1]),
        lambda: vf.expert_merge(packed, plan, out=x.float()),
        lambda: vf.expert_merge_backward(x, packed, plan, None),
        lambda: vf.expert_merge_backward(x, packed.float(), plan, w),
        lambda: vf.expert_merge_backward(x, packed, plan, w, grad_weights=w.double()),
        lambda: vf.expert_pack_q(x, plan, group=48),
        lambda: vf.expert_pack_q(x.half(), plan),
        lambda: vf.expert_restore_q(torch.zeros(6, 32, dtype=torch.int8, device=DEV),
                                    torch.zeros(6, 1, device=DEV), plan, "e4m3"),
        lambda: vf.expert_restore_q(torch.zeros(6, 32, dtype=torch.int8, device=DEV),
                                    torch.zeros(6, 2, device=DEV), plan, "int8"),
        lambda: vf.expert_restore_q(torch.zeros(6, 32, dtype=torch.int8, device=DEV), None, plan,
                                    "int8"),
        lambda: vf.expert_merge_backward_q(x, None, None, plan, w),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("case %d was accepted" % i)


def test_library_refuses_overlaps():
    plan = vf.expert_plan(routing(6, 2, 4, 1, dropped=0.0), 4)
    buf = torch.zeros(12 + 6, 32, device=DEV)
    with pytest.raises(vf.VFError, match="overlap"):
        vf.expert_pack(buf[8:14], plan, out=buf[:12])
    with pytest.raises(vf.VFError, match="overlap"):
        vf.expert_merge(buf[:12], plan, out=buf[11:17])
    with pytest.raises(vf.VFError, match="overlap"):
        vf.expert_merge_backward(buf[12:18], buf[:12], plan, torch.ones(6, 2, device=DEV),
                                 grad_packed=buf[:12])
    with pytest.raises(vf.VFError):                        # a written view over itself
        vf.expert_merge(buf[:12], plan, out=torch.zeros(32, device=DEV).expand(6, 32))
    assert (buf == 0).all()


def test_no_tokens_and_no_rows():
    empty = vf.expert_plan(torch.empty(0, 2, dtype=torch.int64, device=DEV), 4, align=8)
    x = torch.empty(0, 32, dtype=torch.bfloat16, device=DEV)
    w = torch.empty(0, 2, device=DEV)
    assert vf.expert_pack(x, empty).shape == (0, 32)
    assert vf.expert_merge(vf.expert_pack(x, empty), empty, w).shape == (0, 32)
    gp, gw = vf.expert_merge_backward(x, vf.expert_pack(x, empty), empty, w)
    assert gp.shape == (0, 32) and gw.shape == (0, 2)
    packed, codes, scales = vf.expert_pack_q(x, empty)
    assert vf.expert_restore_q(codes, scales, empty).shape == (0, 32)
    # a plan without rows: every slot is dropped
    i32 = dict(dtype=torch.int32, device=DEV)
    for M in (32, 33):
        none = vf.ExpertPlan(torch.zeros(5, 2, **i32), torch.empty(0, **i32),
                             torch.zeros(4, **i32), torch.zeros(5, **i32), 2)
        x = randn((5, M), 1, torch.bfloat16)
        w = torch.ones(5, 2, device=DEV)
        p = vf.expert_pack(x, none)
        assert p.shape == (0, M)
        assert (vf.expert_merge(p, none, w) == 0).all()
        assert (vf.expert_merge_backward(x, p, none, w)[1] == 0).all()
        out, codes, scales = vf.expert_merge_q(p, none, w, "int8", 32)
        assert (out == 0).all()
        assert (vf.expert_merge_backward_q(x, codes, scales, none, w, "int8", 32)[1] == 0).all()
