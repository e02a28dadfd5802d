"""Performance cases of a mixture-of-experts layer's own arithmetic: the products
of the experts' rows with their weights, the gated activation between them, and
the root-mean-square norm in front.

Notation: T tokens, K routing slots per token, E experts.  ``offsets[e]`` is the
first row of expert e in the expert-major buffers of R rows, ``counts[e]`` the
number of its rows; the gap rows up to ``offsets[e + 1]`` hold no slot and are
written as zeros, the rows behind the last expert are left as they were.

Every case is a single pass of one operator:

``product``      out[r, n] = sum_k rows[r, k] * weights[e(r), n, k];
``product_grad`` its gradient to the rows: the product with the weights transposed;
``weight_grad``  its gradient to the weights: for each expert the sum over its
                 rows of grad[r, n] * rows[r, k];
``glu``          out = silu(gate) * up, of the two halves of a product's rows;
``glu_grad``     its gradients to gate and up;
``norm``         total = x + residual, out = total / rms(total) * weight;
``norm_q``       the same to 8-bit codes with a scale for each group of 128
                 columns, and the codes sent to the expert rows of a top-1 routing;
``norm_grad``    its gradients to x and to the weight.

With ``own`` false each pass is computed in plain torch operations, with
``own`` true by this package's calls.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_TOP = {"int8": 127.0, "e4m3": 448.0}
_GROUP = 128
_FLOOR = 2.0 ** -96          # a group whose largest magnitude is below is sent as zeros
_EPS = 1e-6


def _expert_case(name, kind, T, K, E, N, M, dtype="bf16", align=1, drop=False, out="same"):
    """N, M: the product's output and input features (glu: M columns, N unused)."""
    c = {"kind": kind, "T": T, "K": K, "E": E, "N": N, "M": M, "dtype": dtype, "align": align,
         "drop": drop, "out": out}
    if name:
        c["name"] = name
    return c


def _norm_case(name, kind, T, M, dtype="bf16", residual=True, weight="same", fmt="none"):
    c = {"kind": kind, "T": T, "M": M, "dtype": dtype, "residual": residual, "weight": weight,
         "fmt": fmt}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # serving, one new token: the weights of its eight experts are read once
        _expert_case("product_token", "product", 1, 8, 128, 2048, 4096),
        # serving, a batch of 64 new tokens, the experts' second product
        _expert_case("product_batch", "product", 64, 4, 64, 3584, 2048, "fp16", drop=True),
        # a training step's forward pass at the representative sequence length
        _expert_case("product_long", "product", 55414, 2, 16, 4096, 3584, align=128, drop=True),
        # the rows' gradient on a shorter batch with many experts, segments not aligned
        _expert_case("product_grad_4k", "product_grad", 4096, 8, 64, 4096, 2048, drop=True),
        # the weights' gradient of the same batch, kept in 32 bits for accumulation
        _expert_case("weight_grad_4k", "weight_grad", 4096, 8, 32, 4096, 2048, align=128,
                     out="fp32"),
        # the same at ragged lengths and features in no whole tiles
        _expert_case("weight_grad_ragged", "weight_grad", 8191, 2, 8, 3584, 2000, "fp16",
                     drop=True),
        # serving, a batch of 64 new tokens
        _expert_case("glu_batch", "glu", 64, 8, 128, 1, 2048),
        # a training step's backward pass at the representative sequence length
        _expert_case("glu_grad_long", "glu_grad", 55414, 2, 16, 1, 2048, align=128, drop=True),
        # serving, one new token
        _norm_case("norm_token", "norm", 1, 4096),
        # a training step at the representative sequence length
        _norm_case("norm_long", "norm", 55414, 3584),
        # the same with the normalised rows kept in E4M3 and dispatched from there
        _norm_case("norm_q_long", "norm_q", 55414, 3584, fmt="e4m3"),
        # the norm's backward pass at a ragged length, master activations in 32 bits
        _norm_case("norm_grad_ragged", "norm_grad", 55413, 2048, "fp32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _features(rng):
    if rng.random() < 0.25:
        return _log_int(rng, 33, 4096)                     # odd row lengths among them
    return rng.randint(1, 32) * rng.choice([64, 96, 128])


def draw(rng):
    kind = rng.choice(["product", "product", "product_grad", "weight_grad", "glu", "glu_grad",
                       "norm", "norm_q", "norm_grad"])
    if kind.startswith("norm"):
        dtype = "bf16" if kind == "norm_q" else rng.choice(["bf16", "bf16", "fp16", "fp32"])
        c = _norm_case(None, kind, _log_int(rng, 1, 55414), _features(rng), dtype,
                       rng.random() < 0.7, rng.choice(["same", "fp32"]),
                       rng.choice(["int8", "e4m3"]) if kind == "norm_q" else "none")
    else:
        glu = kind.startswith("glu")
        dtype = rng.choice(["bf16", "fp16", "fp32"] if glu else ["bf16", "fp16"])
        T, K = _log_int(rng, 1, 55414), rng.choice([1, 2, 3, 4, 6, 8])
        c = _expert_case(None, kind, T, K, max(K, _log_int(rng, 2, 256)),
                         1 if glu else _features(rng), _features(rng), dtype,
                         rng.choice([1, 1, 8, 16, 128]), T > 4 and rng.random() < 0.5,
                         "fp32" if kind == "weight_grad" and rng.random() < 0.5 else "same")
        while not glu and c["E"] * c["N"] * c["M"] > 1 << 30 and c["E"] > K:
            c["E"] = max(K, c["E"] // 2)
    most = {k: 0.8 * max(work(x)[k] for x in listed()) for k in ("bytes", "flops")}
    while c["T"] > 8 and any(work(c)[k] > most[k] for k in most):
        c["T"] = c["T"] * 2 // 3
    return c


def _dropped(case):
    """Slots dropped: whole tokens at the end (padding), and every 50th slot."""
    T, K = case["T"], case["K"]
    if not case["drop"]:
        return 0, 0
    pad_tokens = T // 64
    return pad_tokens, ((T - pad_tokens) * K + 49) // 50


def work(case):
    kind, T, M, b = case["kind"], case["T"], case["M"], _BYTES[case["dtype"]]
    if kind.startswith("norm"):
        row, extra = T * M * b, 1 if case["residual"] else 0
        w = M * (4 if case["weight"] == "fp32" else b)
        if kind == "norm":                                 # x (and residual), out (and total)
            return {"bytes": (2 + 2 * extra) * row + w, "flops": (4 + extra) * T * M}
        if kind == "norm_grad":                            # grad, total (and its gradient), grad_x
            return {"bytes": (3 + extra) * row + w + 4 * M, "flops": (9 + extra) * T * M}
        kept = T * M + 4 * T * -(-M // _GROUP)             # codes and scales, written and read
        return {"bytes": (2 + 2 * extra) * row + w + 2 * kept + 8 * T,
                "flops": (8 + extra) * T * M}
    pad_tokens, slots = _dropped(case)
    R = (T - pad_tokens) * case["K"] - slots               # rows that hold a token
    N, E = case["N"], case["E"]
    plan = 4 * (2 * E + 1)
    if kind == "glu":
        return {"bytes": 3 * R * M * b + 4 * R, "flops": 5 * R * M}
    if kind == "glu_grad":
        return {"bytes": 5 * R * M * b + 4 * R, "flops": 12 * R * M}
    touched = min(E, R)                                    # at most: others are not read
    if kind == "weight_grad":
        out = 4 if case["out"] == "fp32" else b
        return {"bytes": plan + R * (N + M) * b + E * N * M * out, "flops": 2 * R * N * M}
    return {"bytes": plan + R * (N + M) * b + touched * N * M * b, "flops": 2 * R * N * M}


# ---- inputs ------------------------------------------------------------------

def _routing(case, gen, device):
    """Experts [T, K]: popular and rare ones, no expert twice for a token, dropped
    slots."""
    T, K, E = case["T"], case["K"], case["E"]
    bias = -0.25 * torch.log1p(torch.arange(E, device=device, dtype=torch.float32))
    bias = bias[torch.randperm(E, generator=gen, device=device)]
    experts = torch.topk(torch.randn(T, E, generator=gen, device=device) + bias, K, dim=1).indices
    pad_tokens, slots = _dropped(case)
    if pad_tokens:
        experts[T - pad_tokens:] = -1
    if slots:
        experts = experts.contiguous()
        experts.view(-1)[:(T - pad_tokens) * K:50] = -1
    return experts


def _plan(experts, E, align):
    """row_of, slot_of, counts, offsets (int32) by a stable sort of the slots."""
    T, K = experts.shape
    rows = T * K + min(E, T * K) * (align - 1)
    flat = experts.reshape(-1).to(torch.int64)
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    kept = counts[:E]
    zero = torch.zeros(1, dtype=torch.int64, device=flat.device)
    offsets = torch.cat([zero, torch.cumsum((kept + align - 1) // align * align, 0)])
    first = torch.cat([zero, torch.cumsum(counts, 0)])[:E + 1]
    order = torch.argsort(key, stable=True)
    expert = key[order]
    row = torch.where(expert < E, offsets[expert] + torch.arange(T * K, device=flat.device) -
                      first[expert], -1)
    row_of = torch.empty_like(flat)
    row_of[order] = row
    slot_of = torch.full((rows + 1,), -1, dtype=torch.int64, device=flat.device)
    slot_of[torch.where(row < 0, rows, row)] = torch.where(row < 0, -1, order)
    return (row_of.view(T, K).to(torch.int32), slot_of[:rows].to(torch.int32),
            kept.to(torch.int32), offsets.to(torch.int32))


def _activations(shape, dtype, gen, device):
    """Rows of N(0, 1) with a few channels 20 times larger, as hidden states have."""
    x = torch.empty(shape, dtype=dtype, device=device).normal_(generator=gen)
    x[..., 5::509] *= 20
    return x


def _expert_rows(shape, dtype, gen, device, slot_of):
    """Activations; what no slot owns is never read."""
    x = _activations(shape, dtype, gen, device)
    x[slot_of < 0] = float("nan")
    return x


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(int(seed))
    kind, T, M, dtype = case["kind"], case["T"], case["M"], _DTYPES[case["dtype"]]
    s = {"case": case}
    if kind.startswith("norm"):
        s["x"] = _activations((T, M), dtype, gen, device)
        w = torch.rand(M, generator=gen, device=device) + 0.5
        s["weight"] = w if case["weight"] == "fp32" else w.to(dtype)
        s["residual"] = _activations((T, M), dtype, gen, device) if case["residual"] else None
        if kind == "norm_grad":
            s["grad"] = torch.empty((T, M), dtype=dtype, device=device).normal_(generator=gen)
        if kind == "norm_q":
            experts = torch.randint(0, 16, (T, 1), generator=gen, device=device)
            s["plan"] = _plan(experts, 16, 1)
            s["out"] = torch.zeros((T, M), dtype=dtype, device=device)
        return s
    K, E, N, align = case["K"], case["E"], case["N"], case["align"]
    s["plan"] = _plan(_routing(case, gen, device), E, align)
    slot_of, counts, offsets = s["plan"][1:]
    # a user of a plain loop over the experts has the segments on the host
    s["segments"] = list(zip(offsets.tolist(), counts.tolist()))
    rows = slot_of.numel()
    if kind in ("glu", "glu_grad"):
        both = _expert_rows((rows, 2 * M), dtype, gen, device, slot_of)
        s["gate"], s["up"] = both[:, :M], both[:, M:]
        if kind == "glu":
            s["out"] = torch.zeros((rows, M), dtype=dtype, device=device)
        else:
            s["grad"] = _expert_rows((rows, M), dtype, gen, device, slot_of)
            s["out"] = torch.zeros((rows, 2 * M), dtype=dtype, device=device)
        return s
    if kind != "product_grad":
        s["rows"] = _expert_rows((rows, M), dtype, gen, device, slot_of)
    if kind != "product":
        s["grad"] = _expert_rows((rows, N), dtype, gen, device, slot_of)
    if kind != "weight_grad":
        s["weights"] = torch.empty((E, N, M), dtype=dtype, device=device).normal_(generator=gen)
        s["weights"] *= M ** -0.5
        s["out"] = torch.zeros((rows, N if kind == "product" else M), dtype=dtype, device=device)
    return s


# ---- the plain forms ---------------------------------------------------------

def _plain_product(rows, weights, segments, like):
    """rows times each expert's [in, out] weights."""
    out = torch.zeros_like(like)
    for e, (at, n) in enumerate(segments):
        if n:
            out[at:at + n] = (rows[at:at + n].float() @ weights[e].float()).to(out.dtype)
    return out


def _plain_weight_grad(grad, rows, segments, dtype):
    out = torch.zeros((len(segments), grad.shape[1], rows.shape[1]), dtype=dtype,
                      device=grad.device)
    for e, (at, n) in enumerate(segments):
        if n:
            out[e] = (grad[at:at + n].float().t() @ rows[at:at + n].float()).to(dtype)
    return out


def _plain_glu(gate, up, slot_of):
    g = gate.float()
    y = g / (1.0 + torch.exp(-g)) * up.float()
    return torch.where((slot_of >= 0)[:, None], y, 0).to(gate.dtype)


def _plain_glu_grad(grad, gate, up, slot_of):
    d, g, u = grad.float(), gate.float(), up.float()
    s = 1.0 / (1.0 + torch.exp(-g))
    both = torch.cat([d * u * s * (1.0 + g * (1.0 - s)), d * g * s], dim=1)
    return torch.where((slot_of >= 0)[:, None], both, 0).to(gate.dtype)


def _plain_total(x, residual):
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def _plain_norm(total, weight):
    h = total.float()
    return h * (1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + _EPS)) * weight.float()


def _plain_norm_grad(grad, total, weight, grad_total):
    h, g = total.float(), grad.float()
    r = 1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + _EPS)
    wg = g * weight.float()
    dx = r * (wg - h * (r * r * (wg * h).mean(dim=1, keepdim=True)))
    if grad_total is not None:
        dx = dx + grad_total.float()
    # the sum over all tokens in 64 bits
    return dx.to(grad.dtype), (g * h * r).sum(dim=0, dtype=torch.float64).float()


def _plain_kept(y, fmt):
    """The values that 8-bit codes of y and their scales stand for; the row is
    padded with zeros to whole groups."""
    rows, M = y.shape
    groups, top = -(-M // _GROUP), _TOP[fmt]
    y = torch.nn.functional.pad(y, (0, groups * _GROUP - M)).view(rows, groups, _GROUP)
    amax = y.abs().amax(dim=2, keepdim=True)
    live = amax >= _FLOOR
    safe = torch.where(live, amax, 1.0)
    top = torch.full_like(safe, top)             # a scalar here would divide in two roundings
    q = torch.where(live, y * (top / safe), 0)
    codes = torch.round(q).clamp(-127, 127) if fmt == "int8" else \
        q.to(torch.float8_e4m3fn).float()
    return (codes * torch.where(live, safe / top, 0)).view(rows, -1)[:, :M]


def _run_plain(s):
    case = s["case"]
    kind, dtype = case["kind"], _DTYPES[case["dtype"]]
    if kind == "product":
        return _plain_product(s["rows"], s["weights"].transpose(1, 2), s["segments"], s["out"])
    if kind == "product_grad":
        return _plain_product(s["grad"], s["weights"], s["segments"], s["out"])
    if kind == "weight_grad":
        return _plain_weight_grad(s["grad"], s["rows"], s["segments"],
                                  torch.float32 if case["out"] == "fp32" else dtype)
    if kind == "glu":
        return _plain_glu(s["gate"], s["up"], s["plan"][1])
    if kind == "glu_grad":
        return _plain_glu_grad(s["grad"], s["gate"], s["up"], s["plan"][1])
    if kind == "norm_grad":
        return _plain_norm_grad(s["grad"], s["x"], s["weight"], s["residual"])
    total = _plain_total(s["x"], s["residual"])
    y = _plain_norm(total, s["weight"])
    if kind == "norm":
        return (y.to(dtype), total) if case["residual"] else y.to(dtype)
    rows = _plain_kept(y, case["fmt"]).to(dtype)[s["plan"][1].long()]
    return (rows, total) if case["residual"] else rows


# ---- the package's calls -----------------------------------------------------

def _run_own(s):
    import sequence_head_relayout_gb300 as vf
    case = s["case"]
    kind, dtype = case["kind"], _DTYPES[case["dtype"]]
    if kind == "norm":
        return vf.rms_norm(s["x"], s["weight"], eps=_EPS, residual=s["residual"])
    if kind == "norm_grad":
        # the gradient that reaches the total by the residual path is at hand too
        return vf.rms_norm_backward(s["grad"], s["x"], s["weight"], eps=_EPS,
                                    grad_total=s["residual"])
    plan = vf.ExpertPlan(*s["plan"], case.get("align", 1))
    if kind == "norm_q":
        codes, scales, *total = vf.rms_norm_q(s["x"], s["weight"], eps=_EPS, fmt=case["fmt"],
                                              group=_GROUP, residual=s["residual"])
        rows = vf.expert_restore_q(codes, scales, plan, case["fmt"], _GROUP, out=s["out"])
        return (rows, *total) if total else rows
    if kind == "product":
        return vf.expert_product(s["rows"], s["weights"], plan, out=s["out"])
    if kind == "product_grad":
        return vf.expert_product(s["grad"], s["weights"].transpose(1, 2), plan, out=s["out"])
    if kind == "weight_grad":
        return vf.expert_weight_grad(s["grad"], s["rows"], plan,
                                     dtype=torch.float32 if case["out"] == "fp32" else dtype)
    if kind == "glu":
        return vf.expert_glu(s["gate"], s["up"], plan, out=s["out"])
    M, both = case["M"], s["out"]
    vf.expert_glu_backward(s["grad"], s["gate"], s["up"], plan, grad_gate=both[:, :M],
                           grad_up=both[:, M:])
    return both


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definitions in 64 bits ----------------------------------------------

def _exact_owner(offsets, counts, rows):
    """Each row's expert, -1 for gap rows and the rows behind."""
    at = torch.arange(rows, device=offsets.device)
    e = torch.searchsorted(offsets[1:].long().contiguous(), at, right=True)
    e = e.clamp(max=counts.numel() - 1)
    there = at - offsets[e].long() < counts[e].long()
    return torch.where(there, e, torch.full_like(e, -1))


def _exact_product(rows, weights, plan, transposed):
    owner = _exact_owner(plan[3], plan[2], rows.shape[0])
    out = torch.zeros((rows.shape[0], weights.shape[2 if transposed else 1]),
                      dtype=torch.float64, device=rows.device)
    for e in owner.unique().tolist():
        if e >= 0:
            w = weights[e].double()
            mine = (owner == e).nonzero()[:, 0]
            out[mine] = torch.einsum("rn,nm->rm" if transposed else "rm,nm->rn",
                                     rows[mine].double(), w)
    return out


def _exact_weight_grad(grad, rows, plan):
    owner = _exact_owner(plan[3], plan[2], rows.shape[0])
    out = torch.zeros((plan[2].numel(), grad.shape[1], rows.shape[1]), dtype=torch.float64,
                      device=rows.device)
    for e in owner.unique().tolist():
        if e >= 0:
            mine = (owner == e).nonzero()[:, 0]
            out[e] = torch.einsum("rn,rm->nm", grad[mine].double(), rows[mine].double())
    return out


def _in_chunks(n, size, one, outs):
    """Fills `outs` (tensors of n rows) with one(rows), `size` rows at a time."""
    for at in range(0, n, size):
        mine = slice(at, min(n, at + size))
        for out, value in zip(outs, one(mine)):
            out[mine] = value
    return outs


def _exact_glu(s, backward):
    gate, up = s["gate"], s["up"]
    rows, M = gate.shape
    there = _exact_owner(s["plan"][3], s["plan"][2], rows) >= 0

    def one(mine):
        g, u = gate[mine].double(), up[mine].double()
        t = torch.tanh(g / 2)                              # sigmoid(g) = (1 + t) / 2
        act = g * (1 + t) / 2
        if not backward:
            v = act * u
        else:
            d = s["grad"][mine].double()
            slope = (1 + t) / 2 + g * (1 - t * t) / 4
            v = torch.cat([d * u * slope, d * act], dim=1)
        return [torch.where(there[mine, None], v, torch.zeros_like(v))]

    out = torch.zeros((rows, 2 * M if backward else M), dtype=torch.float64, device=gate.device)
    return _in_chunks(rows, 16384, one, [out])[0]


def _exact_norm(s, grad):
    x, other, w = s["x"], s["residual"], s["weight"].double()
    T, M = x.shape
    out, total = (torch.empty((T, M), dtype=torch.float64, device=x.device) for _ in range(2))
    dw = torch.zeros(M, dtype=torch.float64, device=x.device)

    def one(mine):
        h = x[mine].double()
        if other is not None and not grad:                 # the stored, rounded sum
            h = (h + other[mine].double()).to(x.dtype).double()
        r = torch.rsqrt(h.square().sum(dim=1, keepdim=True) / M + _EPS)
        n = h * r
        if not grad:
            return n * w, h
        g = s["grad"][mine].double()
        dw.add_((g * n).sum(dim=0))
        wg = g * w
        dx = r * (wg - n * ((wg * n).sum(dim=1, keepdim=True) / M))
        return (dx if other is None else dx + other[mine].double()), h

    _in_chunks(T, 16384, one, [out, total])
    return (out, dw) if grad else (out, total)


def _exact_kept(y, fmt):
    """The values that codes and scales of y stand for.  The format's steps are
    roundings to 32 bits; here all is in 64, so that a value next to a border
    between two codes may get the other one."""
    rows, M = y.shape
    top = _TOP[fmt]
    kept = torch.empty_like(y)
    for g in range(0, M, _GROUP):
        v = y[:, g:g + _GROUP]
        amax = v.abs().max(dim=1, keepdim=True).values
        safe = torch.where(amax >= _FLOOR, amax, torch.ones_like(amax))
        q = v * (top / safe)
        if fmt == "int8":
            code = torch.round(q).clamp(-127, 127)
        else:
            # a step of the E4M3 grid at q: 2^(floor(log2|q|) - 3), at least 2^-9
            exponent = (torch.frexp(q).exponent - 1).clamp(min=-6)
            # (built from its bits: a computed power could be one unit off)
            step = ((exponent.long() - 3 + 1023) << 52).view(torch.float64)
            code = (torch.round(q / step) * step).clamp(-448, 448)
        kept[:, g:g + _GROUP] = torch.where(amax >= _FLOOR, code * (safe / top),
                                            torch.zeros_like(code))
    return kept


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "product":
        return _exact_product(s["rows"], s["weights"], s["plan"], False)
    if kind == "product_grad":
        return _exact_product(s["grad"], s["weights"], s["plan"], True)
    if kind == "weight_grad":
        return _exact_weight_grad(s["grad"], s["rows"], s["plan"])
    if kind in ("glu", "glu_grad"):
        return _exact_glu(s, kind == "glu_grad")
    if kind == "norm_grad":
        return _exact_norm(s, True)
    out, total = _exact_norm(s, False)
    if kind == "norm_q":
        out = _exact_kept(out, case["fmt"])[s["plan"][1].long()]
    return (out, total) if case["residual"] else out
