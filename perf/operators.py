"""Performance cases of the expert relayouts: tokens sorted by expert, moved to
expert-major rows and back with their routing weights, the gradients, and the
8-bit checkpoints that the backward pass reads.

Notation: T tokens of M elements, K routing slots per token, E experts.  Slot
i = t*K + k belongs to token t.  A slot whose expert index lies outside [0, E)
is dropped.  ``row_of[t, k]`` is the slot's row in the expert-major buffer (-1
when dropped), ``slot_of[row]`` the inverse (-1 where no slot goes).  Each
expert's segment starts at a multiple of ``align``; the gap rows behind a
segment are written as zeros, the rows behind the last segment not at all.

Every case is a single pass of one operator:

``plan``         experts -> row_of, slot_of, counts, offsets;
``pack``         token rows -> expert-major rows;
``pack_grad``    its gradient: the sum of a token's expert rows;
``merge``        the weighted sum of a token's expert rows;
``merge_grad``   its gradients, to the expert rows and to the weights;
``pack_q``       the pack that keeps an 8-bit checkpoint of the token rows, and
                 the backward pass's use of it: the expert rows restored;
``merge_q``      the merge that keeps an 8-bit checkpoint of the expert rows,
                 and the backward pass that reads the codes.

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


def _case(name, kind, T, K, E, M, dtype="bf16", align=1, drop=False, pad=0, fmt="none"):
    c = {"kind": kind, "T": T, "K": K, "E": E, "M": M, "dtype": dtype, "align": align,
         "drop": drop, "pad": pad, "fmt": fmt}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # serving, one new token: the smallest call there is
        _case("plan_token", "plan", 1, 8, 256, 1),
        # a whole prompt or training batch, segments aligned for a tiled product
        _case("plan_large", "plan", 200000, 8, 256, 1, align=128, drop=True),
        # serving, a batch of 16 new tokens
        _case("pack_decode", "pack", 16, 8, 128, 4096),
        # a training step at the representative sequence length, aligned segments
        _case("pack_long", "pack", 55414, 8, 64, 3584, align=128, drop=True),
        # the pack's gradient at a ragged length, master gradients in 32 bits
        _case("pack_grad_ragged", "pack_grad", 55413, 2, 8, 2048, "fp32", drop=True),
        # serving, a batch of 64 new tokens
        _case("merge_decode", "merge", 64, 8, 256, 4096),
        # a training step's forward pass at the representative sequence length
        _case("merge_long", "merge", 55414, 8, 64, 3584, align=128, drop=True, pad=64),
        # its backward pass on a shorter batch, fp16
        _case("merge_grad_4k", "merge_grad", 4096, 8, 128, 4096, "fp16", drop=True),
        # checkpointed input rows: a short batch in E4M3, a long one in INT8
        _case("pack_q_4k", "pack_q", 4096, 8, 128, 4096, fmt="e4m3"),
        _case("pack_q_ragged", "pack_q", 55413, 2, 8, 2048, drop=True, align=16, fmt="int8"),
        # checkpointed expert rows, forward and backward pass
        _case("merge_q_4k", "merge_q", 4096, 4, 64, 4096, fmt="e4m3"),
        _case("merge_q_long", "merge_q", 55414, 4, 64, 3584, drop=True, align=128, fmt="int8"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["plan", "pack", "pack_grad", "merge", "merge_grad", "pack_q", "merge_q"])
    K = rng.choice([1, 2, 3, 4, 6, 8])
    E = max(K, _log_int(rng, 2, 512))
    align = rng.choice([1, 1, 8, 16, 128])
    drop = rng.random() < 0.5
    if kind == "plan":
        return _case(None, kind, _log_int(rng, 1, 200000), K, E, 1, align=align, drop=drop)
    quantised = kind.endswith("_q")
    dtype = "bf16" if quantised else rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if rng.random() < 0.25:
        M = _log_int(rng, 33, 4096)                        # odd row lengths among them
    else:
        M = rng.randint(1, 32) * rng.choice([64, 96, 128])
    T = _log_int(rng, 1, 55414)
    pad = rng.choice([0, 0, 64, 8]) if M % 8 == 0 else 0
    c = _case(None, kind, T, K, E, M, dtype, align, drop, pad,
              rng.choice(["int8", "e4m3"]) if quantised else "none")
    most = 0.8 * max(work(x)["bytes"] for x in listed())
    while work(c)["bytes"] + 2.0 * M * 4 * align * min(E, T * K) > most and c["T"] > 1:
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
    T, K, E, M = case["T"], case["K"], case["E"], case["M"]
    pad_tokens, slots = _dropped(case)
    R = (T - pad_tokens) * K - slots                       # rows that hold a token
    b = _BYTES[case["dtype"]]
    groups = -(-M // _GROUP)
    index, weights = 4 * T * K, 4 * T * K
    tokens, rows = T * M * b, R * M * b
    kind = case["kind"]
    if kind == "plan":
        return {"bytes": 8 * T * K + 4 * T * K + 4 * R + 4 * (2 * E + 1), "flops": 0}
    if kind == "pack":
        return {"bytes": index + tokens + rows, "flops": 0}
    if kind == "pack_grad":
        return {"bytes": index + tokens + rows, "flops": R * M}
    if kind == "merge":
        return {"bytes": index + weights + tokens + rows, "flops": 2 * R * M}
    if kind == "merge_grad":
        return {"bytes": index + 2 * weights + tokens + 2 * rows, "flops": 3 * R * M}
    if kind == "pack_q":
        kept = T * M + 4 * T * groups
        return {"bytes": 2 * index + tokens + 2 * rows + 2 * kept, "flops": 3 * T * M + R * M}
    kept = R * M + 4 * R * groups
    return {"bytes": 2 * index + 3 * weights + 2 * tokens + 2 * rows + 2 * kept,
            "flops": 8 * R * M}


def _routing(case, gen, device):
    """Experts [T, K] (int64, as a top-k gives them) and float32 weights: popular
    and rare experts, normalised weights, dropped slots."""
    T, K, E = case["T"], case["K"], case["E"]
    bias = -0.5 * torch.log1p(torch.arange(E, device=device, dtype=torch.float32))
    bias = bias[torch.randperm(E, generator=gen, device=device)]
    top = torch.topk(torch.randn(T, E, generator=gen, device=device) + bias, K, dim=1)
    experts, weights = top.indices.contiguous(), torch.softmax(top.values, dim=1)
    pad_tokens, slots = _dropped(case)
    if pad_tokens:
        experts[T - pad_tokens:] = -1
    if slots:
        experts.view(-1)[:(T - pad_tokens) * K:50] = -1
    return experts, weights


def _rows(case):
    T, K, E, align = case["T"], case["K"], case["E"], case["align"]
    return T * K + min(E, T * K) * (align - 1)


def _plan(experts, E, align, rows):
    """row_of, slot_of, counts, offsets (int32) by a stable sort of the slots."""
    T, K = experts.shape
    flat = experts.reshape(-1).to(torch.int64)
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    kept = counts[:E]
    zero = torch.zeros(1, dtype=torch.int64, device=flat.device)
    offsets = torch.cat([zero, torch.cumsum((kept + align - 1) // align * align, 0)])
    first = torch.cat([zero, torch.cumsum(counts, 0)])[:E + 1]
    order = torch.argsort(key, stable=True)
    at = torch.arange(T * K, device=flat.device)
    expert = key[order]
    row = torch.where(expert < E, offsets[expert] + at - first[expert], -1)
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


def prepare(case, seed):
    device = torch.device("cuda")
    gen = torch.Generator(device=device)
    gen.manual_seed(int(seed))
    T, K, E, M, align = case["T"], case["K"], case["E"], case["M"], case["align"]
    dtype, kind, pad = _DTYPES[case["dtype"]], case["kind"], case["pad"]
    experts, weights = _routing(case, gen, device)
    s = {"case": case, "experts": experts, "rows": _rows(case)}
    if kind == "plan":
        return s
    s["row_of"], s["slot_of"], s["counts"], s["offsets"] = _plan(experts, E, align, s["rows"])
    s["weights"] = weights
    if kind in ("pack", "pack_q", "merge_grad", "merge_q"):
        # a token-major view with `pad` unused elements behind each row
        s["tokens"] = _activations((T, M + pad), dtype, gen, device)[:, :M]
    if kind in ("pack_grad", "merge", "merge_grad", "merge_q"):
        s["packed"] = _activations((s["rows"], M), dtype, gen, device)
        # what no slot owns is never read
        s["packed"][s["slot_of"] < 0] = float("nan")
    if kind in ("pack_grad", "merge", "merge_q"):
        s["out_tokens"] = torch.zeros((T, M + pad), dtype=dtype, device=device)[:, :M]
    if kind in ("pack", "merge_grad", "pack_q", "merge_q"):
        s["out_packed"] = torch.zeros((s["rows"], M), dtype=dtype, device=device)
    if kind == "pack_q":
        s["restored"] = torch.zeros((s["rows"], M), dtype=dtype, device=device)
    return s


# ---- the plain forms ---------------------------------------------------------

def _plain_pack(tokens, slot_of, K):
    token = (slot_of.clamp(min=0) // K).long()
    return torch.where((slot_of >= 0)[:, None], tokens[token], 0)


def _expert_rows(packed, row_of):
    """[T, K, M] float32 rows, zeros where the slot is dropped."""
    return torch.where((row_of >= 0)[:, :, None], packed[row_of.clamp(min=0).long()].float(), 0)


def _plain_merge(packed, row_of, weights, dtype):
    rows = _expert_rows(packed, row_of)
    if weights is not None:
        rows = rows * torch.where(row_of >= 0, weights, 0)[:, :, None]
    return rows.sum(dim=1).to(dtype)


def _plain_merge_grad(grad, packed, row_of, slot_of, weights):
    K, dtype = row_of.shape[1], grad.dtype
    grad = grad.float()
    slot = slot_of.clamp(min=0).long()
    grad_packed = grad[slot // K] * weights.reshape(-1)[slot][:, None]
    grad_packed = torch.where((slot_of >= 0)[:, None], grad_packed, 0).to(dtype)
    grad_weights = (grad[:, None, :] * _expert_rows(packed, row_of)).sum(dim=2)
    return grad_packed, grad_weights


def _plain_quantise(x, fmt):
    """Codes (as float32 values) and scales, one scale per group of a row; the
    row is padded with zeros to whole groups."""
    rows, M = x.shape
    groups, top = -(-M // _GROUP), _TOP[fmt]
    x = torch.nn.functional.pad(x.float(), (0, groups * _GROUP - M)).view(rows, groups, _GROUP)
    amax = x.abs().amax(dim=2, keepdim=True)
    live = amax >= _FLOOR
    safe = torch.where(live, amax, 1.0)
    top = torch.full_like(safe, top)             # a scalar here would divide in two roundings
    q = torch.where(live, x * (top / safe), 0)
    codes = torch.round(q).clamp(-127, 127) if fmt == "int8" else \
        q.to(torch.float8_e4m3fn).float()
    return codes, torch.where(live, safe / top, 0)


def _plain_restore(codes, scales, M):
    return (codes * scales).view(codes.shape[0], -1)[:, :M]


def _run_plain(s):
    case = s["case"]
    kind, K, M, dtype = case["kind"], case["K"], case["M"], _DTYPES[case["dtype"]]
    if kind == "plan":
        return _plan(s["experts"], case["E"], case["align"], s["rows"])
    row_of, slot_of = s["row_of"], s["slot_of"]
    if kind == "pack":
        return _plain_pack(s["tokens"], slot_of, K)
    if kind == "pack_grad":
        return _plain_merge(s["packed"], row_of, None, dtype)
    if kind == "merge":
        return _plain_merge(s["packed"], row_of, s["weights"], dtype)
    if kind == "merge_grad":
        return _plain_merge_grad(s["tokens"], s["packed"], row_of, slot_of, s["weights"])
    if kind == "pack_q":
        packed = _plain_pack(s["tokens"], slot_of, K)
        kept = _plain_restore(*_plain_quantise(s["tokens"], case["fmt"]), M).to(dtype)
        return packed, _plain_pack(kept, slot_of, K)
    merged = _plain_merge(s["packed"], row_of, s["weights"], dtype)
    kept = _plain_restore(*_plain_quantise(s["packed"], case["fmt"]), M)
    return (merged, *_plain_merge_grad(s["tokens"], kept, row_of, slot_of, s["weights"]))


# ---- the package's calls -----------------------------------------------------

def _run_own(s):
    import sequence_head_relayout_gb300 as vf
    case = s["case"]
    kind, fmt = case["kind"], case["fmt"]
    if kind == "plan":
        return tuple(vf.expert_plan(s["experts"], case["E"], align=case["align"])[:4])
    plan = vf.ExpertPlan(s["row_of"], s["slot_of"], s["counts"], s["offsets"], case["align"])
    if kind == "pack":
        return vf.expert_pack(s["tokens"], plan, out=s["out_packed"])
    if kind == "pack_grad":
        return vf.expert_merge(s["packed"], plan, out=s["out_tokens"])
    if kind == "merge":
        return vf.expert_merge(s["packed"], plan, s["weights"], out=s["out_tokens"])
    if kind == "merge_grad":
        return vf.expert_merge_backward(s["tokens"], s["packed"], plan, s["weights"],
                                        grad_packed=s["out_packed"])
    if kind == "pack_q":
        packed, codes, scales = vf.expert_pack_q(s["tokens"], plan, fmt, _GROUP,
                                                 out=s["out_packed"])
        return packed, vf.expert_restore_q(codes, scales, plan, fmt, _GROUP, out=s["restored"])
    merged, codes, scales = vf.expert_merge_q(s["packed"], plan, s["weights"], fmt, _GROUP,
                                              out=s["out_tokens"])
    grads = vf.expert_merge_backward_q(s["tokens"], codes, scales, plan, s["weights"], fmt,
                                       _GROUP, grad_packed=s["out_packed"])
    return (merged, *grads)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definitions in 64 bits ----------------------------------------------

def _exact_plan(experts, E, align, rows):
    """Each expert's slots in slot order, by a search for each expert."""
    flat = experts.reshape(-1).cpu()
    row_of, slot_of = torch.full_like(flat, -1), torch.full((rows,), -1, dtype=torch.int64)
    counts, offsets, at = [], [0], 0
    for e in range(E):
        slots = (flat == e).nonzero()[:, 0]
        row_of[slots] = torch.arange(at, at + slots.numel())
        slot_of[at:at + slots.numel()] = slots
        counts.append(slots.numel())
        at += -(-slots.numel() // align) * align
        offsets.append(at)
    return (row_of.view(experts.shape).int(), slot_of.int(),
            torch.tensor(counts, dtype=torch.int32), torch.tensor(offsets, dtype=torch.int32))


def _exact_kept(x, fmt):
    """The values a checkpoint of x stands for.  The format's own steps are
    roundings to 32 bits; each is done here in 64 bits and rounded once (a
    quotient or product of 24-bit numbers survives both roundings unchanged)."""
    rows, M = x.shape
    top = _TOP[fmt]
    kept = torch.empty((rows, M), dtype=torch.float64, device=x.device)
    for g in range(0, M, _GROUP):
        v = x[:, g:g + _GROUP].double()
        amax = v.abs().max(dim=1).values
        safe = torch.where(amax >= _FLOOR, amax, torch.ones_like(amax))
        inv, scale = (top / safe).float().double(), (safe / top).float().double()
        q = (v * inv[:, None]).float().double()
        if fmt == "int8":
            code = torch.round(q).clamp(-127, 127)
        else:
            # a step of the E4M3 grid at q: 2^(floor(log2|q|) - 3), at least 2^-9
            exponent = (torch.frexp(q).exponent - 1).clamp(min=-6)
            # (built from its bits: a computed power could be one unit off)
            step = ((exponent.long() - 3 + 1023) << 52).view(torch.float64)
            code = (torch.round(q / step) * step).clamp(-448, 448)
        kept[:, g:g + _GROUP] = torch.where((amax >= _FLOOR)[:, None], code * scale[:, None],
                                            torch.zeros_like(code))
    return kept


def _exact_scatter(rows_of_token, row_of, rows, M):
    """[rows, M] from each slot's values, zeros elsewhere; one slot k at a time."""
    out = torch.zeros((rows + 1, M), dtype=torch.float64, device=row_of.device)
    for k in range(row_of.shape[1]):
        out[torch.where(row_of[:, k] < 0, rows, row_of[:, k]).long()] = rows_of_token(k)
    out[rows] = 0
    return out[:rows]


def _exact_gather(packed, row_of, k):
    there = row_of[:, k] >= 0
    return torch.where(there[:, None], packed[row_of[:, k].clamp(min=0).long()].double(),
                       torch.zeros((), dtype=torch.float64, device=packed.device))


def _exact_sum(packed, row_of, weights):
    T, K = row_of.shape
    out = torch.zeros((T, packed.shape[1]), dtype=torch.float64, device=packed.device)
    for k in range(K):
        w = 1.0 if weights is None else weights[:, k, None].double()
        out += torch.where((row_of[:, k] >= 0)[:, None], w * _exact_gather(packed, row_of, k),
                           torch.zeros_like(out))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    kind, K, M, rows = case["kind"], case["K"], case["M"], s["rows"]
    if kind == "plan":
        return _exact_plan(s["experts"], case["E"], case["align"], rows)
    row_of, weights, tokens = s["row_of"], s["weights"], s.get("tokens")
    if kind == "pack":
        return _exact_scatter(lambda k: tokens.double(), row_of, rows, M)
    if kind == "pack_grad":
        return _exact_sum(s["packed"], row_of, None)
    if kind == "merge":
        return _exact_sum(s["packed"], row_of, weights)
    if kind == "pack_q":
        kept = _exact_kept(tokens, case["fmt"])
        return (_exact_scatter(lambda k: tokens.double(), row_of, rows, M),
                _exact_scatter(lambda k: kept, row_of, rows, M))
    packed = s["packed"]
    merged = _exact_sum(packed, row_of, weights) if kind == "merge_q" else None
    if kind == "merge_q":
        packed = _exact_kept(torch.nan_to_num(packed), case["fmt"])
    grad = tokens.double()
    grad_packed = _exact_scatter(lambda k: grad * weights[:, k, None].double(), row_of, rows, M)
    grad_weights = torch.stack([(grad * _exact_gather(packed, row_of, k)).sum(1)
                                for k in range(K)], dim=1)
    if kind == "merge_grad":
        return grad_packed, grad_weights
    return merged, grad_packed, grad_weights
