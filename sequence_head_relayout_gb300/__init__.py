"""GB300-native exact destination-major relayouts around sequence-head attention.

Thin ctypes binding over ``libvf_relayout.so`` (C ABI in
``include/vf_relayout.h``): the functions here only marshal tensor pointers,
strides and the current CUDA stream; every element is moved by the library's
sm_103a kernels.  PyTorch provides device memory and streams.  There is no
CPU path: the library must be built (``__graft_entry__.build()``) and the
tensors must be addressable by the GPU -- CUDA memory, or pinned host memory
that the kernels read or write directly over the host link -- otherwise the
calls raise.  A pinned tensor, a returned one too, has to be kept until the
stream is past the calls that use it: torch's pinned-memory allocator does not
know of these kernels and hands its memory out again at once.

Operations ("Sol-Engine alignment on SM86 and SM89", section "What is
enabled"):

* :func:`qkv_pack`   -- fused [T,3,H,D] QKV view -> destination-major send buffer;
* :func:`attn_split` -- attention output [T,H,D] view -> per-destination token shards;
* :func:`head_merge` -- received destination-major buffer -> token-major [T,H,D];
* :func:`qkv_unpack` -- received QKV buffer -> Q, K, V [T,H/P,D] views ("速度、显存与
  质量", section "剖析单次去噪请求": the QKV unpack before Flash-SDPA);
* :func:`qkv_pack3`  -- the pack from three separate Q, K, V views.

Every function takes ``chunks=(c_begin, c_count)`` to move only those overlap
chunks (the packed buffer is always the full one) and ``order`` for the block
order of the packed storage: ``"chunk_major"`` ([c][p], the four-chunk overlap
layout, default) or ``"slot_major"`` ([p][c]).

Opt-in lossy transport (same page, table "Upstream gap and disposition", row
"INT8 QKV and FP8 output transport"): :func:`qkv_pack_q`, :func:`attn_split_q`,
:func:`head_merge_q` and :func:`qkv_unpack_q` quantise each head row to
8-bit codes (``fmt="int8"`` -> int8 codes, ``fmt="e4m3"`` -> float8_e4m3fn
codes) plus one float32 scale per head row, in the exact ops' layout, and
dequantise to bfloat16 on the receive side.  The format is stated in
``include/vf_relayout.h``.

Expert relayouts (mixture-of-experts layers): :func:`expert_plan` sorts the
routing slots by expert, :func:`expert_pack` moves token rows to expert-major
rows, :func:`expert_merge` takes them back with the routing weights and
:func:`expert_merge_backward` gives its gradients.  With 8-bit checkpoints for
the backward pass: :func:`expert_pack_q`, :func:`expert_restore_q`,
:func:`expert_merge_q` and :func:`expert_merge_backward_q`.  None of the calls
records an autograd graph: the gradients are calls of their own, and the packs
and merges refuse a tensor that requires a gradient while grad mode is on.

An expert layer's arithmetic, in the same manner: :func:`expert_product` (the packed
rows times their experts' weights) and :func:`expert_weight_grad`,
:func:`expert_glu` and :func:`expert_glu_backward` (the gated activation between
two products), :func:`rms_norm`, :func:`rms_norm_q` and :func:`rms_norm_backward` (the
root-mean-square norm in front, with the residual's addition).
"""
import ctypes
import os
import struct
from typing import NamedTuple

import torch

__all__ = ["qkv_pack", "qkv_pack3", "attn_split", "head_merge", "qkv_unpack", "packed_elems",
           "piece_table", "VFError", "lib", "OP_QKV_PACK", "OP_ATTN_SPLIT", "OP_HEAD_MERGE",
           "OP_QKV_UNPACK", "qkv_pack_q", "attn_split_q", "head_merge_q", "qkv_unpack_q",
           "scale_count", "FORMATS", "ExpertPlan", "expert_rows", "expert_plan", "expert_pack",
           "expert_merge", "expert_merge_backward", "expert_pack_q", "expert_restore_q",
           "expert_merge_q", "expert_merge_backward_q", "expert_product", "expert_weight_grad",
           "expert_glu", "expert_glu_backward", "rms_norm", "rms_norm_q", "rms_norm_backward"]

OP_QKV_PACK, OP_ATTN_SPLIT, OP_HEAD_MERGE, OP_QKV_UNPACK = 0, 1, 2, 3
ORDERS = {"chunk_major": 0, "slot_major": 1}
FORMATS = {"int8": 1, "e4m3": 2}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvf_relayout.so")

_lib = None
_I64 = ctypes.c_int64
_P = ctypes.c_void_p
_I64P = ctypes.POINTER(_I64)


class _Desc(ctypes.Structure):
    """vf_relayout_desc of the C ABI."""
    _fields_ = [("op", ctypes.c_int32), ("order", ctypes.c_int32),
                ("T", _I64), ("H", _I64), ("D", _I64), ("P", _I64), ("C", _I64),
                ("c_begin", _I64), ("c_count", _I64), ("packed", _P),
                ("strided", _P * 3), ("strides", _I64 * 3)]


class _ExpertDesc(ctypes.Structure):
    """vf_expert_desc of the C ABI."""
    _fields_ = [("type", ctypes.c_int32), ("format", ctypes.c_int32),
                ("T", _I64), ("K", _I64), ("M", _I64), ("E", _I64), ("rows", _I64),
                ("align", _I64), ("group", _I64),
                ("row_of", _P), ("counts", _P), ("offsets", _P),
                ("tokens", _P), ("token_strides", _I64 * 2), ("packed", _P),
                ("weights", _P), ("weight_strides", _I64 * 2), ("codes", _P), ("scales", _P),
                ("grad_packed", _P), ("grad_weights", _P)]


# The descriptors of the calls below the expert relayouts are packed by one call each,
# which takes 1 us where setting the fields of a ctypes structure takes 3 to 4.
_PRODUCT_DESC = struct.Struct("@ii16q")      # vf_product_desc of the C ABI, but for the
_POINTER = struct.Struct("@q")               # workspace at its end
_GLU_DESC = struct.Struct("@iq22q")          # vf_glu_desc
_NORM_DESC = struct.Struct("@iiif29q")       # vf_norm_desc


class VFError(RuntimeError):
    """A negative status returned by the library."""

    def __init__(self, fn, status):
        self.status = status
        msg = lib().vf_status_string(status).decode()
        super().__init__("%s failed: %s (status %d)" % (fn, msg, status))


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libvf_relayout.so is not built; run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        l = ctypes.CDLL(LIB_PATH)
        sig = {
            "vf_qkv_pack": [_P, _I64P] + [_I64] * 5 + [_P, _P],
            "vf_attn_split": [_P, _I64P] + [_I64] * 5 + [_P, _P],
            "vf_head_merge": [_P, _I64P] + [_I64] * 5 + [_P, _P],
            "vf_qkv_unpack": [_P] + [_I64] * 5 + [_P, _P, _P, _I64P, _P],
            "vf_qkv_pack_chunks": [_P, _I64P] + [_I64] * 7 + [_P, _P],
            "vf_attn_split_chunks": [_P, _I64P] + [_I64] * 7 + [_P, _P],
            "vf_head_merge_chunks": [_P, _I64P] + [_I64] * 7 + [_P, _P],
            "vf_qkv_unpack_chunks": [_P] + [_I64] * 7 + [_P, _P, _P, _I64P, _P],
            "vf_qkv_pack3": [_P, _P, _P, _I64P] + [_I64] * 7 + [_P, _P],
        }
        for name, args in sig.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        l.vf_packed_elems.argtypes = [ctypes.c_int, _I64, _I64, _I64, _I64, _I64]
        l.vf_packed_elems.restype = _I64
        l.vf_piece_table.argtypes = [ctypes.c_int, _I64, _I64, _I64, _I64, _I64,
                                     _I64P, _I64P, _I64P, _I64]
        l.vf_piece_table.restype = _I64
        l.vf_piece_table_ex.argtypes = [ctypes.c_int, ctypes.c_int, _I64, _I64, _I64, _I64,
                                        _I64, _I64P, _I64P, _I64P, _I64]
        l.vf_piece_table_ex.restype = _I64
        l.vf_relayout.argtypes = [ctypes.POINTER(_Desc), _P]
        l.vf_relayout.restype = ctypes.c_int
        l.vf_relayout_q.argtypes = [ctypes.POINTER(_Desc), ctypes.c_int, _P, _P]
        l.vf_relayout_q.restype = ctypes.c_int
        for name, args in {
            "vf_qkv_pack_int8": [_P, _I64P] + [_I64] * 5 + [_P, _P, _P],
            "vf_qkv_unpack_int8": [_P, _P] + [_I64] * 5 + [_P, _P, _P, _I64P, _P],
            "vf_attn_split_fp8": [_P, _I64P] + [_I64] * 5 + [_P, _P, _P],
            "vf_head_merge_fp8": [_P, _P, _I64P] + [_I64] * 5 + [_P, _P],
        }.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        l.vf_scale_count.argtypes = [ctypes.c_int, _I64, _I64, _I64, _I64, _I64]
        l.vf_scale_count.restype = _I64
        l.vf_expert_rows.argtypes = [_I64] * 4
        l.vf_expert_rows.restype = _I64
        l.vf_expert_workspace.argtypes = [_I64] * 3
        l.vf_expert_workspace.restype = _I64
        l.vf_expert_plan.argtypes = [_P, ctypes.c_int, _I64P] + [_I64] * 4 + [_P] * 6
        l.vf_expert_plan.restype = ctypes.c_int
        for name in ("vf_expert_pack", "vf_expert_restore", "vf_expert_merge",
                     "vf_expert_merge_backward"):
            f = getattr(l, name)
            f.argtypes = [ctypes.POINTER(_ExpertDesc), _P]
            f.restype = ctypes.c_int
        for name in ("vf_expert_product", "vf_expert_weight_grad", "vf_expert_glu",
                     "vf_expert_glu_backward", "vf_rms_norm", "vf_rms_norm_backward"):
            f = getattr(l, name)
            f.argtypes = [ctypes.c_char_p, _P]
            f.restype = ctypes.c_int
        for name in ("vf_expert_product_workspace", "vf_expert_weight_grad_workspace"):
            f = getattr(l, name)
            f.argtypes = [ctypes.c_char_p]
            f.restype = _I64
        l.vf_rms_norm_workspace.argtypes = [_I64, _I64]
        l.vf_rms_norm_workspace.restype = _I64
        l.vf_status_string.argtypes = [ctypes.c_int]
        l.vf_status_string.restype = ctypes.c_char_p
        _lib = l
    return _lib


def _check16(t: torch.Tensor, what: str):
    """A 16-bit tensor the GPU can address: CUDA memory, or pinned (page-locked,
    mapped) host memory, which the kernels read and write directly over the
    host link.  Pageable host memory is refused: there is no CPU path."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    if t.device.type != "cuda" and not (t.device.type == "cpu" and t.is_pinned()):
        raise ValueError("%s must be a CUDA tensor or pinned host memory "
                         "(there is no CPU path)" % what)
    if t.element_size() != 2:
        raise ValueError("%s must hold 16-bit elements (bf16/fp16/int16)" % what)


def _strides(t: torch.Tensor):
    return (_I64 * t.dim())(*t.stride())


def _stream(stream, device):
    """The stream to enqueue on: the given one, else the current stream of the
    tensor's device (of the current device for pinned host tensors)."""
    if stream is not None:
        return stream.cuda_stream
    # (the handle itself: building a Stream object costs 2 us a call)
    index = device.index                                   # None for host memory
    return torch._C._cuda_getCurrentRawStream(
        torch.cuda.current_device() if index is None else index)


def _call(fn, *args):
    rc = getattr(_lib or lib(), fn)(*args)
    if rc != 0:
        raise VFError(fn, rc)


def _n_packed(op, T, H, D, P):
    """Packed element count for sizing outputs (the library validates the
    shape again on every call); odd shapes go through the library's check."""
    if P < 1 or min(T, H, D) < 0:
        return packed_elems(op, T, H, D, P, 1)            # raises VFError
    if op == OP_QKV_PACK:
        return 3 * T * H * D
    if op == OP_QKV_UNPACK:
        return 3 * T * (H // P) * D
    return T * H * D


def packed_elems(op: int, T: int, H: int, D: int, P: int, C: int) -> int:
    """Elements of the packed side of ``op`` (3*T*H*D for the pack, T*H*D for the
    split and the merge, 3*T*(H/P)*D for the unpack)."""
    n = lib().vf_packed_elems(op, T, H, D, P, C)
    if n < 0:
        raise VFError("vf_packed_elems", n)
    return n


def _order(order) -> int:
    o = ORDERS.get(order)
    if o is None:
        raise ValueError("order must be one of %s" % sorted(ORDERS))
    return o


def piece_table(op: int, T: int, H: int, D: int, P: int, C: int, order="chunk_major"):
    """(tok_start, tok_len, packed_off) lists; entry c*P + p is block (c, p),
    packed_off places the blocks in the given storage order."""
    m = P * C
    a, b, c = (_I64 * m)(), (_I64 * m)(), (_I64 * m)()
    n = lib().vf_piece_table_ex(op, _order(order), T, H, D, P, C, a, b, c, m)
    if n < 0:
        raise VFError("vf_piece_table", n)
    return list(a), list(b), list(c)


def _range(chunks, C):
    return (0, C) if chunks is None else (int(chunks[0]), int(chunks[1]))


def _relayout(op, order, T, H, D, P, C, chunks, packed, strided, strides, stream,
              fmt=0, scales=None):
    """vf_relayout (or vf_relayout_q with a format) with a descriptor: the
    general entry, any block order."""
    c0, cn = _range(chunks, C)
    d = _Desc(op=op, order=order, T=T, H=H, D=D, P=P, C=C, c_begin=c0, c_count=cn,
              packed=packed)
    for i, ptr in enumerate(strided):
        d.strided[i] = ptr
    for i, st in enumerate(strides):
        d.strides[i] = st
    if fmt:
        rc = lib().vf_relayout_q(ctypes.byref(d), fmt, scales, stream)
        if rc != 0:
            raise VFError("vf_relayout_q", rc)
        return
    rc = lib().vf_relayout(ctypes.byref(d), stream)
    if rc != 0:
        raise VFError("vf_relayout", rc)


def _flat_out(out, n, like):
    if out is None:
        out = torch.empty(n, dtype=like.dtype, device=like.device,
                          pin_memory=like.device.type == "cpu")
    _check16(out, "out")
    if not out.is_contiguous() or out.numel() != n:
        raise ValueError("out must be contiguous with %d elements" % n)
    return out


def qkv_pack(src: torch.Tensor, P: int, C: int, out: torch.Tensor = None,
             stream: torch.cuda.Stream = None, chunks=None,
             order="chunk_major") -> torch.Tensor:
    """QKV destination pack of a [T,3,H,D] CUDA view (any strides).

    Returns (or fills) a flat tensor of 3*T*H*D elements: blocks (c, p) in
    order, each head group p of chunk c as q, k, v slabs [L_c][H/P][D].
    """
    _check16(src, "src")
    if src.dim() != 4 or src.shape[1] != 3:
        raise ValueError("src must be a [T,3,H,D] view")
    T, _, H, D = src.shape
    out = _flat_out(out, _n_packed(OP_QKV_PACK, T, H, D, P), src)
    o = _order(order)
    if o:
        st = src.stride()
        bases = [src.data_ptr() + s * st[1] * src.element_size() for s in range(3)]
        _relayout(OP_QKV_PACK, o, T, H, D, P, C, chunks, out.data_ptr(), bases,
                  (st[0], st[2], st[3]), _stream(stream, src.device))
        return out
    c0, cn = _range(chunks, C)
    _call("vf_qkv_pack_chunks", src.data_ptr(), _strides(src), T, H, D, P, C, c0, cn,
          out.data_ptr(), _stream(stream, src.device))
    return out


def qkv_pack3(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, P: int, C: int,
              out: torch.Tensor = None, stream: torch.cuda.Stream = None,
              chunks=None, order="chunk_major") -> torch.Tensor:
    """QKV destination pack from three [T,H,D] CUDA views with equal strides."""
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _check16(t, name)
    if q.dim() != 3 or q.shape != k.shape or q.shape != v.shape:
        raise ValueError("q, k, v must be [T,H,D] views of one shape")
    if q.stride() != k.stride() or q.stride() != v.stride():
        raise ValueError("q, k, v must share their strides")
    T, H, D = q.shape
    out = _flat_out(out, _n_packed(OP_QKV_PACK, T, H, D, P), q)
    o = _order(order)
    if o:
        _relayout(OP_QKV_PACK, o, T, H, D, P, C, chunks, out.data_ptr(),
                  [q.data_ptr(), k.data_ptr(), v.data_ptr()], q.stride(),
                  _stream(stream, q.device))
        return out
    c0, cn = _range(chunks, C)
    _call("vf_qkv_pack3", q.data_ptr(), k.data_ptr(), v.data_ptr(), _strides(q), T, H, D, P,
          C, c0, cn, out.data_ptr(), _stream(stream, q.device))
    return out


def attn_split(src: torch.Tensor, P: int, C: int, out: torch.Tensor = None,
               stream: torch.cuda.Stream = None, chunks=None,
               order="chunk_major") -> torch.Tensor:
    """Attention-result split of a [T,H,D] CUDA view (any strides).

    Returns (or fills) a flat tensor of T*H*D elements: blocks (c, p) in
    order, each chunk c of token shard p as [L][H][D].
    """
    _check16(src, "src")
    if src.dim() != 3:
        raise ValueError("src must be a [T,H,D] view")
    T, H, D = src.shape
    out = _flat_out(out, _n_packed(OP_ATTN_SPLIT, T, H, D, P), src)
    o = _order(order)
    if o:
        _relayout(OP_ATTN_SPLIT, o, T, H, D, P, C, chunks, out.data_ptr(), [src.data_ptr()],
                  src.stride(), _stream(stream, src.device))
        return out
    c0, cn = _range(chunks, C)
    _call("vf_attn_split_chunks", src.data_ptr(), _strides(src), T, H, D, P, C, c0, cn,
          out.data_ptr(), _stream(stream, src.device))
    return out


def head_merge(src: torch.Tensor, T: int, H: int, D: int, P: int, C: int,
               out: torch.Tensor = None, stream: torch.cuda.Stream = None,
               chunks=None, order="chunk_major") -> torch.Tensor:
    """Returned-head merge of a flat received buffer into a [T,H,D] view.

    ``out`` may be any non-overlapping strided [T,H,D] CUDA view; a
    contiguous tensor is allocated when it is omitted.
    """
    _check16(src, "src")
    n = _n_packed(OP_HEAD_MERGE, T, H, D, P)
    if not src.is_contiguous() or src.numel() != n:
        raise ValueError("src must be contiguous with %d elements" % n)
    if out is None:
        out = torch.empty((T, H, D), dtype=src.dtype, device=src.device,
                          pin_memory=src.device.type == "cpu")
    _check16(out, "out")
    if tuple(out.shape) != (T, H, D):
        raise ValueError("out must have shape [T,H,D]")
    o = _order(order)
    if o:
        _relayout(OP_HEAD_MERGE, o, T, H, D, P, C, chunks, src.data_ptr(), [out.data_ptr()],
                  out.stride(), _stream(stream, src.device))
        return out
    c0, cn = _range(chunks, C)
    _call("vf_head_merge_chunks", src.data_ptr(), _strides(out), T, H, D, P, C, c0, cn,
          out.data_ptr(), _stream(stream, src.device))
    return out


def qkv_unpack(recv: torch.Tensor, T: int, H: int, D: int, P: int, C: int, outs=None,
               stream: torch.cuda.Stream = None, chunks=None, order="chunk_major"):
    """Receive-side QKV unpack: flat received buffer of 3*T*(H/P)*D elements
    into (Q, K, V), each a [T, H/P, D] view (global token order).

    ``outs`` may give three non-overlapping [T, H/P, D] CUDA views sharing one
    stride tuple; contiguous tensors are allocated when it is omitted.
    """
    _check16(recv, "recv")
    n = _n_packed(OP_QKV_UNPACK, T, H, D, P)
    if not recv.is_contiguous() or recv.numel() != n:
        raise ValueError("recv must be contiguous with %d elements" % n)
    Hp = H // P
    if outs is None:
        outs = tuple(torch.empty((T, Hp, D), dtype=recv.dtype, device=recv.device,
                                 pin_memory=recv.device.type == "cpu") for _ in range(3))
    q, k, v = outs
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _check16(t, name)
        if tuple(t.shape) != (T, Hp, D):
            raise ValueError("%s must have shape [T,H/P,D]" % name)
    if q.stride() != k.stride() or q.stride() != v.stride():
        raise ValueError("q, k, v must share their strides")
    o = _order(order)
    if o:
        _relayout(OP_QKV_UNPACK, o, T, H, D, P, C, chunks, recv.data_ptr(),
                  [q.data_ptr(), k.data_ptr(), v.data_ptr()], q.stride(),
                  _stream(stream, recv.device))
        return outs
    c0, cn = _range(chunks, C)
    _call("vf_qkv_unpack_chunks", recv.data_ptr(), T, H, D, P, C, c0, cn, q.data_ptr(),
          k.data_ptr(), v.data_ptr(), _strides(q), _stream(stream, recv.device))
    return outs


# ---- opt-in lossy transport --------------------------------------------------

def _fmt(fmt) -> int:
    f = FORMATS.get(fmt)
    if f is None:
        raise ValueError("fmt must be one of %s" % sorted(FORMATS))
    return f


def _code_dtype(f):
    return torch.int8 if f == 1 else torch.float8_e4m3fn


def _gpu_addressable(t, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    if t.device.type != "cuda" and not (t.device.type == "cpu" and t.is_pinned()):
        raise ValueError("%s must be a CUDA tensor or pinned host memory "
                         "(there is no CPU path)" % what)


def scale_count(op: int, T: int, H: int, D: int, P: int, C: int) -> int:
    """Scales (one per head row) of the packed side of ``op``."""
    n = lib().vf_scale_count(op, T, H, D, P, C)
    if n < 0:
        raise VFError("vf_scale_count", n)
    return n


def _codes_scales(codes, scales, n, rows, f, like, what):
    """Check (or allocate) the flat codes and scales buffers."""
    if codes is None:
        codes = torch.empty(n, dtype=_code_dtype(f), device=like.device,
                            pin_memory=like.device.type == "cpu")
    if scales is None:
        scales = torch.empty(rows, dtype=torch.float32, device=like.device,
                             pin_memory=like.device.type == "cpu")
    _gpu_addressable(codes, what + " codes")
    _gpu_addressable(scales, what + " scales")
    if codes.element_size() != 1 or not codes.is_contiguous() or codes.numel() != n:
        raise ValueError("codes must be a contiguous 8-bit tensor of %d elements" % n)
    if scales.dtype != torch.float32 or not scales.is_contiguous() or scales.numel() != rows:
        raise ValueError("scales must be a contiguous float32 tensor of %d elements" % rows)
    return codes, scales


def _rows(n, D):
    return n // D if D > 0 else 0


def _check_bf16(t: torch.Tensor, what: str):
    """The lossy transport reads and writes BF16 values (int16 views of BF16
    bit patterns are accepted too); float16 would be misread."""
    if isinstance(t, torch.Tensor) and t.dtype not in (torch.bfloat16, torch.int16):
        raise ValueError("%s must hold bfloat16 values (or their int16 bit patterns)" % what)
    _check16(t, what)


def qkv_pack_q(src: torch.Tensor, P: int, C: int, fmt="int8", codes=None, scales=None,
               stream: torch.cuda.Stream = None, chunks=None, order="chunk_major"):
    """Quantising QKV pack of a [T,3,H,D] bf16 view -> (codes, scales): the
    layout of :func:`qkv_pack`, one byte per element, one scale per head row."""
    _check_bf16(src, "src")
    if src.dim() != 4 or src.shape[1] != 3:
        raise ValueError("src must be a [T,3,H,D] view")
    f = _fmt(fmt)
    T, _, H, D = src.shape
    n = _n_packed(OP_QKV_PACK, T, H, D, P)
    codes, scales = _codes_scales(codes, scales, n, _rows(n, D), f, src, "pack")
    st = src.stride()
    bases = [src.data_ptr() + s * st[1] * src.element_size() for s in range(3)]
    _relayout(OP_QKV_PACK, _order(order), T, H, D, P, C, chunks, codes.data_ptr(), bases,
              (st[0], st[2], st[3]), _stream(stream, src.device), f, scales.data_ptr())
    return codes, scales


def attn_split_q(src: torch.Tensor, P: int, C: int, fmt="e4m3", codes=None, scales=None,
                 stream: torch.cuda.Stream = None, chunks=None, order="chunk_major"):
    """Quantising attention-result split of a [T,H,D] bf16 view -> (codes, scales)."""
    _check_bf16(src, "src")
    if src.dim() != 3:
        raise ValueError("src must be a [T,H,D] view")
    f = _fmt(fmt)
    T, H, D = src.shape
    n = _n_packed(OP_ATTN_SPLIT, T, H, D, P)
    codes, scales = _codes_scales(codes, scales, n, _rows(n, D), f, src, "split")
    _relayout(OP_ATTN_SPLIT, _order(order), T, H, D, P, C, chunks, codes.data_ptr(),
              [src.data_ptr()], src.stride(), _stream(stream, src.device), f,
              scales.data_ptr())
    return codes, scales


def head_merge_q(codes: torch.Tensor, scales: torch.Tensor, T: int, H: int, D: int, P: int,
                 C: int, fmt="e4m3", out: torch.Tensor = None,
                 stream: torch.cuda.Stream = None, chunks=None, order="chunk_major"):
    """Dequantising returned-head merge -> [T,H,D] bfloat16 (or into ``out``)."""
    f = _fmt(fmt)
    n = _n_packed(OP_HEAD_MERGE, T, H, D, P)
    codes, scales = _codes_scales(codes, scales, n, _rows(n, D), f, codes, "merge")
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device=codes.device,
                          pin_memory=codes.device.type == "cpu")
    _check_bf16(out, "out")
    if tuple(out.shape) != (T, H, D):
        raise ValueError("out must have shape [T,H,D]")
    _relayout(OP_HEAD_MERGE, _order(order), T, H, D, P, C, chunks, codes.data_ptr(),
              [out.data_ptr()], out.stride(), _stream(stream, codes.device), f,
              scales.data_ptr())
    return out


def qkv_unpack_q(codes: torch.Tensor, scales: torch.Tensor, T: int, H: int, D: int, P: int,
                 C: int, fmt="int8", outs=None, stream: torch.cuda.Stream = None,
                 chunks=None, order="chunk_major"):
    """Dequantising receive-side unpack -> (Q, K, V), each [T,H/P,D] bfloat16."""
    f = _fmt(fmt)
    n = _n_packed(OP_QKV_UNPACK, T, H, D, P)
    codes, scales = _codes_scales(codes, scales, n, _rows(n, D), f, codes, "unpack")
    Hp = H // P
    if outs is None:
        outs = tuple(torch.empty((T, Hp, D), dtype=torch.bfloat16, device=codes.device,
                                 pin_memory=codes.device.type == "cpu") for _ in range(3))
    q, k, v = outs
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _check_bf16(t, name)
        if tuple(t.shape) != (T, Hp, D):
            raise ValueError("%s must have shape [T,H/P,D]" % name)
    if q.stride() != k.stride() or q.stride() != v.stride():
        raise ValueError("q, k, v must share their strides")
    _relayout(OP_QKV_UNPACK, _order(order), T, H, D, P, C, chunks, codes.data_ptr(),
              [q.data_ptr(), k.data_ptr(), v.data_ptr()], q.stride(),
              _stream(stream, codes.device), f, scales.data_ptr())
    return outs


# ---- expert relayouts ----------------------------------------------------------

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


class ExpertPlan(NamedTuple):
    """A routing's rows, as :func:`expert_plan` writes them (all int32).

    row_of  [T, K]   row of each slot (slot t*K + k), -1 when it is dropped;
    slot_of [rows]   slot of each row, -1 where none goes;
    counts  [E]      slots of each expert;
    offsets [E + 1]  first row of each expert, a multiple of ``align``.
    """
    row_of: torch.Tensor
    slot_of: torch.Tensor
    counts: torch.Tensor
    offsets: torch.Tensor
    align: int = 1


def _rows_type(t: torch.Tensor, what: str) -> int:
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        _gpu_addressable(t, what)
    f = _TYPES.get(t.dtype)
    if f is None:
        raise ValueError("%s must hold bfloat16, float16 or float32 values" % what)
    return f


def _unrecorded(t: torch.Tensor, what: str, gradient: str):
    """Refuse a tensor whose gradient autograd would expect to be recorded: the
    result of these calls has none, and it would be lost without a word."""
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError("%s requires a gradient, which this call does not record: pass "
                         "%s.detach() or call it under torch.no_grad() (or in a "
                         "torch.autograd.Function), with %s as its gradient"
                         % (what, what, gradient))


def _check_plan(plan, T=None):
    """(T, K, rows, E) of a plan whose tensors have the types and shapes that
    the kernels take; what they hold is checked by the kernels."""
    row_of, slot_of, counts, offsets, _ = plan
    i32 = torch.int32
    for t in (row_of, slot_of, counts, offsets):
        if not (isinstance(t, torch.Tensor) and t.is_cuda):
            _gpu_addressable(t, "plan")
        if t.dtype != i32 or not t.is_contiguous():
            raise ValueError("the tensors of a plan must be contiguous and int32")
    a, rows, E, o = row_of.shape, slot_of.shape, counts.shape, offsets.shape
    if len(a) != 2 or len(rows) != 1 or len(E) != 1 or len(o) != 1 or o[0] != E[0] + 1:
        raise ValueError("plan must hold row_of [T,K], slot_of [rows], counts [E] and "
                         "offsets [E+1]")
    if T is not None and a[0] != T:
        raise ValueError("plan is for %d tokens, not %d" % (a[0], T))
    return a[0], a[1], rows[0], E[0]


def _new(stream, like, shape, dtype):
    """An output tensor beside ``like``.  Device memory is allocated on the stream
    that fills it, so that it is not handed out while that stream still uses it.
    Pinned host memory has no such order: whoever holds the tensor keeps it until
    the stream is done with it."""
    if not like.is_cuda:
        return torch.empty(shape, dtype=dtype, pin_memory=True)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _workspace(stream, like, words):
    """int32 scratch memory that a call drops when it returns: always device
    memory, on the current device where ``like`` is host memory."""
    device = like.device if like.is_cuda else "cuda"
    if stream is None:
        return torch.empty((words,), dtype=torch.int32, device=device)
    with torch.cuda.stream(stream):
        return torch.empty((words,), dtype=torch.int32, device=device)


def _rows_out(t, stream, like, shape, dtype, what):
    """Check (or allocate) a contiguous [rows, M] tensor."""
    if t is None:
        return _new(stream, like, shape, dtype)
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        _gpu_addressable(t, what)
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s" % (what, dtype, shape))
    return t


def _tokens_out(t, stream, like, shape, dtype, what):
    """Check (or allocate) a [T, M] view."""
    if t is None:
        return _new(stream, like, shape, dtype)
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        _gpu_addressable(t, what)
    if t.dtype != dtype or t.shape != shape:
        raise ValueError("%s must be a %s view of shape %s" % (what, dtype, shape))
    return t


def _kept(codes, scales, stream, like, n, M, f, group):
    """Check (or allocate) a checkpoint: codes [n, M], scales [n, groups]."""
    if group not in (32, 64, 128, 256):
        raise ValueError("group must be 32, 64, 128 or 256")
    codes = _rows_out(codes, stream, like, (n, M), _code_dtype(f), "codes")
    scales = _rows_out(scales, stream, like, (n, -(-M // group)), torch.float32, "scales")
    return codes, scales


def _expert_desc(typ, plan, dims, M):
    d = _ExpertDesc(typ, 0, dims[0], dims[1], M, dims[3], dims[2], plan[4])
    d.row_of, d.counts, d.offsets = plan[0].data_ptr(), plan[2].data_ptr(), plan[3].data_ptr()
    return d


def _set_tokens(d, t):
    d.tokens = t.data_ptr()
    d.token_strides = t.stride()


def _set_weights(d, weights, T, K):
    if weights is None:
        return
    if not (isinstance(weights, torch.Tensor) and weights.is_cuda):
        _gpu_addressable(weights, "weights")
    if weights.dtype != torch.float32 or weights.shape != (T, K):
        raise ValueError("weights must be a float32 view of shape [T,K]")
    d.weights = weights.data_ptr()
    d.weight_strides = weights.stride()


def _set_kept(d, codes, scales, f, group):
    d.format, d.group = f, group
    d.codes, d.scales = codes.data_ptr(), scales.data_ptr()


def _expert_call(fn, d, stream, like):
    rc = getattr(_lib or lib(), fn)(ctypes.byref(d), _stream(stream, like.device))
    if rc != 0:
        raise VFError(fn, rc)


def _matrix(t, what):
    if t.dim() != 2:
        raise ValueError("%s must have two dimensions" % what)
    return t.shape


def expert_rows(T: int, K: int, E: int, align: int = 1) -> int:
    """Rows of the expert-major side: T*K + min(E, T*K) * (align - 1), the most
    that any routing of T tokens to K of E experts takes."""
    n = lib().vf_expert_rows(T, K, E, align)
    if n < 0:
        raise VFError("vf_expert_rows", n)
    return n


def expert_plan(experts: torch.Tensor, E: int, align: int = 1, out: ExpertPlan = None,
                stream: torch.cuda.Stream = None) -> ExpertPlan:
    """Sort the slots of a [T,K] view of expert indices (int32 or int64) by
    expert, stably; indices outside [0, E) are dropped.

    Each expert's rows start at a multiple of ``align``.  ``out`` gives the
    tensors of an earlier plan of the same sizes to be written again.
    """
    if not (isinstance(experts, torch.Tensor) and experts.is_cuda):
        _gpu_addressable(experts, "experts")
    if experts.dtype not in (torch.int32, torch.int64) or experts.dim() != 2:
        raise ValueError("experts must be an int32 or int64 view of shape [T,K]")
    T, K = experts.shape
    words = lib().vf_expert_workspace(T, K, E) // 4
    rows = T * K + min(E, T * K) * (align - 1)             # without another library call
    if words < 0 or not 1 <= align <= 65536 or rows > 0x7FFFFFFF:    # the limits of the header
        rows = expert_rows(T, K, E, align)                 # raises VFError
    if out is None:
        # (views of one allocation take longer to make than four allocations)
        out = ExpertPlan(_new(stream, experts, (T, K), torch.int32),
                         _new(stream, experts, (rows,), torch.int32),
                         _new(stream, experts, (E,), torch.int32),
                         _new(stream, experts, (E + 1,), torch.int32), align)
    elif _check_plan(out) != (T, K, rows, E) or out.align != align:
        raise ValueError("out is a plan of other sizes")
    work = _workspace(stream, experts, words) if words else None
    _call("vf_expert_plan", experts.data_ptr(), experts.element_size(), _strides(experts), T, K,
          E, align, out.row_of.data_ptr(), out.slot_of.data_ptr(), out.counts.data_ptr(),
          out.offsets.data_ptr(), None if work is None else work.data_ptr(),
          _stream(stream, experts.device))
    return out


def expert_pack(x: torch.Tensor, plan: ExpertPlan, out: torch.Tensor = None,
                stream: torch.cuda.Stream = None) -> torch.Tensor:
    """Token rows of a [T,M] view to expert-major rows [rows,M], bit for bit:
    ``out[plan.row_of[t,k]] = x[t]``.

    Gap rows (``plan.align``) are written as zeros, rows behind the last expert
    are left as they were.  The gradient of ``x`` is :func:`expert_merge` of the
    gradient of the result.  No graph is recorded: an ``x`` that requires a
    gradient is refused while grad mode is on.
    """
    typ = _rows_type(x, "x")
    _unrecorded(x, "x", "expert_merge")
    T, M = _matrix(x, "x")
    dims = _check_plan(plan, T)
    out = _rows_out(out, stream, x, (dims[2], M), x.dtype, "out")
    d = _expert_desc(typ, plan, dims, M)
    _set_tokens(d, x)
    d.packed = out.data_ptr()
    _expert_call("vf_expert_pack", d, stream, x)
    return out


def expert_merge(packed: torch.Tensor, plan: ExpertPlan, weights: torch.Tensor = None,
                 out: torch.Tensor = None, stream: torch.cuda.Stream = None) -> torch.Tensor:
    """Expert-major rows [rows,M] back to tokens [T,M]: the sum over k of
    ``weights[t,k] * packed[plan.row_of[t,k]]`` (float32 weights; None: the
    plain sum), dropped slots left out, summed in float32 and rounded once.

    ``out`` may be any non-overlapping [T,M] view.  The gradient of ``packed``
    without weights is :func:`expert_pack` of the gradient of the result; with
    weights see :func:`expert_merge_backward`.  No graph is recorded: rows or
    weights that require a gradient are refused while grad mode is on.
    """
    typ = _rows_type(packed, "packed")
    _unrecorded(packed, "packed", "expert_pack" if weights is None else "expert_merge_backward")
    rows, M = _matrix(packed, "packed")
    dims = _check_plan(plan)
    T, K = dims[:2]
    _rows_out(packed, stream, packed, (dims[2], M), packed.dtype, "packed")
    out = _tokens_out(out, stream, packed, (T, M), packed.dtype, "out")
    d = _expert_desc(typ, plan, dims, M)
    _set_tokens(d, out)
    _set_weights(d, weights, T, K)
    if weights is not None:
        _unrecorded(weights, "weights", "expert_merge_backward")
    d.packed = packed.data_ptr()
    _expert_call("vf_expert_merge", d, stream, packed)
    return out


def _backward(grad, plan, weights, grad_packed, grad_weights, stream):
    """What the two backward passes share: (descriptor, gradients, dims)."""
    typ = _rows_type(grad, "grad")
    T, M = _matrix(grad, "grad")
    dims = _check_plan(plan, T)
    if weights is None:
        raise ValueError("weights are required (without, the gradient is expert_pack)")
    grad_packed = _rows_out(grad_packed, stream, grad, (dims[2], M), grad.dtype, "grad_packed")
    grad_weights = _rows_out(grad_weights, stream, grad, (T, dims[1]), torch.float32,
                             "grad_weights")
    d = _expert_desc(typ, plan, dims, M)
    _set_tokens(d, grad)
    _set_weights(d, weights, T, dims[1])
    d.grad_packed, d.grad_weights = grad_packed.data_ptr(), grad_weights.data_ptr()
    return d, grad_packed, grad_weights, dims


def expert_merge_backward(grad: torch.Tensor, packed: torch.Tensor, plan: ExpertPlan,
                          weights: torch.Tensor, grad_packed: torch.Tensor = None,
                          grad_weights: torch.Tensor = None,
                          stream: torch.cuda.Stream = None):
    """Gradients of :func:`expert_merge` with weights, given the gradient
    ``grad`` [T,M] of its result: (grad_packed [rows,M], grad_weights [T,K]).

    ``grad_packed[row_of[t,k]] = weights[t,k] * grad[t]`` (gap rows zero, rows
    behind the last expert left as they were); ``grad_weights[t,k]`` is the dot
    product of ``grad[t]`` and the slot's row, 0 for a dropped slot.
    """
    d, grad_packed, grad_weights, dims = _backward(grad, plan, weights, grad_packed,
                                                   grad_weights, stream)
    _rows_out(packed, stream, grad, (dims[2], grad.shape[1]), grad.dtype, "packed")
    d.packed = packed.data_ptr()
    _expert_call("vf_expert_merge_backward", d, stream, grad)
    return grad_packed, grad_weights


def _bf16_matrix(t, what):
    if isinstance(t, torch.Tensor) and t.dtype != torch.bfloat16:
        raise ValueError("%s must hold bfloat16 values" % what)
    _gpu_addressable(t, what)
    return _matrix(t, what)


def expert_pack_q(x: torch.Tensor, plan: ExpertPlan, fmt="e4m3", group: int = 128,
                  out: torch.Tensor = None, codes: torch.Tensor = None,
                  scales: torch.Tensor = None, stream: torch.cuda.Stream = None):
    """:func:`expert_pack` of bfloat16 tokens that also keeps them in 8 bits for
    the backward pass -> (packed, codes [T,M], scales [T, ceil(M/group)]).

    The packed rows are exact; the checkpoint takes 1/(2K) of their memory, and
    :func:`expert_restore_q` packs it again when the backward pass needs the
    rows.  Each ``group`` consecutive elements share a scale, in the format of
    the lossy transport.
    """
    T, M = _bf16_matrix(x, "x")
    _unrecorded(x, "x", "expert_merge")
    f = _fmt(fmt)
    dims = _check_plan(plan, T)
    codes, scales = _kept(codes, scales, stream, x, T, M, f, group)
    out = _rows_out(out, stream, x, (dims[2], M), x.dtype, "out")
    d = _expert_desc(0, plan, dims, M)
    _set_tokens(d, x)
    _set_kept(d, codes, scales, f, group)
    d.packed = out.data_ptr()
    _expert_call("vf_expert_pack", d, stream, x)
    return out, codes, scales


def expert_restore_q(codes: torch.Tensor, scales: torch.Tensor, plan: ExpertPlan, fmt="e4m3",
                     group: int = 128, out: torch.Tensor = None,
                     stream: torch.cuda.Stream = None) -> torch.Tensor:
    """Expert-major bfloat16 rows [rows,M] of a checkpoint that
    :func:`expert_pack_q` kept (gap rows and the rows behind as there)."""
    f = _fmt(fmt)
    _gpu_addressable(codes, "codes")
    T, M = _matrix(codes, "codes")
    dims = _check_plan(plan, T)
    if scales is None:
        raise ValueError("scales are required")
    _kept(codes, scales, stream, codes, T, M, f, group)
    out = _rows_out(out, stream, codes, (dims[2], M), torch.bfloat16, "out")
    d = _expert_desc(0, plan, dims, M)
    _set_kept(d, codes, scales, f, group)
    d.packed = out.data_ptr()
    _expert_call("vf_expert_restore", d, stream, codes)
    return out


def expert_merge_q(packed: torch.Tensor, plan: ExpertPlan, weights: torch.Tensor = None,
                   fmt="e4m3", group: int = 128, out: torch.Tensor = None,
                   codes: torch.Tensor = None, scales: torch.Tensor = None,
                   stream: torch.cuda.Stream = None):
    """:func:`expert_merge` of bfloat16 rows that also keeps the rows in 8 bits
    for :func:`expert_merge_backward_q` -> (merged [T,M], codes [rows,M],
    scales [rows, ceil(M/group)]).  Rows that no slot owns are not written."""
    rows, M = _bf16_matrix(packed, "packed")
    _unrecorded(packed, "packed", "expert_pack" if weights is None else
                "expert_merge_backward_q")
    f = _fmt(fmt)
    dims = _check_plan(plan)
    T, K = dims[:2]
    _rows_out(packed, stream, packed, (dims[2], M), packed.dtype, "packed")
    codes, scales = _kept(codes, scales, stream, packed, rows, M, f, group)
    out = _tokens_out(out, stream, packed, (T, M), packed.dtype, "out")
    d = _expert_desc(0, plan, dims, M)
    _set_tokens(d, out)
    _set_weights(d, weights, T, K)
    if weights is not None:
        _unrecorded(weights, "weights", "expert_merge_backward_q")
    _set_kept(d, codes, scales, f, group)
    d.packed = packed.data_ptr()
    _expert_call("vf_expert_merge", d, stream, packed)
    return out, codes, scales


def expert_merge_backward_q(grad: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                            plan: ExpertPlan, weights: torch.Tensor, fmt="e4m3",
                            group: int = 128, grad_packed: torch.Tensor = None,
                            grad_weights: torch.Tensor = None,
                            stream: torch.cuda.Stream = None):
    """:func:`expert_merge_backward` with the expert rows read from the
    checkpoint that :func:`expert_merge_q` kept; only ``grad_weights`` depends
    on it."""
    _bf16_matrix(grad, "grad")
    f = _fmt(fmt)
    d, grad_packed, grad_weights, dims = _backward(grad, plan, weights, grad_packed,
                                                   grad_weights, stream)
    if codes is None or scales is None:
        raise ValueError("codes and scales are required")
    _kept(codes, scales, stream, grad, dims[2], grad.shape[1], f, group)
    _set_kept(d, codes, scales, f, group)
    _expert_call("vf_expert_merge_backward", d, stream, grad)
    return grad_packed, grad_weights


# ---- expert products -------------------------------------------------------------

def _desc_call(fn, desc, stream, like):
    rc = getattr(_lib or lib(), fn)(desc, _stream(stream, like.device))
    if rc != 0:
        raise VFError(fn, rc)


def _product_call(fn, desc, stream, like):
    """A product; with a workspace where the library asks for one."""
    f = getattr(_lib or lib(), fn)
    handle = _stream(stream, like.device)
    rc = f(desc + b"\0" * 8, handle)
    if rc == -5:                                           # operands that need a copy
        size = getattr(_lib, fn + "_workspace")(desc + b"\0" * 8)
        if size < 0:
            raise VFError(fn + "_workspace", size)
        work = _workspace(stream, like, -(-size // 4))
        rc = f(desc + _POINTER.pack(work.data_ptr()), handle)
    if rc != 0:
        raise VFError(fn, rc)


def _product_rows(t, what):
    """vf_type of contiguous packed rows that a product takes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % what)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    f = _TYPES.get(t.dtype)
    if f is None or f == 2:
        raise ValueError("%s must hold bfloat16 or float16 values" % what)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return f


def _packed_plan(plan, n):
    """(T, K, rows, E) of a plan for n packed rows."""
    dims = _check_plan(plan)
    if n != dims[2]:
        raise ValueError("plan is for %d packed rows, not %d" % (dims[2], n))
    return dims


def expert_product(rows: torch.Tensor, weights: torch.Tensor, plan: ExpertPlan,
                   out: torch.Tensor = None, stream: torch.cuda.Stream = None) -> torch.Tensor:
    """Expert-major rows [rows,M] times their experts' weights, an [E,N,M] view
    of any strides -> [rows,N]: ``out[r] = weights[e(r)] @ rows[r]``, bfloat16 or
    float16, summed in float32 and rounded once.

    Gap rows (``plan.align``) are written as zeros, rows behind the last expert
    are left as they were; what such rows hold in ``rows`` does not matter.  The
    gradient of ``rows`` is ``expert_product(grad, weights.transpose(1, 2), plan)``,
    that of ``weights`` :func:`expert_weight_grad`.  No graph is recorded: rows
    or weights that require a gradient are refused while grad mode is on.

    M that is no multiple of 8, or operands that do not start at multiples of 16
    bytes, cost a copy of what is read of them (for weights without unit stride along
    N or M too).
    """
    typ = _product_rows(rows, "rows")
    _unrecorded(rows, "rows", "expert_product with the transposed weights")
    n, M = _matrix(rows, "rows")
    T, K, _, E = _packed_plan(plan, n)
    if not (isinstance(weights, torch.Tensor) and weights.is_cuda):
        _product_rows(weights, "weights")                  # raises
    w = weights.shape
    if weights.dtype != rows.dtype or len(w) != 3 or w[0] != E or w[2] != M:
        raise ValueError("weights must be a %s view of shape [%d,N,%d]" % (rows.dtype, E, M))
    _unrecorded(weights, "weights", "expert_weight_grad")
    N = w[1]
    out = _rows_out(out, stream, rows, (n, N), rows.dtype, "out")
    _product_call("vf_expert_product", _PRODUCT_DESC.pack(
        typ, typ, E, N, M, n, T * K, plan[4], plan[2].data_ptr(), plan[3].data_ptr(),
        rows.data_ptr(), weights.data_ptr(), *weights.stride(), 0, out.data_ptr(), 0),
        stream, rows)
    return out


def expert_weight_grad(grad: torch.Tensor, rows: torch.Tensor, plan: ExpertPlan,
                       out: torch.Tensor = None, dtype: torch.dtype = None,
                       stream: torch.cuda.Stream = None) -> torch.Tensor:
    """The gradient of :func:`expert_product`'s weights [E,N,M], given the
    gradient ``grad`` [rows,N] of its result: for each expert the sum over its
    rows of the outer products of ``grad[r]`` and ``rows[r]``; zeros for an expert
    without rows.

    ``dtype`` is the result's: that of ``rows`` (default) or float32.  Gap rows
    and the rows behind the last expert are not read into it.
    """
    typ = _product_rows(grad, "grad")
    if _product_rows(rows, "rows") != typ:
        raise ValueError("grad and rows must have one type")
    n, N = _matrix(grad, "grad")
    n_rows, M = _matrix(rows, "rows")
    if n_rows != n:
        raise ValueError("grad and rows must have the same number of rows")
    if dtype is None:
        dtype = rows.dtype if out is None else out.dtype
    if dtype != rows.dtype and dtype != torch.float32:
        raise ValueError("dtype must be that of rows or torch.float32")
    T, K, _, E = _packed_plan(plan, n)
    out = _rows_out(out, stream, rows, (E, N, M), dtype, "out")
    _product_call("vf_expert_weight_grad", _PRODUCT_DESC.pack(
        typ, _TYPES[dtype], E, N, M, n, T * K, plan[4], plan[2].data_ptr(), plan[3].data_ptr(),
        rows.data_ptr(), 0, 0, 0, 0, grad.data_ptr(), 0, out.data_ptr()), stream, grad)
    return out


# ---- gated activation ------------------------------------------------------------

_NO_VIEW = (0, 0, 0)


def _view(t):
    s = t.stride()
    return t.data_ptr(), s[0], s[1]


def _same_view(t, like, what):
    """Check a view of ``like``'s shape and type."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        _gpu_addressable(t, what)
    if t.dtype != like.dtype or t.shape != like.shape:
        raise ValueError("%s must be a %s view of shape %s" % (what, like.dtype,
                                                               tuple(like.shape)))


def _glu(gate, up, plan):
    """The descriptor's fields that both calls fill in."""
    typ = _rows_type(gate, "gate")
    n, F = _matrix(gate, "gate")
    _same_view(up, gate, "up")
    E = _packed_plan(plan, n)[3]
    return (typ, E, n, F, plan[1].data_ptr(), plan[3].data_ptr(), *_view(gate), *_view(up))


def expert_glu(gate: torch.Tensor, up: torch.Tensor, plan: ExpertPlan,
               out: torch.Tensor = None, stream: torch.cuda.Stream = None) -> torch.Tensor:
    """The gated activation of expert-major rows, ``silu(gate) * up``, of two
    [rows,F] views (the halves of a product's rows), bfloat16, float16 or float32;
    computed in float32 and rounded once.

    Gap rows are written as zeros, rows behind the last expert are left as they
    were.  ``out`` may be any non-overlapping [rows,F] view.  No graph is recorded
    (the gradient is :func:`expert_glu_backward`): views that require a gradient
    are refused while grad mode is on.
    """
    fields = _glu(gate, up, plan)
    _unrecorded(gate, "gate", "expert_glu_backward")
    _unrecorded(up, "up", "expert_glu_backward")
    out = _tokens_out(out, stream, gate, gate.shape, gate.dtype, "out")
    _desc_call("vf_expert_glu", _GLU_DESC.pack(*fields, *_view(out), *_NO_VIEW * 3), stream, gate)
    return out


def expert_glu_backward(grad: torch.Tensor, gate: torch.Tensor, up: torch.Tensor,
                        plan: ExpertPlan, grad_gate: torch.Tensor = None,
                        grad_up: torch.Tensor = None, stream: torch.cuda.Stream = None):
    """Gradients of :func:`expert_glu`, given the gradient ``grad`` [rows,F] of its
    result: (grad_gate, grad_up), by default the halves of one [rows,2F] buffer,
    the rows' gradient of the product in front.  Gap rows are written as zeros, rows
    behind the last expert are left as they were."""
    fields = _glu(gate, up, plan)
    _same_view(grad, gate, "grad")
    shape, dtype = gate.shape, gate.dtype
    if grad_gate is None and grad_up is None:
        n, F = shape
        both = _new(stream, gate, (n, 2 * F), dtype)
        grad_gate, grad_up = both[:, :F], both[:, F:]
    grad_gate = _tokens_out(grad_gate, stream, gate, shape, dtype, "grad_gate")
    grad_up = _tokens_out(grad_up, stream, gate, shape, dtype, "grad_up")
    _desc_call("vf_expert_glu_backward", _GLU_DESC.pack(
        *fields, *_NO_VIEW, *_view(grad), *_view(grad_gate), *_view(grad_up)), stream, gate)
    return grad_gate, grad_up


# ---- root-mean-square norm -------------------------------------------------------

def _norm(x, weight):
    """(vf_type, the weight's, T, M) of the arguments that all calls take."""
    typ = _rows_type(x, "x")
    T, M = _matrix(x, "x")
    if not (isinstance(weight, torch.Tensor) and weight.is_cuda):
        _gpu_addressable(weight, "weight")
    w = weight.dtype
    if w != x.dtype and w != torch.float32:
        raise ValueError("weight must have the type of x or float32")
    if weight.shape != (M,) or not weight.is_contiguous():
        raise ValueError("weight must be contiguous with %d elements" % M)
    return typ, _TYPES[w], T, M


def _norm_inputs(x, weight, residual, total, stream):
    """The total's tensor (None without a residual), and the descriptor's fields of
    both."""
    _unrecorded(x, "x", "rms_norm_backward")
    _unrecorded(weight, "weight", "rms_norm_backward")
    if residual is None:
        if total is not None:
            raise ValueError("total is written only with a residual")
        return None, _NO_VIEW + _NO_VIEW
    _same_view(residual, x, "residual")
    _unrecorded(residual, "residual", "rms_norm_backward")
    total = _tokens_out(total, stream, x, x.shape, x.dtype, "total")
    return total, _view(residual) + _view(total)


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
             residual: torch.Tensor = None, out: torch.Tensor = None,
             total: torch.Tensor = None, stream: torch.cuda.Stream = None):
    """Root-mean-square norm of the rows of a [T,M] view (any strides; bfloat16,
    float16 or float32): ``out = h / sqrt(mean(h^2) + eps) * weight``, computed in
    float32 and rounded once.  weight: [M], of x's type or float32.

    With a ``residual`` h is ``x + residual``, rounded to the type, and the call
    returns (out, total) with h in ``total``; else h is x and it returns out.  ``out``
    and ``total`` may be any non-overlapping [T,M] views.  No graph is recorded (the
    gradients are :func:`rms_norm_backward`): tensors that require a gradient are
    refused while grad mode is on.

    Rows that all start at multiples of 16 bytes give the same bits in any batch.  Where
    they do not (M odd, odd row strides), a row's last bits may go by its address, and views
    that lie otherwise than x (a residual that is a slice of wider rows) are read element
    by element, which takes about twice as long; so does a weight at no such multiple.
    """
    typ, wtyp, T, M = _norm(x, weight)
    total, sums = _norm_inputs(x, weight, residual, total, stream)
    out = _tokens_out(out, stream, x, x.shape, x.dtype, "out")
    _desc_call("vf_rms_norm", _NORM_DESC.pack(
        typ, wtyp, 0, eps, T, M, 0, *_view(x), weight.data_ptr(), *sums, *_view(out), 0, 0,
        0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0), stream, x)
    return out if total is None else (out, total)


def rms_norm_q(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, fmt="e4m3",
               group: int = 128, residual: torch.Tensor = None, codes: torch.Tensor = None,
               scales: torch.Tensor = None, total: torch.Tensor = None,
               stream: torch.cuda.Stream = None):
    """:func:`rms_norm` of bfloat16 rows to 8 bits -> (codes [T,M], scales
    [T, ceil(M/group)]), with a residual (codes, scales, total).  Each ``group``
    consecutive columns of the float32 result share a scale, in the format of the
    lossy transport: what :func:`expert_restore_q` packs to expert-major rows."""
    _bf16_matrix(x, "x")
    f = _fmt(fmt)
    typ, wtyp, T, M = _norm(x, weight)
    total, sums = _norm_inputs(x, weight, residual, total, stream)
    codes, scales = _kept(codes, scales, stream, x, T, M, f, group)
    _desc_call("vf_rms_norm", _NORM_DESC.pack(
        typ, wtyp, f, eps, T, M, group, *_view(x), weight.data_ptr(), *sums, 0, 0, 0,
        codes.data_ptr(), scales.data_ptr(), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0), stream, x)
    return (codes, scales) if total is None else (codes, scales, total)


def rms_norm_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                      eps: float = 1e-6, grad_total: torch.Tensor = None,
                      grad_x: torch.Tensor = None, grad_weight: torch.Tensor = None,
                      stream: torch.cuda.Stream = None):
    """Gradients of :func:`rms_norm` -> (grad_x [T,M], grad_weight [M] float32),
    given the gradient ``grad`` of its result and ``x``, the rows that were normed
    (with a residual its ``total``).

    ``grad_total`` [T,M], if given, is the gradient that reaches those rows by other
    paths (the residual stream's) and is added.  With a residual ``grad_x`` is the
    gradient of both summands.
    """
    typ, wtyp, T, M = _norm(x, weight)
    _same_view(grad, x, "grad")
    more = _NO_VIEW
    if grad_total is not None:
        _same_view(grad_total, x, "grad_total")
        more = _view(grad_total)
    grad_x = _tokens_out(grad_x, stream, x, x.shape, x.dtype, "grad_x")
    grad_weight = _rows_out(grad_weight, stream, x, (M,), torch.float32, "grad_weight")
    size = lib().vf_rms_norm_workspace(T, M)
    if size < 0:
        raise VFError("vf_rms_norm_workspace", size)
    work = _workspace(stream, x, size // 4)
    _desc_call("vf_rms_norm_backward", _NORM_DESC.pack(
        typ, wtyp, 0, eps, T, M, 0, *_view(x), weight.data_ptr(), 0, 0, 0, 0, 0, 0, 0, 0, 0,
        0, 0, *_view(grad), *more, *_view(grad_x), grad_weight.data_ptr(), work.data_ptr()),
        stream, x)
    return grad_x, grad_weight
