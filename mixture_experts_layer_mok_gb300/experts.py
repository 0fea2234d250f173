"""Routed experts as operators of their own: the router, the projections grouped
by expert with their gradients, and the projections with 4-bit weights
(argument marshalling only; the arithmetic is in libmok's kernels,
``include/mok.h``).

They serve experts that the layer's fixed SwiGLU does not express, and the
decoding of single tokens.  The calls follow those of ``ops``: ``stream``,
contiguous tensors on the current GPU, 16-byte aligned; autograd does not
record them (``autograd.route`` and ``autograd.grouped_linear`` are its faces).
"""
from __future__ import annotations

import ctypes as C
import functools
from dataclasses import dataclass

import torch

from . import _lib, ops
from .ops import _BF16, _BF16_F32, _DTYPE, _F32, _U8, _check, _fail, _opt

_I32, _I64 = torch.int32, torch.int64

# A contiguous tensor on the current device.  A call here makes up to six, and a
# small kernel takes less time than torch.empty's argument parsing does; the
# allocation underneath is the same.  Where something watches over allocations (a
# dispatch or function mode, the filling of fresh memory in deterministic runs),
# they go through torch.empty, which shows them to it.
_strided = getattr(getattr(torch._C._dynamo, "guards", None), "_empty_strided_cuda", None)
_dispatch_modes = getattr(torch._C, "_len_torch_dispatch_stack", None)
_function_modes = getattr(torch._C, "_len_torch_function_stack", None)
if _dispatch_modes is None or _function_modes is None:
    _strided = None


def _new(shape, dtype, dev):
    if _strided is None or _dispatch_modes() or _function_modes() or torch.are_deterministic_algorithms_enabled():
        return ops._empty(shape, dtype=dtype, device=dev)
    shape = tuple(shape)   # (not a torch.Size)
    n = len(shape)
    if n == 1:
        return _strided(shape, (1,), dtype)
    if n == 2:
        return _strided(shape, (max(shape[1], 1), 1), dtype)
    stride, at = [], 1
    for size in shape[::-1]:
        stride.append(at)
        at *= max(size, 1)
    return _strided(shape, tuple(stride[::-1]), dtype)


@functools.lru_cache(maxsize=4096)
def _workspace(name, *sizes):
    return getattr(_lib.load(), name)(*sizes)


# ---------------------------------------------------------------- router
@dataclass
class Routing:
    """What ``route`` returns."""
    experts: torch.Tensor                 # int64 [..., k], largest first
    weights: torch.Tensor                 # fp32 [..., k]
    lse: torch.Tensor                     # fp32 [...]: log sum exp of the logits
    counts: torch.Tensor | None           # int32 [E]: how often each expert was chosen
    mean_score: torch.Tensor | None       # fp32 [E]


def _route_args(logits, k, score):
    s = _lib.SCORES.get(score)
    if s is None:
        raise ValueError(f"score must be one of {sorted(_lib.SCORES)}")
    at = _check(logits, "logits", None, _BF16_F32)
    if not logits.dim() or not 1 <= logits.shape[-1] <= _lib.MOK_ROUTE_MAX_E:
        raise ValueError(f"logits: expected a last axis of 1 to {_lib.MOK_ROUTE_MAX_E} experts, got {tuple(logits.shape)}")
    E = logits.shape[-1]
    if not 1 <= k <= min(E, _lib.MOK_ROUTE_MAX_K):
        raise ValueError(f"k must be 1 to min(experts, {_lib.MOK_ROUTE_MAX_K}), got {k}")
    return logits.numel() // E, E, s, logits.shape[:-1], at


def route(logits, k: int, score: str = "softmax", normalize: bool = True, scale: float = 1.0, bias=None, balance: bool = False,
          stream=None) -> Routing:
    """Each token's k experts and their weights.  logits bf16 or fp32 [..., E];
    scores s = softmax or sigmoid of them; the choice is by s + ``bias`` (fp32
    [E]), ties to the larger logit, and then to the lowest index; weights scale
    s_j / sum of the chosen s, or scale s_j without ``normalize``.  ``balance``:
    also counts and mean_score, for a balance loss.  E up to 1024, k up to 64."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return route(logits, k, score, normalize, scale, bias, balance)
    T, E, s, lead, at = _route_args(logits, k, score)
    if bias is not None:
        _check(bias, "bias", (E,), (_F32,), at)
    lib, dev = _lib.load(), logits.device
    experts = _new((*lead, k), _I64, dev)
    weights = _new((*lead, k), _F32, dev)
    lse = _new(lead, _F32, dev)
    counts = mean = ws = None
    nbytes = 0
    if balance:
        counts = _new((E,), _I32, dev)
        mean = _new((E,), _F32, dev)
        nbytes = _workspace("mok_route_workspace_bytes", T, E)
        ws = _new((nbytes,), _U8, dev)
    st = lib.mok_route(logits.data_ptr(), _DTYPE[logits.dtype], _opt(bias), T, E, k, s, bool(normalize), scale, experts.data_ptr(),
                       weights.data_ptr(), lse.data_ptr(), _opt(counts), _opt(mean), _opt(ws), nbytes, ops._raw_stream(at))
    if st:
        _fail(st, "mok_route")
    return Routing(experts, weights, lse, counts, mean)


def route_backward(d_weights, logits, experts, score: str = "softmax", normalize: bool = True, scale: float = 1.0, d_lse=None,
                   d_mean_score=None, stream=None) -> torch.Tensor:
    """The gradient of the logits, in their type: d_weights fp32 [..., k],
    experts from ``route``, ``d_lse`` fp32 [...] and ``d_mean_score`` fp32 [E]
    where the loss uses these."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return route_backward(d_weights, logits, experts, score, normalize, scale, d_lse, d_mean_score)
    if not isinstance(experts, torch.Tensor) or not experts.dim():
        raise ValueError("experts: expected an int64 tensor [..., k]")
    k = experts.shape[-1]
    T, E, s, lead, at = _route_args(logits, k, score)
    _check(experts, "experts", (*lead, k), (_I64,), at)
    _check(d_weights, "d_weights", (*lead, k), (_F32,), at)
    if d_lse is not None:
        _check(d_lse, "d_lse", lead, (_F32,), at)
    if d_mean_score is not None:
        _check(d_mean_score, "d_mean_score", (E,), (_F32,), at)
    out = _new(logits.shape, logits.dtype, logits.device)
    st = _lib.load().mok_route_bwd(d_weights.data_ptr(), logits.data_ptr(), _DTYPE[logits.dtype], experts.data_ptr(), _opt(d_lse),
                                   _opt(d_mean_score), T, E, k, s, bool(normalize), scale, out.data_ptr(), ops._raw_stream(at))
    if st:
        _fail(st, "mok_route_bwd")
    return out


# ---------------------------------------------------------------- projections grouped by expert
def _grouped_args(x, weight, counts, activation):
    """(M, E, N, K, activation code, device) of checked operands."""
    act = _lib.ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(_lib.ACTIVATIONS)}")
    at = _check(x, "x")
    _check(weight, "weight", dev=at)
    ws = weight.shape
    if len(ws) != 3 or not 1 <= ws[0] <= _lib.MOK_GROUPED_MAX_E or ws[1] % 8 or ws[2] % 8 or not ws[1] or not ws[2]:
        raise ValueError(f"weight: expected [E, N, K] with up to {_lib.MOK_GROUPED_MAX_E} experts, N and K positive multiples of 8, "
                         f"got {tuple(ws)}")
    if x.dim() != 2 or x.shape[1] != ws[2]:
        raise ValueError(f"x: expected [rows, {ws[2]}], got {tuple(x.shape)}")
    _check(counts, "counts", (ws[0],), (_I32,), at)
    return x.shape[0], ws[0], ws[1], ws[2], act, at


def grouped_linear(x, weight, counts, bias=None, activation: str = "none", out_dtype=torch.bfloat16, save_z: bool = False,
                   stream=None):
    """y = act(x weight[e]^T + bias[e]) for rows sorted by expert; returns (y, z).
    x bf16 [M, K]: the rows of expert 0, then those of expert 1 and so on,
    ``counts`` int32 [E] of them, on the device; weight bf16 [E, N, K] (N and K
    multiples of 8), bias [E, N] bf16 or fp32.  y [M, N] has ``out_dtype``
    (bf16 or fp32), rounded once from fp32, with zeros in the rows behind the
    last expert's.  ``save_z`` keeps the pre-activations in bf16 for
    ``grouped_linear_backward`` (else z is None)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return grouped_linear(x, weight, counts, bias, activation, out_dtype, save_z)
    M, E, N, K, act, at = _grouped_args(x, weight, counts, activation)
    out_type = _DTYPE.get(out_dtype)
    if out_type is None:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    bias_type = 0
    if bias is not None:
        _check(bias, "bias", (E, N), _BF16_F32, at)
        bias_type = _DTYPE[bias.dtype]
    y = _new((M, N), out_dtype, x.device)
    z = _new((M, N), _BF16, x.device) if save_z else None
    st = _lib.load().mok_grouped_linear(x.data_ptr(), weight.data_ptr(), counts.data_ptr(), _opt(bias), bias_type, act, M, E, N, K,
                                        y.data_ptr(), out_type, _opt(z), ops._raw_stream(at))
    if st:
        _fail(st, "mok_grouped_linear")
    return y, z


def grouped_linear_backward(dy, x, weight, counts, z=None, activation: str = "none", bias: bool = False,
                            need=("dx", "d_weight"), stream=None) -> dict:
    """Gradients of ``grouped_linear``: dy bf16 or fp32 [M, N], z from its
    ``save_z`` (with an activation).  Returns those of dx bf16 [M, K] and
    d_weight bf16 [E, N, K] that ``need`` names, and with ``bias`` d_bias fp32
    [E, N]; zeros in dx behind the last expert's rows and for experts without
    rows."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return grouped_linear_backward(dy, x, weight, counts, z, activation, bias, need)
    M, E, N, K, act, at = _grouped_args(x, weight, counts, activation)
    _check(dy, "dy", (M, N), _BF16_F32, at)
    if act:
        _check(z, "z", (M, N), dev=at)
    lib, dev, dy_type = _lib.load(), x.device, _DTYPE[dy.dtype]
    nbytes = _workspace("mok_grouped_linear_bwd_workspace_bytes", M, E, N, act, dy_type, bool(bias))
    if nbytes == 0:
        raise ValueError("shape outside the kernels' contract")
    out = {}
    for name in need:
        if name == "dx":
            out[name] = _new((M, K), _BF16, dev)
        elif name == "d_weight":
            out[name] = _new((E, N, K), _BF16, dev)
        else:
            raise ValueError("need names dx and d_weight")
    if bias:
        out["d_bias"] = _new((E, N), _F32, dev)
    ws = _new((nbytes,), _U8, dev)
    st = lib.mok_grouped_linear_bwd(dy.data_ptr(), dy_type, x.data_ptr(), weight.data_ptr(), counts.data_ptr(),
                                    z.data_ptr() if act else None, act, M, E, N, K, _opt(out.get("dx")), _opt(out.get("d_weight")),
                                    _opt(out.get("d_bias")), ws.data_ptr(), nbytes, ops._raw_stream(at))
    if st:
        _fail(st, "mok_grouped_linear_bwd")
    return out


# ---------------------------------------------------------------- 4-bit weights
@dataclass
class Int4Weight:
    """A weight [..., N, K] of one matrix, or of several (one leading axis), in 4
    bits: value = (q - zero) scale, a scale (and a zero) for each ``group``
    columns.  The tensors hold the library's own layout."""
    codes: torch.Tensor             # uint8
    scales: torch.Tensor            # bf16
    zeros: torch.Tensor | None      # uint8, or None: 8 everywhere
    shape: tuple
    group: int


@functools.lru_cache(maxsize=1024)
def _int4_sizes(matrices, N, K, group):
    """Elements of a weight's codes, scales and zeros."""
    lib = _lib.load()
    n = [C.c_size_t() for _ in range(3)]
    st = lib.mok_int4_bytes(matrices, N, K, group, *(C.byref(v) for v in n))
    if st:
        raise ValueError(lib.mok_last_error().decode(errors="replace"))
    return n[0].value, n[1].value // 2, n[2].value


def _int4_new(shape, group, zeros, dev):
    if len(shape) not in (2, 3):
        raise ValueError(f"expected [N, K] or [matrices, N, K], got {tuple(shape)}")
    matrices = shape[0] if len(shape) == 3 else 1
    nc, ns, nz = _int4_sizes(matrices, shape[-2], shape[-1], group)
    w = Int4Weight(_new((nc,), _U8, dev), _new((ns,), _BF16, dev),
                   _new((nz,), _U8, dev) if zeros else None, tuple(shape), group)
    return w, matrices


def _int4_args(weight):
    """(matrices, N, K, device) of a checked weight."""
    if not isinstance(weight, Int4Weight):
        raise ValueError(f"weight: expected an Int4Weight, got {type(weight).__name__}")
    matrices, (N, K) = weight.shape[0] if len(weight.shape) == 3 else 1, weight.shape[-2:]
    nc, ns, nz = _int4_sizes(matrices, N, K, weight.group)
    at = _check(weight.codes, "weight.codes", (nc,), (_U8,))
    _check(weight.scales, "weight.scales", (ns,), (_BF16,), at)
    if weight.zeros is not None:
        _check(weight.zeros, "weight.zeros", (nz,), (_U8,), at)
    return matrices, N, K, at


def int4_quantize(w, group: int = 128, zeros: bool = False, stream=None) -> Int4Weight:
    """w bf16 or fp32 [N, K] or [matrices, N, K] in 4 bits, to the nearest:
    symmetric about 8, or with ``zeros`` over each group's own range.  group 32,
    64 or 128, K a multiple of it.  A group with a NaN or an infinity becomes NaN
    as a whole."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return int4_quantize(w, group, zeros)
    at = _check(w, "w", None, _BF16_F32)
    out, matrices = _int4_new(w.shape, group, zeros, w.device)
    st = _lib.load().mok_int4_quantize(w.data_ptr(), _DTYPE[w.dtype], matrices, *out.shape[-2:], group, out.codes.data_ptr(),
                                       out.scales.data_ptr(), _opt(out.zeros), ops._raw_stream(at))
    if st:
        _fail(st, "mok_int4_quantize")
    return out


def int4_pack(codes, scales, zeros=None, stream=None) -> Int4Weight:
    """An ``Int4Weight`` of codes made elsewhere: uint8 [..., N, K / 2], two to a
    byte, the even column's in the low half; scales bf16 [..., N, K / group],
    zeros uint8 of their shape, 0..15 in the low four bits (the others do not
    count: a zero of 16 would be 0), or None."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return int4_pack(codes, scales, zeros)
    at = _check(codes, "codes", None, (_U8,))
    if codes.dim() not in (2, 3) or not codes.shape[-1]:
        raise ValueError(f"codes: expected [N, K / 2] or [matrices, N, K / 2], got {tuple(codes.shape)}")
    K = 2 * codes.shape[-1]
    _check(scales, "scales", None, (_BF16,), at)
    groups = scales.shape[-1] if scales.dim() else 0
    if scales.shape[:-1] != codes.shape[:-1] or not groups or K % groups:
        raise ValueError(f"scales: expected {tuple(codes.shape[:-1])} and a divisor of {K}, got {tuple(scales.shape)}")
    if zeros is not None:
        _check(zeros, "zeros", scales.shape, (_U8,), at)
    out, matrices = _int4_new((*codes.shape[:-1], K), K // groups, zeros is not None, codes.device)
    st = _lib.load().mok_int4_pack(codes.data_ptr(), scales.data_ptr(), _opt(zeros), matrices, *out.shape[-2:], out.group,
                                   out.codes.data_ptr(), out.scales.data_ptr(), _opt(out.zeros), ops._raw_stream(at))
    if st:
        _fail(st, "mok_int4_pack")
    return out


def int4_dequantize(weight: Int4Weight, stream=None) -> torch.Tensor:
    """The values in bf16 [..., N, K], for ``linear`` and ``grouped_linear`` with
    many rows."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return int4_dequantize(weight)
    matrices, N, K, at = _int4_args(weight)
    out = _new(weight.shape, _BF16, weight.codes.device)
    st = _lib.load().mok_int4_dequantize(weight.codes.data_ptr(), weight.scales.data_ptr(), _opt(weight.zeros), matrices, N, K,
                                         weight.group, out.data_ptr(), ops._raw_stream(at))
    if st:
        _fail(st, "mok_int4_dequantize")
    return out


def int4_linear(x, weight: Int4Weight, bias=None, activation: str = "none", experts=None, out_dtype=torch.bfloat16, stream=None
                ) -> torch.Tensor:
    """y = act(x W^T + bias) with W in 4 bits, for few rows.  One matrix: x bf16
    [..., K], y [..., N], bias [N].  ``experts`` int64 [..., k]: y [..., k, N],
    x [..., K] times each of its row's matrices (or x [..., k, K], a row for
    each), bias [matrices, N]; id -1 gives zeros.  bias bf16 or fp32; y in
    ``out_dtype`` (bf16 or fp32), rounded once from fp32; the weights' values are
    not rounded.  For decoding: autograd does not record it, and y has no graph
    where x requires a gradient; a frozen 4-bit weight that is trained through is
    ``int4_dequantize`` under ``autograd.linear`` or ``autograd.grouped_linear``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return int4_linear(x, weight, bias, activation, experts, out_dtype)
    act = _lib.ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(_lib.ACTIVATIONS)}")
    out_type = _DTYPE.get(out_dtype)
    if out_type is None:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    matrices, N, K, at = _int4_args(weight)
    _check(x, "x", None, (_BF16,), at)
    if not x.dim() or x.shape[-1] != K:
        raise ValueError(f"x: expected a last axis of {K}, got {tuple(x.shape)}")
    lead, each = x.shape[:-1], 1
    if (experts is None) != (len(weight.shape) == 2):
        raise ValueError("a weight of several matrices goes with experts, and one matrix without")
    if experts is not None:
        _check(experts, "experts", None, (_I64,), at)
        if not experts.dim() or not experts.shape[-1]:
            raise ValueError("experts: expected int64 [..., k] with k of at least 1")
        if lead != experts.shape:
            if lead != experts.shape[:-1]:
                raise ValueError(f"x: expected {(*experts.shape[:-1], K)} or {(*experts.shape, K)}, got {tuple(x.shape)}")
            each = experts.shape[-1]
        lead = experts.shape
    bias_type = 0
    if bias is not None:
        _check(bias, "bias", (N,) if experts is None else (matrices, N), _BF16_F32, at)
        bias_type = _DTYPE[bias.dtype]
    rows = x.numel() // K * each
    if rows > _lib.MOK_INT4_MAX_ROWS:
        raise ValueError(f"int4_linear is for up to {_lib.MOK_INT4_MAX_ROWS} rows of y, got {rows}: take int4_dequantize with linear "
                         "or grouped_linear")
    y = _new((*lead, N), out_dtype, x.device)
    st = _lib.load().mok_int4_linear(x.data_ptr(), weight.codes.data_ptr(), weight.scales.data_ptr(), _opt(weight.zeros), matrices, N,
                                     K, weight.group, _opt(experts), rows, each, _opt(bias), bias_type, act, y.data_ptr(), out_type,
                                     ops._raw_stream(at))
    if st:
        _fail(st, "mok_int4_linear")
    return y
