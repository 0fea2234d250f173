"""The operators around the layer: the norm with the residual's addition and
an MXFP8 output, the MXFP8 reader, the dense projection with its epilogue, and
their gradients (argument marshalling
only; the arithmetic is in libmok's kernels, ``include/mok.h``).

Every call takes ``stream``: the work, and the memory of what the call
allocates, then belong to that stream instead of the current one.  As for the
layer's calls, tensors are contiguous, on the current GPU (``stream``'s, where
one is given) and 16-byte aligned.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch

from . import _lib

_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_DTYPE = {_BF16: _lib.MOK_DTYPE_BF16, _F32: _lib.MOK_DTYPE_F32}
_empty = torch.empty
# the current stream's handle by device index; torch.cuda.current_stream()
# builds a Stream object around it, which takes longer than a small launch
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _refuse(t, name, shape, dtypes, dev):
    want = " or ".join(str(d) for d in dtypes)
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a CUDA tensor ({want}), got {type(t).__name__}")
    at = "CUDA" if dev is None else f"cuda:{dev}"
    raise ValueError(f"{name}: expected contiguous {at} {want}{'' if shape is None else ' ' + str(tuple(shape))}, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', strided'}")


def _check(t, name, shape=None, dtypes=(_BF16,), dev=None):
    """Refuses t unless it is contiguous, of the types and the shape, and on
    device `dev`.  None: on the GPU, which is returned, and on the current one:
    the library launches there, whatever device its pointers belong to."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or not t.is_contiguous() or (
            shape is not None and t.shape != shape):
        _refuse(t, name, shape, dtypes, dev)
    at = t.get_device()
    if dev is None:
        if at < 0:
            _refuse(t, name, shape, dtypes, dev)
        if at != _current_device():
            raise ValueError(f"{name} is on cuda:{at}, but the current device (or the stream's) is cuda:{_current_device()}")
    elif at != dev:
        _refuse(t, name, shape, dtypes, dev)
    return at


def _opt(t):
    return None if t is None else t.data_ptr()


def _fail(status, where):
    raise _lib.MokError(status, where)


_BF16_F32 = (torch.bfloat16, torch.float32)


def mxfp8_dequantize(codes: torch.Tensor, scales: torch.Tensor, stream=None) -> torch.Tensor:
    """The bf16 values of MXFP8 ``codes`` uint8 [..., K] with ``scales`` uint8
    [..., ceil(K/32)], as ``mxfp8_quantize``, ``rms_norm`` and the optimiser's
    states hold them.  K % 32 == 0, or a single row of any length."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mxfp8_dequantize(codes, scales)
    at = _check(codes, "codes", None, (_U8,))
    shape = codes.shape
    if not shape:
        raise ValueError("codes: expected at least one dimension")
    K = shape[-1]
    _check(scales, "scales", shape[:-1] + ((K + 31) // 32,), (_U8,), at)
    out = _empty(shape, dtype=_BF16, device=codes.device)
    st = _lib.load().mok_mxfp8_dequantize(codes.data_ptr(), scales.data_ptr(), codes.numel() // K if K else 0, K,
                                          out.data_ptr(), _raw_stream(at))
    if st:
        _fail(st, "mok_mxfp8_dequantize")
    return out


@dataclass
class NormOutput:
    """What ``rms_norm`` returns; ``h`` and ``rstd`` are the backward's."""
    y: torch.Tensor | None                            # bf16 [..., H]
    mx: tuple[torch.Tensor, torch.Tensor] | None      # (codes [..., H], scales [..., H/32])
    h: torch.Tensor                                   # x + residual, or x itself
    rstd: torch.Tensor                                # fp32 [...]


def rms_norm(x, weight, residual=None, eps: float = 1e-6, bf16: bool = True, mxfp8: bool = False, stream=None
             ) -> NormOutput:
    """Root-mean-square norm over the last axis, of x + residual when a
    residual is given: h = x + residual, y = weight * h / sqrt(mean(h^2) + eps),
    in fp32 from the unrounded sum.  x bf16 or fp32 [..., H]; residual of x's
    shape, bf16 or fp32; weight [H], bf16 or fp32.  ``bf16`` and ``mxfp8``
    choose the outputs (``NormOutput``); h has the residual's type."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rms_norm(x, weight, residual, eps, bf16, mxfp8)
    at = _check(x, "x", None, _BF16_F32)
    shape = x.shape
    if not shape or not shape[-1]:
        raise ValueError("x: expected a last axis of at least one element")
    H = shape[-1]
    _check(weight, "weight", (H,), _BF16_F32, at)
    if not bf16 and not mxfp8:
        raise ValueError("ask for bf16, mxfp8 or both")
    dev, lead = x.device, shape[:-1]
    h, h_ptr, res_ptr, res_type = x, None, None, 0
    if residual is not None:
        _check(residual, "residual", shape, _BF16_F32, at)
        h = torch.empty_like(residual)
        h_ptr, res_ptr, res_type = h.data_ptr(), residual.data_ptr(), _DTYPE[residual.dtype]
    y = mx = y_ptr = codes_ptr = scales_ptr = None
    if bf16:
        y = _empty(shape, dtype=_BF16, device=dev)
        y_ptr = y.data_ptr()
    if mxfp8:
        if H % 32:
            raise ValueError("the MXFP8 output needs a last axis that is a multiple of 32")
        mx = (_empty(shape, dtype=_U8, device=dev), _empty((*lead, H // 32), dtype=_U8, device=dev))
        codes_ptr, scales_ptr = mx[0].data_ptr(), mx[1].data_ptr()
    rstd = _empty(lead, dtype=_F32, device=dev)
    st = _lib.load().mok_rms_norm(x.data_ptr(), _DTYPE[x.dtype], res_ptr, res_type, weight.data_ptr(),
                                  _DTYPE[weight.dtype], x.numel() // H, H, eps, h_ptr, y_ptr, codes_ptr, scales_ptr,
                                  rstd.data_ptr(), _raw_stream(at))
    if st:
        _fail(st, "mok_rms_norm")
    return NormOutput(y, mx, h, rstd)


def rms_norm_backward(dy, h, weight, rstd, d_h=None, bf16_dx: bool = False, stream=None, f32_dx: bool = False) -> dict:
    """Gradients of ``rms_norm``: dy bf16 [..., H]; h, rstd from its output;
    ``d_h`` the gradient that reaches h from its other uses (the residual
    stream), in h's type.  Returns dx in h's type, the gradient of x and of
    the residual alike, and d_weight fp32 [H]; with ``bf16_dx`` and an fp32 h
    also dx_bf16, with ``f32_dx`` and a bf16 h also dx_f32 (each rounded once,
    for an x of another type than the residual's)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rms_norm_backward(dy, h, weight, rstd, d_h, bf16_dx, f32_dx=f32_dx)
    at = _check(h, "h", None, _BF16_F32)
    shape = h.shape
    if not shape or not shape[-1]:
        raise ValueError("h: expected a last axis of at least one element")
    H = shape[-1]
    _check(dy, "dy", shape, dev=at)
    _check(weight, "weight", (H,), _BF16_F32, at)
    _check(rstd, "rstd", shape[:-1], (_F32,), at)
    if d_h is not None:
        _check(d_h, "d_h", shape, (h.dtype,), at)
    lib, dev = _lib.load(), h.device
    rows = h.numel() // H
    nbytes = lib.mok_rms_norm_bwd_workspace_bytes(rows, H)
    if nbytes == 0:
        raise ValueError("shape outside the kernels' contract")
    out = {"dx": torch.empty_like(h), "d_weight": _empty((H,), dtype=_F32, device=dev)}
    other = None
    if bf16_dx and h.dtype == _F32:
        other = out["dx_bf16"] = _empty(shape, dtype=_BF16, device=dev)
    elif f32_dx and h.dtype == _BF16:
        other = out["dx_f32"] = _empty(shape, dtype=_F32, device=dev)
    ws = _empty((nbytes,), dtype=_U8, device=dev)
    st = lib.mok_rms_norm_bwd_both(dy.data_ptr(), h.data_ptr(), _DTYPE[h.dtype], weight.data_ptr(), _DTYPE[weight.dtype],
                                   rstd.data_ptr(), _opt(d_h), rows, H, out["dx"].data_ptr(), _opt(other),
                                   out["d_weight"].data_ptr(), ws.data_ptr(), nbytes, _raw_stream(at))
    if st:
        _fail(st, "mok_rms_norm_bwd_both")
    return out


def _linear_args(x, weight, activation):
    """(M, N, K, activation code, x's leading axes, device) of a projection's checked operands."""
    act = _lib.ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(_lib.ACTIVATIONS)}")
    at = _check(x, "x")
    _check(weight, "weight", dev=at)
    ws, xs = weight.shape, x.shape
    if len(ws) != 2 or ws[0] % 8 or ws[1] % 8 or not ws[0] or not ws[1]:
        raise ValueError(f"weight: expected [N, K] with N and K positive multiples of 8, got {tuple(ws)}")
    if not xs or xs[-1] != ws[1]:
        raise ValueError(f"x: expected a last axis of {ws[1]}, got {tuple(xs)}")
    return x.numel() // ws[1], ws[0], ws[1], act, xs[:-1], at


def linear(x, weight, bias=None, activation: str = "none", residual=None, out_dtype=torch.bfloat16,
           save_z: bool = False, stream=None):
    """y = act(x weight^T + bias) + residual; returns (y, z).  x bf16 [..., K],
    weight bf16 [N, K] (N and K multiples of 8); bias [N] and residual
    [..., N], bf16 or fp32; ``activation`` "none", "relu", "silu", "gelu" (by
    erf) or "gelu_tanh".  y has ``out_dtype`` (bf16 or fp32), rounded once from
    fp32.  ``save_z`` keeps the pre-activations in bf16 for ``linear_backward``
    (else z is None)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear(x, weight, bias, activation, residual, out_dtype, save_z)
    M, N, K, act, lead, at = _linear_args(x, weight, activation)
    shape = (*lead, N)
    out_type = _DTYPE.get(out_dtype)
    if out_type is None:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    bias_ptr, bias_type, res_ptr, res_type, z, z_ptr = None, 0, None, 0, None, None
    if bias is not None:
        _check(bias, "bias", (N,), _BF16_F32, at)
        bias_ptr, bias_type = bias.data_ptr(), _DTYPE[bias.dtype]
    if residual is not None:
        _check(residual, "residual", shape, _BF16_F32, at)
        res_ptr, res_type = residual.data_ptr(), _DTYPE[residual.dtype]
    dev = x.device
    y = _empty(shape, dtype=out_dtype, device=dev)
    if save_z:
        z = _empty(shape, dtype=_BF16, device=dev)
        z_ptr = z.data_ptr()
    st = _lib.load().mok_linear(x.data_ptr(), weight.data_ptr(), bias_ptr, bias_type, res_ptr, res_type, act, M, N, K,
                                y.data_ptr(), out_type, z_ptr, _raw_stream(at))
    if st:
        _fail(st, "mok_linear")
    return y, z


def linear_backward(dy, x, weight, z=None, activation: str = "none", bias: bool = False,
                    need=("dx", "d_weight"), stream=None) -> dict:
    """Gradients of ``linear``: dy bf16 or fp32 [..., N], z from its
    ``save_z`` (with an activation).  Returns those of dx bf16 [..., K] and
    d_weight bf16 [N, K] that ``need`` names, and with ``bias`` d_bias fp32
    [N].  The residual's gradient is dy itself."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_backward(dy, x, weight, z, activation, bias, need)
    M, N, K, act, lead, at = _linear_args(x, weight, activation)
    shape = (*lead, N)
    _check(dy, "dy", shape, _BF16_F32, at)
    if act:
        _check(z, "z", shape, dev=at)
    lib, dev, dy_type = _lib.load(), x.device, _DTYPE[dy.dtype]
    nbytes = lib.mok_linear_bwd_workspace_bytes(M, N, act, dy_type, bool(bias))
    if nbytes == 0:
        raise ValueError("shape outside the kernels' contract")
    out, ptrs = {}, {}
    for name in need:
        if name == "dx":
            out[name] = torch.empty_like(x)
        elif name == "d_weight":
            out[name] = torch.empty_like(weight)
        else:
            raise ValueError("need names dx and d_weight")
    if bias:
        out["d_bias"] = _empty((N,), dtype=_F32, device=dev)
    for name, t in out.items():
        ptrs[name] = t.data_ptr()
    ws = _empty((nbytes,), dtype=_U8, device=dev)
    st = lib.mok_linear_bwd(dy.data_ptr(), dy_type, x.data_ptr(), weight.data_ptr(), z.data_ptr() if act else None, act,
                            M, N, K, ptrs.get("dx"), ptrs.get("d_weight"), ptrs.get("d_bias"), ws.data_ptr(), nbytes,
                            _raw_stream(at))
    if st:
        _fail(st, "mok_linear_bwd")
    return out


def linear_status() -> int:
    """Synchronises and returns the projections' device status since the last
    call: 0, or MOK_ERR_TIMEOUT when a bounded wait gave up."""
    st = C.c_int32()
    _lib.check(_lib.load().mok_linear_status(C.byref(st)), "mok_linear_status")
    return st.value
