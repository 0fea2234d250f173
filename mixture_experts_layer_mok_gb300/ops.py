"""The operators around the layer: the norm with the residual's addition and
an MXFP8 output, the MXFP8 reader, the dense projection with its epilogue, and
their gradients (argument marshalling
only; the arithmetic is in libmok's kernels, ``include/mok.h``).

Every call takes ``stream``: the work, and the memory of what the call
allocates, then belong to that stream instead of the current one.  As for the
layer's calls, tensors are contiguous, on the GPU and 16-byte aligned.
"""
from __future__ import annotations

import contextlib
import ctypes as C
from dataclasses import dataclass

import torch

from . import _lib

_DTYPE = {torch.bfloat16: _lib.MOK_DTYPE_BF16, torch.float32: _lib.MOK_DTYPE_F32}
_NO_STREAM = contextlib.nullcontext()


def _on(stream):
    """The context that allocations of a call on ``stream`` are made in."""
    return _NO_STREAM if stream is None else torch.cuda.stream(stream)


def _handle():
    return torch.cuda.current_stream().cuda_stream


def _check(t, name, shape=None, dtypes=(torch.bfloat16,)):
    if t is None:
        raise ValueError(f"{name} is required")
    if not t.is_cuda or t.dtype not in dtypes or not t.is_contiguous() or (shape is not None and t.shape != shape):
        want = " or ".join(str(d) for d in dtypes)
        raise ValueError(f"{name}: expected contiguous CUDA {want}{'' if shape is None else ' ' + str(tuple(shape))}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}{'' if t.is_contiguous() else ', strided'}")
    return t


def _opt(t):
    return None if t is None else t.data_ptr()


_BF16_F32 = (torch.bfloat16, torch.float32)


def mxfp8_dequantize(codes: torch.Tensor, scales: torch.Tensor, stream=None) -> torch.Tensor:
    """The bf16 values of MXFP8 ``codes`` uint8 [..., K] with ``scales`` uint8
    [..., ceil(K/32)], as ``mxfp8_quantize``, ``rms_norm`` and the optimiser's
    states hold them.  K % 32 == 0, or a single row of any length."""
    _check(codes, "codes", None, (torch.uint8,))
    if codes.dim() < 1:
        raise ValueError("codes: expected at least one dimension")
    K = codes.shape[-1]
    _check(scales, "scales", codes.shape[:-1] + ((K + 31) // 32,), (torch.uint8,))
    lib = _lib.load()
    rows = codes.numel() // K if K else 0
    with _on(stream):
        out = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
        _lib.check(lib.mok_mxfp8_dequantize(codes.data_ptr(), scales.data_ptr(), rows, K, out.data_ptr(), _handle()),
                   "mok_mxfp8_dequantize")
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
    _check(x, "x", None, _BF16_F32)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x: expected a last axis of at least one element")
    H = x.shape[-1]
    _check(weight, "weight", (H,), _BF16_F32)
    if residual is not None:
        _check(residual, "residual", x.shape, _BF16_F32)
    if not bf16 and not mxfp8:
        raise ValueError("ask for bf16, mxfp8 or both")
    if mxfp8 and H % 32:
        raise ValueError("the MXFP8 output needs a last axis that is a multiple of 32")
    lib = _lib.load()
    dev, lead = x.device, x.shape[:-1]
    with _on(stream):
        y = torch.empty(x.shape, dtype=torch.bfloat16, device=dev) if bf16 else None
        codes = torch.empty(x.shape, dtype=torch.uint8, device=dev) if mxfp8 else None
        scales = torch.empty(lead + (H // 32,), dtype=torch.uint8, device=dev) if mxfp8 else None
        rstd = torch.empty(lead, dtype=torch.float32, device=dev)
        h = x if residual is None else torch.empty_like(residual)
        _lib.check(lib.mok_rms_norm(x.data_ptr(), _DTYPE[x.dtype], _opt(residual),
                                    0 if residual is None else _DTYPE[residual.dtype], weight.data_ptr(),
                                    _DTYPE[weight.dtype], x.numel() // H, H, eps,
                                    None if residual is None else h.data_ptr(), _opt(y), _opt(codes), _opt(scales),
                                    rstd.data_ptr(), _handle()), "mok_rms_norm")
    return NormOutput(y, (codes, scales) if mxfp8 else None, h, rstd)


def rms_norm_backward(dy, h, weight, rstd, d_h=None, bf16_dx: bool = False, stream=None) -> dict:
    """Gradients of ``rms_norm``: dy bf16 [..., H]; h, rstd from its output;
    ``d_h`` the gradient that reaches h from its other uses (the residual
    stream), in h's type.  Returns dx in h's type, the gradient of x and of
    the residual alike, and d_weight fp32 [H]; with ``bf16_dx`` and an fp32 h
    also dx_bf16."""
    _check(h, "h", None, _BF16_F32)
    if h.dim() < 1 or h.shape[-1] < 1:
        raise ValueError("h: expected a last axis of at least one element")
    H = h.shape[-1]
    _check(dy, "dy", h.shape)
    _check(weight, "weight", (H,), _BF16_F32)
    _check(rstd, "rstd", h.shape[:-1], (torch.float32,))
    if d_h is not None:
        _check(d_h, "d_h", h.shape, (h.dtype,))
    lib = _lib.load()
    rows = h.numel() // H
    nbytes = lib.mok_rms_norm_bwd_workspace_bytes(rows, H)
    if nbytes == 0:
        raise ValueError("shape outside the kernels' contract")
    with _on(stream):
        out = {"dx": torch.empty_like(h), "d_weight": torch.empty(H, dtype=torch.float32, device=h.device)}
        if bf16_dx and h.dtype == torch.float32:
            out["dx_bf16"] = torch.empty(h.shape, dtype=torch.bfloat16, device=h.device)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=h.device)
        _lib.check(lib.mok_rms_norm_bwd(dy.data_ptr(), h.data_ptr(), _DTYPE[h.dtype], weight.data_ptr(),
                                        _DTYPE[weight.dtype], rstd.data_ptr(), _opt(d_h), rows, H,
                                        out["dx"].data_ptr(), _opt(out.get("dx_bf16")), out["d_weight"].data_ptr(),
                                        ws.data_ptr(), ws.numel(), _handle()), "mok_rms_norm_bwd")
    return out


def _activation(name):
    if name not in _lib.ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_lib.ACTIVATIONS)}")
    return _lib.ACTIVATIONS[name]


def _linear_dims(x, weight):
    _check(weight, "weight")
    if weight.dim() != 2 or weight.shape[0] % 8 or weight.shape[1] % 8 or 0 in weight.shape:
        raise ValueError(f"weight: expected [N, K] with N and K positive multiples of 8, got {tuple(weight.shape)}")
    _check(x, "x")
    if x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError(f"x: expected a last axis of {weight.shape[1]}, got {tuple(x.shape)}")
    N, K = weight.shape
    return x.numel() // K, N, K


def linear(x, weight, bias=None, activation: str = "none", residual=None, out_dtype=torch.bfloat16,
           save_z: bool = False, stream=None):
    """y = act(x weight^T + bias) + residual; returns (y, z).  x bf16 [..., K],
    weight bf16 [N, K] (N and K multiples of 8); bias [N] and residual
    [..., N], bf16 or fp32; ``activation`` "none", "relu", "silu", "gelu" (by
    erf) or "gelu_tanh".  y has ``out_dtype`` (bf16 or fp32), rounded once from
    fp32.  ``save_z`` keeps the pre-activations in bf16 for ``linear_backward``
    (else z is None)."""
    M, N, K = _linear_dims(x, weight)
    act = _activation(activation)
    if out_dtype not in _DTYPE:
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    shape = x.shape[:-1] + (N,)
    if bias is not None:
        _check(bias, "bias", (N,), _BF16_F32)
    if residual is not None:
        _check(residual, "residual", shape, _BF16_F32)
    lib = _lib.load()
    with _on(stream):
        y = torch.empty(shape, dtype=out_dtype, device=x.device)
        z = torch.empty(shape, dtype=torch.bfloat16, device=x.device) if save_z else None
        _lib.check(lib.mok_linear(x.data_ptr(), weight.data_ptr(), _opt(bias),
                                  0 if bias is None else _DTYPE[bias.dtype], _opt(residual),
                                  0 if residual is None else _DTYPE[residual.dtype], act, M, N, K, y.data_ptr(),
                                  _DTYPE[out_dtype], _opt(z), _handle()), "mok_linear")
    return y, z


def linear_backward(dy, x, weight, z=None, activation: str = "none", bias: bool = False,
                    need=("dx", "d_weight"), stream=None) -> dict:
    """Gradients of ``linear``: dy bf16 or fp32 [..., N], z from its
    ``save_z`` (with an activation).  Returns those of dx bf16 [..., K] and
    d_weight bf16 [N, K] that ``need`` names, and with ``bias`` d_bias fp32
    [N].  The residual's gradient is dy itself."""
    M, N, K = _linear_dims(x, weight)
    act = _activation(activation)
    shape = x.shape[:-1] + (N,)
    _check(dy, "dy", shape, _BF16_F32)
    if act:
        _check(z, "z", shape)
    if not set(need) <= {"dx", "d_weight"}:
        raise ValueError("need names dx and d_weight")
    lib = _lib.load()
    nbytes = lib.mok_linear_bwd_workspace_bytes(M, N, act, _DTYPE[dy.dtype], int(bias))
    if nbytes == 0:
        raise ValueError("shape outside the kernels' contract")
    with _on(stream):
        out = {}
        if "dx" in need:
            out["dx"] = torch.empty_like(x)
        if "d_weight" in need:
            out["d_weight"] = torch.empty_like(weight)
        if bias:
            out["d_bias"] = torch.empty(N, dtype=torch.float32, device=x.device)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        _lib.check(lib.mok_linear_bwd(dy.data_ptr(), _DTYPE[dy.dtype], x.data_ptr(), weight.data_ptr(),
                                      _opt(z) if act else None, act, M, N, K, _opt(out.get("dx")),
                                      _opt(out.get("d_weight")), _opt(out.get("d_bias")), ws.data_ptr(), ws.numel(),
                                      _handle()), "mok_linear_bwd")
    return out


def linear_status() -> int:
    """Synchronises and returns the projections' device status since the last
    call: 0, or MOK_ERR_TIMEOUT when a bounded wait gave up."""
    st = C.c_int32()
    _lib.check(_lib.load().mok_linear_status(C.byref(st)), "mok_linear_status")
    return st.value
