"""torch.autograd face of the layer (``MoKFunction``, ``MoKLayer``) and of the
operators around it (``rms_norm``, ``MoKRMSNorm``; ``linear``, ``MoKLinear``;
``route``, ``MoKRouter``; ``grouped_linear``, ``MoKGroupedLinear``).

The pages' PyTorch-facing pieces are a runtime whose forward returns the
output plus an opaque context and whose backward consumes it, returning
"gradients matching every forward input" ("nemo_automodel.components.moe.
mok_experts": ``_MoKRuntime.forward`` / ``backward``, ``GroupedExpertsMoK``).
This module puts those two calls under torch.autograd, so that a model can
call the layer like any other module.  It only marshals arguments: the
schedule, forward and backward run in libmok's kernels through the binding.
First derivatives only: differentiating a gradient raises RuntimeError.
"""
from __future__ import annotations

import functools

import torch

from . import Context, Schedule, Weights, backward, experts, forward, ops, quantize_weights, schedule


class _NoSecondDerivative(torch.autograd.Function):
    """The identity, with a backward that refuses."""

    @staticmethod
    def forward(ctx, name, *grads):
        ctx.name = name
        return grads

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError(f"{ctx.name}: the gradients come from a kernel and have no derivative of their own")


def _first_order(backward):
    """A backward whose gradients refuse to be differentiated.  Under
    ``create_graph`` they would otherwise pass for constants, and what a loss
    makes of them would be lost without a word; that holds even where the
    incoming gradient needs none, as they depend on the saved tensors too."""

    @functools.wraps(backward)
    def wrapper(ctx, *args):
        with torch.no_grad():
            out = backward(ctx, *args)
        if torch.is_grad_enabled():
            at = [i for i, g in enumerate(out) if g is not None]
            marked = _NoSecondDerivative.apply(type(ctx).__name__.removesuffix("Backward"),
                                               *(out[i].detach().requires_grad_() for i in at))
            out = list(out)
            for i, g in zip(at, marked):
                out[i] = g
            out = tuple(out)
        return out

    return wrapper


def _incoming(grad):
    """A gradient as the library takes it: contiguous, and 16-byte aligned, which
    a contiguous one need not be (the backward of a ``cat`` hands on views)."""
    grad = grad.contiguous()
    return grad.clone() if grad.data_ptr() & 15 else grad


class MoKFunction(torch.autograd.Function):
    """y = MoK layer(x, router_w, top_experts; routed and optional shared
    SwiGLU weights).  Differentiable in x, router_w and every weight; the
    expert ids are integers and get no gradient."""

    @staticmethod
    def forward(ctx, x, router_w, top_experts, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, mode, capacity,
                minibatch, swiglu_limit=0.0, macrobatch=0, x_mx=None):
        E = w_gate.shape[0]
        sched = schedule(top_experts, E, capacity)
        weights = Weights(w_gate, w_up, w_down, ws_gate, ws_up, ws_down)
        if mode in ("mxfp8", "mxfp8_full"):
            weights = quantize_weights(weights, backward=(mode == "mxfp8_full"))
        y, mctx = forward(x, router_w, sched, weights, mode=mode, minibatch=minibatch, swiglu_limit=swiglu_limit,
                          macrobatch=macrobatch, x_mx=x_mx)
        # the schedule and the context go through save_for_backward as their
        # buffers, so saved-tensor hooks (offload, checkpointing) see them
        sbuf, smeta = sched.flatten()
        cbuf, cmeta = mctx.flatten()
        ctx.save_for_backward(x, router_w, sbuf, cbuf)
        ctx.mok = (smeta, cmeta, weights, minibatch, macrobatch, ws_gate is not None)
        return y

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x, router_w, sbuf, cbuf = ctx.saved_tensors
        smeta, cmeta, weights, minibatch, macrobatch, shared = ctx.mok
        sched = Schedule.unflatten(sbuf, smeta)     # over wherever the hooks put the buffers
        mctx = Context.unflatten(cbuf, cmeta)
        g = backward(_incoming(dy.to(torch.bfloat16)), x, router_w, sched, mctx, weights, minibatch=minibatch,
                     macrobatch=macrobatch)
        ctx.mok = None
        return (g["dx"], g["d_router_w"], None, g["d_w_gate"], g["d_w_up"], g["d_w_down"],
                g["d_ws_gate"] if shared else None, g["d_ws_up"] if shared else None,
                g["d_ws_down"] if shared else None, None, None, None, None, None, None)


def mok_layer(x, router_w, top_experts, w_gate, w_up, w_down, ws_gate=None, ws_up=None, ws_down=None,
              mode: str = "bf16", capacity: float = 0.5, minibatch: int = 0, swiglu_limit: float = 0.0,
              macrobatch: int = 0, x_mx=None):
    """Functional form: x bf16 [T, H], router_w fp32 [T, k], top_experts int64
    [T, k]; routed weights [E, I, H], [E, I, H], [E, H, I]; shared weights
    [I_s, H], [I_s, H], [H, I_s] or None.  ``macrobatch``: rows of the token
    ring, forward and backward (0: one pass).  ``x_mx``: x's MXFP8 codes and
    scales (see ``forward``); the quantisation counts as the identity in the
    gradient."""
    return MoKFunction.apply(x, router_w, top_experts, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, mode, capacity,
                             minibatch, swiglu_limit, macrobatch, x_mx)


class MoKLayer(torch.nn.Module):
    """Routed experts (E of them, intermediate size I) plus an optional shared
    expert (intermediate size I_s), in the weight layouts of the pages'
    ``GroupedExpertsMoK``.  The router stays outside (the caller passes the
    chosen experts and their weights), as on the pages."""

    def __init__(self, E: int, H: int, I: int, I_s: int = 0, mode: str = "bf16", capacity: float = 0.5,
                 minibatch: int = 0, swiglu_limit: float = 0.0, macrobatch: int = 0, device=None,
                 init_std: float = 0.02, generator=None):
        super().__init__()
        kw = dict(dtype=torch.bfloat16, device=device)

        def param(*shape):
            t = torch.empty(*shape, **kw)
            t.normal_(0.0, init_std, generator=generator)
            return torch.nn.Parameter(t)

        self.w_gate, self.w_up, self.w_down = param(E, I, H), param(E, I, H), param(E, H, I)
        if I_s:
            self.ws_gate, self.ws_up, self.ws_down = param(I_s, H), param(I_s, H), param(H, I_s)
        else:
            self.ws_gate = self.ws_up = self.ws_down = None
        self.mode, self.capacity, self.minibatch, self.swiglu_limit = mode, capacity, minibatch, swiglu_limit
        self.macrobatch = macrobatch

    def forward(self, x, router_w, top_experts, x_mx=None):
        return mok_layer(x, router_w, top_experts, self.w_gate, self.w_up, self.w_down, self.ws_gate, self.ws_up,
                         self.ws_down, self.mode, self.capacity, self.minibatch, self.swiglu_limit, self.macrobatch,
                         x_mx)


class RMSNormFunction(torch.autograd.Function):
    """(y, h, codes, scales) = norm(x + residual); the last two (empty without
    ``mxfp8``) are integers and get no gradient."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps, mxfp8):
        out = ops.rms_norm(x, weight, residual, eps, mxfp8=mxfp8)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(out.h, weight, out.rstd)
        ctx.types = x.dtype, None if residual is None else residual.dtype
        codes, scales = out.mx if mxfp8 else (x.new_empty(0, dtype=torch.uint8), x.new_empty(0, dtype=torch.uint8))
        ctx.mark_non_differentiable(codes, scales)
        return out.y, x.view_as(x) if residual is None else out.h, codes, scales

    @staticmethod
    @_first_order
    def backward(ctx, dy, dh, _codes, _scales):
        h, weight, rstd = ctx.saved_tensors
        x_type, res_type = ctx.types
        if dy is None and dh is None:
            return None, None, None, None, None
        d_weight = None
        if dy is None:
            d_x = dx = dh
        else:
            g = ops.rms_norm_backward(_incoming(dy), h, weight, rstd, None if dh is None else _incoming(dh),
                                      bf16_dx=x_type == torch.bfloat16, f32_dx=x_type == torch.float32)
            dx, d_weight = g["dx"], g["d_weight"].to(weight.dtype)
            # x's own, in x's type where that is not the stream's
            d_x = g.get("dx_bf16" if x_type == torch.bfloat16 else "dx_f32", dx)
        d_x = d_x.to(x_type)
        return d_x, d_weight, None if res_type is None else dx.to(res_type), None, None


def rms_norm(x, weight, residual=None, eps: float = 1e-6, mxfp8: bool = False):
    """``ops.rms_norm`` under autograd.  Returns (y, h) with h = x + residual
    (x itself without one), the stream to hand on; with ``mxfp8`` (y, h,
    (codes, scales))."""
    y, h, codes, scales = RMSNormFunction.apply(x, weight, residual, eps, mxfp8)
    return (y, h, (codes, scales)) if mxfp8 else (y, h)


class MoKRMSNorm(torch.nn.Module):
    """Root-mean-square norm over the last axis with the residual's addition."""

    def __init__(self, H: int, eps: float = 1e-6, mxfp8: bool = False, dtype=torch.bfloat16, device=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.ones(H, dtype=dtype, device=device))
        self.eps, self.mxfp8 = eps, mxfp8

    def forward(self, x, residual=None):
        return rms_norm(x, self.weight, residual, self.eps, self.mxfp8)


class LinearFunction(torch.autograd.Function):
    """y = act(x W^T + bias) + residual, the pre-activations kept for the
    backward where an activation needs them."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, activation, out_dtype):
        keep = activation != "none" and any(ctx.needs_input_grad[:3])
        y, z = ops.linear(x, weight, bias, activation, residual, out_dtype, save_z=keep)
        ctx.save_for_backward(x, weight, z)
        ctx.linear = (activation, None if bias is None else bias.dtype, None if residual is None else residual.dtype)
        return y

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x, weight, z = ctx.saved_tensors
        activation, bias_type, res_type = ctx.linear
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        g = {}
        if need_x or need_w or need_b:
            need = [n for n, on in (("dx", need_x), ("d_weight", need_w)) if on]
            g = ops.linear_backward(_incoming(dy), x, weight, z, activation, bias=bool(need_b), need=need)
        return (g.get("dx"), g.get("d_weight"), g["d_bias"].to(bias_type) if need_b else None,
                dy.to(res_type) if need_r else None, None, None)


def linear(x, weight, bias=None, activation: str = "none", residual=None, out_dtype=torch.bfloat16):
    """``ops.linear`` under autograd; returns y."""
    return LinearFunction.apply(x, weight, bias, residual, activation, out_dtype)


class MoKLinear(torch.nn.Module):
    """A dense projection K -> N with its epilogue: activation, and a residual
    given at the call."""

    def __init__(self, K: int, N: int, bias: bool = True, activation: str = "none", out_dtype=torch.bfloat16,
                 device=None, init_std: float = 0.02, generator=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty(N, K, dtype=torch.bfloat16, device=device))
        with torch.no_grad():
            self.weight.normal_(0.0, init_std, generator=generator)
        self.bias = torch.nn.Parameter(torch.zeros(N, dtype=torch.float32, device=device)) if bias else None
        self.activation, self.out_dtype = activation, out_dtype

    def forward(self, x, residual=None):
        return linear(x, self.weight, self.bias, self.activation, residual, self.out_dtype)


class RouteFunction(torch.autograd.Function):
    """(experts, weights, lse, counts, mean_score) of router logits; the choice
    and the counts are integers and get no gradient, nor does the bias, which
    decides the choice alone."""

    @staticmethod
    def forward(ctx, logits, bias, k, score, normalize, scale, balance):
        r = experts.route(logits, k, score, normalize, scale, bias, balance)
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(r.experts, *([r.counts] if balance else []))
        ctx.save_for_backward(logits, r.experts)
        ctx.route = (score, normalize, scale)
        return r.experts, r.weights, r.lse, r.counts, r.mean_score

    @staticmethod
    @_first_order
    def backward(ctx, _experts, d_weights, d_lse, _counts, d_mean_score):
        logits, chosen = ctx.saved_tensors
        if d_weights is None and d_lse is None and d_mean_score is None:
            return (None,) * 7
        d_weights = (torch.zeros(chosen.shape, dtype=torch.float32, device=chosen.device) if d_weights is None
                     else _incoming(d_weights))
        d = experts.route_backward(d_weights, logits, chosen, *ctx.route, None if d_lse is None else _incoming(d_lse),
                                   None if d_mean_score is None else _incoming(d_mean_score))
        return d, None, None, None, None, None, None


def route(logits, k: int, score: str = "softmax", normalize: bool = True, scale: float = 1.0, bias=None, balance: bool = False):
    """``experts.route`` under autograd: a ``Routing`` whose weights, lse and
    mean_score are differentiable in the logits."""
    return experts.Routing(*RouteFunction.apply(logits, bias, k, score, normalize, scale, balance))


class MoKRouter(torch.nn.Module):
    """The router: logits in 32 bits by the projection operator (E a multiple of
    8), and the choice.
    Its ``Routing`` feeds ``MoKLayer``, or ``grouped_linear`` by its counts."""

    def __init__(self, H: int, E: int, k: int, score: str = "softmax", normalize: bool = True, scale: float = 1.0,
                 balance: bool = False, device=None, init_std: float = 0.02, generator=None):
        super().__init__()
        self.proj = MoKLinear(H, E, bias=False, out_dtype=torch.float32, device=device, init_std=init_std, generator=generator)
        self.k, self.score, self.normalize, self.scale, self.balance = k, score, normalize, scale, balance

    def forward(self, x, bias=None):
        return route(self.proj(x), self.k, self.score, self.normalize, self.scale, bias, self.balance)


class GroupedLinearFunction(torch.autograd.Function):
    """y = act(x W_e^T + bias_e) for rows sorted by expert, the pre-activations
    kept for the backward where an activation needs them."""

    @staticmethod
    def forward(ctx, x, weight, counts, bias, activation, out_dtype):
        keep = activation != "none" and any(ctx.needs_input_grad)
        y, z = experts.grouped_linear(x, weight, counts, bias, activation, out_dtype, save_z=keep)
        ctx.save_for_backward(x, weight, counts, z)
        ctx.linear = (activation, None if bias is None else bias.dtype)
        return y

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x, weight, counts, z = ctx.saved_tensors
        activation, bias_type = ctx.linear
        need_x, need_w, _, need_b = ctx.needs_input_grad[:4]
        need = [n for n, on in (("dx", need_x), ("d_weight", need_w)) if on]
        g = experts.grouped_linear_backward(_incoming(dy), x, weight, counts, z, activation, bias=bool(need_b), need=need)
        return g.get("dx"), g.get("d_weight"), None, g["d_bias"].to(bias_type) if need_b else None, None, None


def grouped_linear(x, weight, counts, bias=None, activation: str = "none", out_dtype=torch.bfloat16):
    """``experts.grouped_linear`` under autograd; returns y."""
    return GroupedLinearFunction.apply(x, weight, counts, bias, activation, out_dtype)


class MoKGroupedLinear(torch.nn.Module):
    """E projections K -> N, one for each expert's rows."""

    def __init__(self, E: int, K: int, N: int, bias: bool = True, activation: str = "none", out_dtype=torch.bfloat16, device=None,
                 init_std: float = 0.02, generator=None):
        super().__init__()
        self.weight = torch.nn.Parameter(torch.empty(E, N, K, dtype=torch.bfloat16, device=device))
        with torch.no_grad():
            self.weight.normal_(0.0, init_std, generator=generator)
        self.bias = torch.nn.Parameter(torch.zeros(E, N, dtype=torch.float32, device=device)) if bias else None
        self.activation, self.out_dtype = activation, out_dtype

    def forward(self, x, counts):
        return grouped_linear(x, self.weight, counts, self.bias, self.activation, self.out_dtype)
