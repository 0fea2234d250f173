"""The autograd faces over restatements of the kernels on the CPU: what the
faces themselves do with the gradients they are given and hand on."""
from types import SimpleNamespace

import pytest
import torch

from mixture_experts_layer_mok_gb300 import autograd, ops

F32 = torch.float32


def _norm(x, weight, residual=None, eps=1e-6, mxfp8=False):
    h = x if residual is None else x + residual
    rstd = (h.float().square().mean(-1) + eps).rsqrt()
    return ops.NormOutput((h * rstd[..., None] * weight).to(x.dtype), None, h, rstd)


def _norm_backward(dy, h, weight, rstd, d_h=None, bf16_dx=False, f32_dx=False):
    xhat, g = h * rstd[..., None], dy * weight
    dx = rstd[..., None] * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    return {"dx": dx if d_h is None else dx + d_h, "d_weight": (dy * xhat).sum(0)}


def _linear(x, weight, bias=None, activation="none", residual=None, out_dtype=F32, save_z=False):
    return x @ weight.t() + (0 if bias is None else bias), None


def _linear_backward(dy, x, weight, z=None, activation="none", bias=False, need=()):
    out = {"dx": dy @ weight, "d_weight": dy.t() @ x}
    return {k: v for k, v in out.items() if k in need} | ({"d_bias": dy.sum(0)} if bias else {})


def _layer_forward(x, router_w, sched, weights, **kw):
    y = x * weights.w_gate.sum()
    return y, SimpleNamespace(flatten=lambda: (y, None))


def _layer_backward(dy, x, router_w, sched, ctx, weights, **kw):
    s = weights.w_gate.sum()
    return {"dx": dy * s, "d_router_w": torch.zeros_like(router_w), "d_w_gate": (dy * x).sum() * torch.ones_like(weights.w_gate),
            "d_w_up": torch.zeros_like(weights.w_up), "d_w_down": torch.zeros_like(weights.w_down)}


@pytest.fixture
def restated(monkeypatch):
    monkeypatch.setattr(ops, "rms_norm", _norm)
    monkeypatch.setattr(ops, "rms_norm_backward", _norm_backward)
    monkeypatch.setattr(ops, "linear", _linear)
    monkeypatch.setattr(ops, "linear_backward", _linear_backward)
    monkeypatch.setattr(autograd, "schedule", lambda te, E, c: SimpleNamespace(flatten=lambda: (te, None)))
    monkeypatch.setattr(autograd, "forward", _layer_forward)
    monkeypatch.setattr(autograd, "backward", _layer_backward)
    for name in ("Schedule", "Context"):
        monkeypatch.setattr(autograd, name, SimpleNamespace(unflatten=lambda buf, meta: None))


def _losses():
    g = torch.Generator().manual_seed(0)
    t = lambda *s: torch.randn(*s, generator=g).requires_grad_()  # noqa: E731
    x, w, e = t(4, 8), t(8), [t(2, 3, 8), t(2, 3, 8), t(2, 8, 3)]
    return {"norm": (lambda: autograd.rms_norm(x, w)[0].sum(), x, w),
            "norm, residual": (lambda: autograd.rms_norm(x, w, t(4, 8))[1].sum() + autograd.rms_norm(x, w, x)[0].sum(), x, w),
            "linear": (lambda: autograd.linear(x, e[0][0], e[1][0, :, 0], out_dtype=F32).sum(), x, e[0])}


@pytest.mark.parametrize("which", ["norm", "norm, residual", "linear"])
def test_a_gradients_derivative_is_refused(restated, which):
    """A gradient penalty: its term used to vanish from the weight's gradient
    without a word.  First derivatives under create_graph are as without."""
    loss, x, w = _losses()[which]
    plain = torch.autograd.grad(loss(), [x, w])
    first = torch.autograd.grad(loss(), [x, w], create_graph=True)
    for a, b in zip(plain, first):
        assert torch.equal(a, b) and not a.requires_grad and b.requires_grad
    with pytest.raises(RuntimeError, match="no derivative of their own"):
        (loss() + first[0].square().sum()).backward()


def test_the_layers_gradients_derivative_is_refused(restated):
    x, rw = torch.randn(4, 8, requires_grad=True), torch.ones(4, 1, requires_grad=True)
    w = [torch.randn(*s).requires_grad_() for s in ((2, 3, 8), (2, 3, 8), (2, 8, 3))]
    ids = torch.zeros(4, 1, dtype=torch.int64)
    y = autograd.mok_layer(x, rw, ids, *w)
    first, = torch.autograd.grad(y.float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="MoKFunction.*no derivative of their own"):
        first.float().square().sum().backward()
    y = autograd.mok_layer(x, rw, ids, *w)
    y.float().sum().backward()
    assert x.grad is not None and w[0].grad is not None


def _odd(t):
    """t's values at an address that is not a multiple of 16 bytes."""
    flat = torch.empty(t.numel() + 9, dtype=t.dtype)
    at = next(i for i in range(1, 9) if flat[i:].data_ptr() % 16)
    view = flat[at:at + t.numel()].view(t.shape)
    view.copy_(t)
    assert view.is_contiguous() and view.data_ptr() % 16
    return view


@pytest.mark.parametrize("which", ["norm", "norm's stream", "linear", "layer"])
def test_a_gradient_at_an_odd_address_reaches_the_library_aligned(restated, monkeypatch, which):
    """The library refuses such a tensor, which the middle of a backward is no
    place for."""
    seen = []

    def watch(module, name):
        inner = getattr(module, name)

        def call(*a, **k):
            seen.extend(t for t in (*a, *k.values()) if isinstance(t, torch.Tensor))
            return inner(*a, **k)
        monkeypatch.setattr(module, name, call)

    for module, name in ((ops, "rms_norm_backward"), (ops, "linear_backward"), (autograd, "backward")):
        watch(module, name)
    g = torch.Generator().manual_seed(0)
    t = lambda *s: torch.randn(*s, generator=g).requires_grad_()  # noqa: E731
    x, w, e = t(4, 8), t(8), [t(2, 3, 8), t(2, 3, 8), t(2, 8, 3)]
    if which == "layer":
        y = autograd.mok_layer(x.bfloat16(), torch.ones(4, 1, requires_grad=True), torch.zeros(4, 1, dtype=torch.int64),
                               *(v.bfloat16() for v in e))
    elif which == "linear":
        y = autograd.linear(x, e[0][0], out_dtype=F32)
    else:
        y, h = autograd.rms_norm(x, w, t(4, 8))
        y = y if which == "norm" else y.sum() + h
    dy = torch.randn(y.shape, generator=g).to(y.dtype)
    y.backward(_odd(dy))
    assert seen and all(v.data_ptr() % 16 == 0 for v in seen)
