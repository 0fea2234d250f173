"""The router's autograd face over a restatement of its kernels on the CPU: the
gradients that it makes up where a loss leaves out an output."""
import pytest
import torch

from mixture_experts_layer_mok_gb300 import autograd, experts

F32 = torch.float32


def _outputs(logits, chosen, score, normalize, scale):
    s = torch.softmax(logits, -1) if score == "softmax" else torch.sigmoid(logits)
    w = s.gather(-1, chosen)
    return (w / w.sum(-1, keepdim=True) if normalize else w) * scale, torch.logsumexp(logits, -1), s.mean(0)


def _route(logits, k, score="softmax", normalize=True, scale=1.0, bias=None, balance=False):
    chosen = logits.topk(k, -1).indices
    w, lse, mean = _outputs(logits, chosen, score, normalize, scale)
    counts = torch.bincount(chosen.flatten(), minlength=logits.shape[-1]).to(torch.int32)
    return experts.Routing(chosen, w, lse, counts if balance else None, mean if balance else None)


def _route_backward(d_weights, logits, chosen, score="softmax", normalize=True, scale=1.0, d_lse=None, d_mean_score=None):
    for name, g in (("d_weights", d_weights), ("d_lse", d_lse), ("d_mean_score", d_mean_score)):   # as the library's own face checks
        if (g is None and name == "d_weights") or (g is not None and (g.dtype != F32 or not g.is_contiguous())):
            raise ValueError(f"{name}: expected fp32")
    with torch.enable_grad():
        at = logits.detach().requires_grad_()
        outs = _outputs(at, chosen, score, normalize, scale)
        loss = sum((o * g).sum() for o, g in zip(outs, (d_weights, d_lse, d_mean_score)) if g is not None)
        return torch.autograd.grad(loss, at)[0]


@pytest.mark.parametrize("default", [torch.float32, torch.float64, torch.bfloat16])
@pytest.mark.parametrize("used", [("lse",), ("mean_score",), ("lse", "mean_score"), ("weights",), ("weights", "lse", "mean_score")])
def test_a_loss_of_some_outputs_under_any_default_type(monkeypatch, default, used):
    monkeypatch.setattr(experts, "route", _route)
    monkeypatch.setattr(experts, "route_backward", _route_backward)
    logits = torch.randn(5, 12, generator=torch.Generator().manual_seed(0), dtype=F32)
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        x = logits.clone().requires_grad_()
        r = autograd.route(x, 3, balance=True)
        sum(getattr(r, name).square().sum() for name in used).backward()
    finally:
        torch.set_default_dtype(before)
    y = logits.clone().requires_grad_()
    w, lse, mean = _outputs(y, r.experts, "softmax", True, 1.0)
    outs = dict(weights=w, lse=lse, mean_score=mean)
    sum(outs[name].square().sum() for name in used).backward()
    # the same operations in another order: a dozen roundings of terms of a few units
    assert (x.grad - y.grad).abs().max().item() <= 64 * 2.0 ** -24 * max(1.0, y.grad.abs().max().item())
