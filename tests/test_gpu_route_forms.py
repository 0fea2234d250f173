"""The router in every way that tokens are dealt to warps: one token or several to
a round, blocks of 1, 4, 8 and 16 warps, more picks than lanes, with loads and
with a bias; bounds as derived in ``test_gpu_route``.

Mean scores: a warp adds its tokens one after the other.  A round is 1, 4 or 8
tokens and there are 608 warps at least where there are as many rounds, so that a
warp has T / 608 + 8 tokens at most.  Then up to 3 shuffles, 4 warps' rows in
each of up to 4 places, 608 blocks in steps of 64, 2 shuffles and 16 warps'
sums: 48 additions."""
import pytest
import torch

from tests.gpu_util import mok
from tests.test_gpu_route import U, _close, _logits, _rel, _scores

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64

FORMS = [(40000, 20, 9), (5000, 32, 32), (5000, 40, 12), (5000, 64, 33), (2433, 65, 9), (3000, 100, 12), (3000, 128, 64), (3000, 256, 20),
         (20000, 256, 40), (2500, 384, 40), (9800, 300, 5), (10001, 512, 9), (2432, 512, 33), (10001, 1000, 33), (20001, 1024, 8)]


def _outputs(r, x, experts, score, scale):
    """Against the definition, for the experts that were chosen."""
    T, E = x.shape
    s = _scores(x.double(), score)
    w = s.gather(1, experts)
    w = w / w.sum(1, keepdim=True) * scale
    rel = _rel(x)
    _close(r.weights, w, rel * w, "weights")
    lse = torch.logsumexp(x.double(), 1)
    _close(r.lse, lse, rel + 4 * U * lse.abs(), "lse")
    assert torch.equal(r.counts.long(), torch.bincount(experts.reshape(-1), minlength=E))
    _close(r.mean_score, s.mean(0), (rel + (T / 608 + 8 + 48) * U) * s.mean(0), "mean")


@pytest.mark.parametrize("T,E,k", FORMS)
@pytest.mark.parametrize("score,scale", [("softmax", 1.0), ("sigmoid", 2.5)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward(T, E, k, score, scale, dtype):
    m = mok()
    x = _logits(T, E, dtype, seed=5)
    r = m.route(x, k, score=score, scale=scale, balance=True)
    experts = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.experts, experts)
    _outputs(r, x, experts, score, scale)
    plain = m.route(x, k, score=score, scale=scale)
    assert torch.equal(plain.experts, r.experts) and torch.equal(plain.weights, r.weights) and torch.equal(plain.lse, r.lse)


@pytest.mark.parametrize("E,k", [(8, 3), (40, 5), (40, 12), (96, 6), (96, 40), (200, 8), (200, 20), (384, 10), (384, 33), (1000, 12)])
@pytest.mark.parametrize("T", [1, 600, 3000, 11000])
@pytest.mark.parametrize("score,dtype", [("softmax", F32), ("sigmoid", F32), ("sigmoid", BF16)])
def test_bias(E, k, T, score, dtype):
    m = mok()
    x = _logits(T, E, dtype, seed=6)
    g = torch.Generator("cuda").manual_seed(E)
    bias = torch.randn(E, device="cuda", generator=g) * (0.3 if score == "sigmoid" else 2.0 / E)
    r = m.route(x, k, score=score, scale=2.5, bias=bias, balance=True)
    assert (r.experts.sort(1).values.diff(dim=1) > 0).all()
    by = _scores(x.double(), score) + bias.double()
    # the score's error and the sum's rounding, of the expert chosen and of the one left
    _close(by.gather(1, r.experts), by.topk(k).values, 2 * (_rel(x) + U) * (by.abs() + bias.double().abs()).amax(1, keepdim=True), "choice")
    _outputs(r, x, r.experts, score, 2.5)
    again = m.route(x, k, score=score, scale=2.5, bias=bias)
    assert torch.equal(again.experts, r.experts) and torch.equal(again.weights, r.weights) and torch.equal(again.lse, r.lse)


@pytest.mark.parametrize("T,E,k", [(5000, 40, 12), (3000, 128, 64), (20000, 256, 40), (10001, 512, 9), (9000, 1000, 33)])
@pytest.mark.parametrize("score,normalize", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_backward(T, E, k, score, normalize):
    m = mok()
    x = _logits(T, E, F32, seed=7)
    g = torch.Generator("cuda").manual_seed(T)
    experts = m.route(x, k).experts
    dw, d_lse, d_mean = (torch.randn(s, device="cuda", generator=g) for s in ((T, k), (T,), (E,)))
    d = m.route_backward(dw, x, experts, score=score, normalize=normalize, d_lse=d_lse, d_mean_score=d_mean)
    l64 = x.double().requires_grad_(True)
    s = _scores(l64, score)
    w = s.gather(1, experts)
    w = w / w.sum(1, keepdim=True) if normalize else w
    ref, = torch.autograd.grad((w * dw.double()).sum() + (torch.logsumexp(l64, 1) * d_lse.double()).sum()
                               + (s.mean(0) * d_mean.double()).sum(), l64)
    most, p = dw.abs().max().item(), torch.softmax(x.double(), 1)
    size = 2 * most * torch.zeros_like(ref).scatter_(1, experts, w.detach())
    if score == "softmax":
        size = size + 2 * most * p
    size = size + p * d_lse.double().abs()[:, None] + s.detach() * 2 * d_mean.abs().max().item() / T
    _close(d, ref, 4 * _rel(x) * size + 1e-30, "d_logits")
