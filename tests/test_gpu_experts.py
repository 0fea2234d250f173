"""Routed experts from their parts, as a model uses them: the router, two
projections grouped by expert and the weighted sum, forward and backward under
autograd; and a token's decoding through the same experts in 4 bits.

Tolerances, relative L2: every rounding to bf16 is at random within 2^-9, 1.7e-3
in norm.  Up to five of them in turn (h, dz, dh, and the result's own) stay below
6e-3; the router's gradient is made of differences of such sums: five times that."""
import pytest
import torch

from tests.gpu_util import mok, rel_l2
from tests.test_gpu_linear import act64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _experts(x, r, up, down, k):
    """The experts' weighted sum for tokens x, rows sorted by expert."""
    order = r.experts.flatten().argsort(stable=True)
    rows = down(up(x[order // k], r.counts), r.counts) * r.weights.flatten()[order, None]
    return torch.zeros_like(rows).index_copy(0, order, rows).view(x.shape[0], k, -1).sum(1)


def _losses(r, T, E):
    """A balance loss and a z loss, weighed to matter."""
    return 0.5 * E * (r.counts.to(r.mean_score.dtype) / T * r.mean_score).sum() + 0.1 * r.lse.square().mean()


@pytest.mark.parametrize("T,H,I,E,k,score", [(1, 64, 72, 4, 2, "softmax"), (300, 136, 264, 12, 3, "sigmoid"),
                                             (2000, 256, 512, 64, 8, "softmax")])
def test_training(T, H, I, E, k, score):
    mok()
    from mixture_experts_layer_mok_gb300.autograd import MoKGroupedLinear, MoKRouter

    g = torch.Generator("cuda").manual_seed(T)
    router = MoKRouter(H, 8 * ((E + 7) // 8), k, score=score, balance=True, device="cuda", generator=g, init_std=H ** -0.5)
    E = 8 * ((E + 7) // 8)
    up = MoKGroupedLinear(E, H, I, activation="gelu", device="cuda", generator=g, init_std=H ** -0.5)
    down = MoKGroupedLinear(E, I, H, out_dtype=F32, device="cuda", generator=g, init_std=I ** -0.5)
    with torch.no_grad():
        up.bias.normal_(generator=g)
        down.bias.normal_(generator=g)
    x = torch.randn(T, H, generator=g, device="cuda").to(BF16).requires_grad_(True)
    cot = torch.randn(T, H, generator=g, device="cuda")
    r = router(x)
    y = _experts(x, r, up, down, k)
    params = [x, router.proj.weight, up.weight, up.bias, down.weight, down.bias]
    grads = torch.autograd.grad((y * cot).sum() + T * _losses(r, T, E), params)

    d = [p.detach().double().requires_grad_(True) for p in params]
    logits = d[0] @ d[1].t()
    s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    w = s.gather(1, r.experts)
    w = w / w.sum(1, keepdim=True)
    y64 = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(r.experts == e, as_tuple=True)
        o = act64(d[0][t] @ d[2][e].t() + d[3][e], "gelu") @ d[4][e].t() + d[5][e]
        y64 = y64.index_add(0, t, o * w[t, j, None])
    assert rel_l2(y, y64) <= 6e-3
    losses = 0.5 * E * (r.counts.double() / T * s.mean(0)).sum() + 0.1 * torch.logsumexp(logits, 1).square().mean()
    ref = torch.autograd.grad((y64 * cot.double()).sum() + T * losses, d)
    for name, a, b in zip(("x", "router", "w1", "b1", "w2", "b2"), grads, ref):
        assert rel_l2(a, b) <= (3e-2 if name in ("x", "router") else 6e-3), name
    assert mok().linear_status() == 0


@pytest.mark.parametrize("T,H,I,E,k,group,zeros", [(1, 256, 384, 16, 4, 64, False), (5, 512, 256, 8, 2, 128, True), (1, 2048, 1024, 64, 8, 32, True)])
def test_decoding_in_4_bits(T, H, I, E, k, group, zeros):
    m = mok()
    g = torch.Generator("cuda").manual_seed(T + H)
    rand = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    w1 = m.int4_quantize(rand(E, I, H, std=H ** -0.5), group, zeros)
    w2 = m.int4_quantize(rand(E, H, I, std=I ** -0.5), group, zeros)
    b1 = rand(E, I)
    router = rand(E, H, std=H ** -0.5).to(BF16)
    xs, y = rand(T, H).to(BF16), None

    def step(x):
        logits, _ = m.linear(x, router, out_dtype=F32)
        r = m.route(logits, k)
        h = m.int4_linear(x, w1, bias=b1, activation="silu", experts=r.experts)
        o = m.int4_linear(h, w2, experts=r.experts, out_dtype=F32)
        return r, (o * r.weights[..., None]).sum(-2)

    r, y = step(xs)
    v1, v2 = m.int4_dequantize(w1).double(), m.int4_dequantize(w2).double()
    w = torch.softmax((xs.double() @ router.double().t()), 1).gather(1, r.experts)
    w = w / w.sum(1, keepdim=True)
    ref = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j, e in enumerate(r.experts[t].tolist()):
            ref[t] += w[t, j] * (v2[e] @ act64(v1[e] @ xs[t].double() + b1[e].double(), "silu"))
    assert rel_l2(y, ref) <= 6e-3       # (the dequantised values' own rounding is one of the five)
    # the same step captured and replayed on other tokens
    buf = xs.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, out = step(buf)
    for _ in range(3):
        buf.copy_(rand(T, H).to(BF16))
        graph.replay()
        assert torch.equal(out, step(buf)[1])
    # many tokens take the dequantised weights through the grouped products
    many = rand(64, H).to(BF16)
    r, y = step(many)
    order = r.experts.flatten().argsort(stable=True)
    counts = torch.bincount(r.experts.flatten(), minlength=E).to(torch.int32)
    h, _ = m.grouped_linear(many[order // k], m.int4_dequantize(w1), counts, bias=b1, activation="silu")
    o, _ = m.grouped_linear(h, m.int4_dequantize(w2), counts, out_dtype=F32)
    rows = torch.empty_like(o).index_copy_(0, order, o).view(64, k, H)
    assert rel_l2((rows * r.weights[..., None]).sum(1), y) <= 6e-3


def test_refuses_second_derivatives():
    mok()
    from mixture_experts_layer_mok_gb300.autograd import grouped_linear, route

    x = torch.randn(6, 16, device="cuda", requires_grad=True)
    g, = torch.autograd.grad(route(x, 2).weights.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    r = torch.randn(6, 16, device="cuda").to(BF16).requires_grad_(True)
    w = torch.randn(2, 8, 16, device="cuda").to(BF16).requires_grad_(True)
    y = grouped_linear(r, w, torch.tensor([2, 3], dtype=torch.int32, device="cuda"))
    g, = torch.autograd.grad(y.float().square().sum(), w, create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()


def test_dispatch_modes_see_the_outputs():
    m = mok()
    from torch.utils._python_dispatch import TorchDispatchMode

    class Count(TorchDispatchMode):
        made = 0

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if "empty" in str(func):
                Count.made += out.numel() * out.element_size()
            return out

    x = torch.randn(64, 32, device="cuda")
    plain = m.route(x, 4)
    with Count():
        r = m.route(x, 4)
    assert Count.made == 64 * 4 * (8 + 4) + 64 * 4
    assert torch.equal(r.experts, plain.experts) and torch.equal(r.weights, plain.weights) and torch.equal(r.lse, plain.lse)
