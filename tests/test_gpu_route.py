"""The router and its gradient against 64-bit restatements.

Error bounds, from the arithmetic, in units of u = 2^-24: an exponential's
argument x - top is rounded (its size, up to `span`, times u) and the function
itself is good to 2 ulp (4 u); a sum over E is a chain of at most E / 32 + 5
additions; a handful of further operations.  So each score, weight and gradient
term is good to (2 span + E / 32 + 32) u of its size, a sigmoid, whose argument
is not rounded, to less."""
import pytest
import torch

from tests.gpu_util import mok

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24


def _rel(x):
    finite = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).double()
    span = (finite.max() - finite.min()).item() if x.numel() else 0.0
    return (2 * span + x.shape[-1] / 32 + 32) * U


def _scores(l64, score):
    return torch.softmax(l64, -1) if score == "softmax" else torch.sigmoid(l64)


def _logits(T, E, dtype, seed=0, std=2.0):
    g = torch.Generator().manual_seed(seed + 31 * T + 7 * E)
    return (torch.randn(T, E, generator=g) * std).to(dtype).cuda()


def _close(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), what
    assert (err <= bound).all(), (what, (err - bound).max().item())


SHAPES = [(1, 1, 1), (1, 4, 2), (3, 5, 5), (7, 31, 3), (64, 32, 32), (9, 33, 8), (257, 64, 8), (100, 100, 12), (5, 127, 7),
          (33, 129, 64), (1, 256, 8), (4099, 256, 8), (12, 257, 1), (18, 384, 6), (70, 512, 9), (11, 1000, 10), (6, 1024, 64),
          (20000, 8, 2)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score,normalize,scale", [("softmax", True, 1.0), ("softmax", False, 1.0), ("sigmoid", True, 2.5),
                                                   ("sigmoid", False, 1.0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward(T, E, k, score, normalize, scale, dtype):
    m = mok()
    x = _logits(T, E, dtype)
    r = m.route(x, k, score=score, normalize=normalize, scale=scale, balance=True)
    l64 = x.double()
    experts = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(r.experts, experts)
    s = _scores(l64, score)
    w = s.gather(1, experts)
    w = w / w.sum(1, keepdim=True) * scale if normalize else w * scale
    rel = _rel(x)
    _close(r.weights, w, rel * w, "weights")
    lse = torch.logsumexp(l64, 1)
    _close(r.lse, lse, rel + 4 * U * lse.abs(), "lse")
    assert torch.equal(r.counts.long(), torch.bincount(experts.reshape(-1), minlength=E))
    # a warp's tokens one after the other, then 8 warps and up to 608 blocks in steps of 32
    _close(r.mean_score, s.mean(0), (rel + (T / 64 + 64) * U) * s.mean(0), "mean")
    plain = m.route(x, k, score=score, normalize=normalize, scale=scale)
    assert plain.counts is None and plain.mean_score is None
    assert torch.equal(plain.experts, r.experts) and torch.equal(plain.weights, r.weights) and torch.equal(plain.lse, r.lse)
    again = m.route(x, k, score=score, normalize=normalize, scale=scale, balance=True)
    assert torch.equal(again.mean_score, r.mean_score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_bias_decides_the_choice_alone(score):
    m = mok()
    T, E, k = 500, 96, 6
    x = _logits(T, E, F32)
    x[3, 5:] = -float("inf")     # fewer open experts than k: the rest by index, whatever their bias
    bias = (torch.randn(E, generator=torch.Generator().manual_seed(1)) * 0.3).cuda()
    r = m.route(x, k, score=score, bias=bias, balance=True)
    s = _scores(x.double(), score)
    by = torch.where(torch.isinf(x), torch.full_like(s, -float("inf")), s + bias.double())
    top = by.topk(k, 1).values
    got = by.gather(1, r.experts)
    got[3, 5:], top[3, 5:] = 0.0, 0.0
    # neighbours closer than the scores' error may change places
    _close(got, top, 2 * _rel(x) + 4 * U, "choice")
    assert r.experts[3, 5].item() == 5
    w = s.gather(1, r.experts)
    w = w / w.sum(1, keepdim=True)
    _close(r.weights, w, _rel(x) * w, "weights")
    assert torch.equal(r.counts.long(), torch.bincount(r.experts.reshape(-1), minlength=E))


def test_ties_go_to_the_lowest_index():
    m = mok()
    for E in (8, 64, 200, 256, 777, 1024):
        x = torch.randint(0, 3, (300, E), generator=torch.Generator().manual_seed(E)).float().cuda()
        x[0] = 0.0
        x[1, ::2] = -0.0                      # equal to 0
        x[1, 1::2] = 0.0
        ref = torch.sort(x, dim=1, descending=True, stable=True).indices
        for dtype in (F32, BF16):
            assert torch.equal(m.route(x.to(dtype), 8).experts, ref[:, :8])


def test_masked_and_extreme_logits():
    m = mok()
    inf = float("inf")
    low = torch.finfo(F32).min
    x = torch.full((6, 40), -inf, device="cuda")
    x[0, 7] = 2.0                             # one open expert, fewer than k
    x[1] = -inf                               # none
    x[2] = low                                # all at the lowest value
    x[3] = low
    x[3, 11] = 50.0
    x[4] = torch.linspace(-200, 200, 40)
    x[5] = 3.0e38
    r = m.route(x, 3, balance=True)
    assert r.experts.tolist()[0] == [7, 0, 1] and r.weights[0].tolist() == [1.0, 0.0, 0.0] and r.lse[0].item() == 2.0
    assert r.experts.tolist()[1] == [0, 1, 2] and r.weights[1].tolist() == [0.0] * 3 and r.lse[1].item() == -inf
    for row, first in ((2, [0, 1, 2]), (5, [0, 1, 2])):
        assert r.experts.tolist()[row] == first
        assert torch.allclose(r.weights[row], torch.full((3,), 1 / 3, device="cuda"), rtol=4 * U, atol=0)
    assert r.experts[3, 0].item() == 11 and r.weights[3].tolist() == [1.0, 0.0, 0.0]
    assert r.experts.tolist()[4] == [39, 38, 37] and torch.isfinite(r.weights).all()
    d = m.route_backward(torch.randn(6, 3, device="cuda"), x, r.experts, d_lse=torch.ones(6, device="cuda"),
                         d_mean_score=torch.ones(40, device="cuda"))
    assert torch.isfinite(d).all() and (d[1] == 0).all() and (d[0, :7] == 0).all()
    # scores that underflow among the others, renormalised among the chosen: by the 64-bit definition
    y = torch.full((2, 40), 120.0, device="cuda")
    y[:, :4] = torch.tensor([1.0, 0.5, 0.0, -1.0], device="cuda")
    chosen = torch.tensor([[0, 1, 2, 3], [3, 2, 1, 0]], device="cuda")
    dw = torch.randn(2, 4, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    d = m.route_backward(dw, y, chosen)
    u = torch.softmax(y.double().gather(1, chosen), 1)
    ref = torch.zeros_like(y, dtype=F64).scatter_(1, chosen, u * (dw - (u * dw).sum(1, keepdim=True)))
    _close(d, ref, 64 * U * torch.ones_like(ref), "underflow")


def test_nan_and_inf_rows_leave_the_others_alone():
    m = mok()
    x = _logits(40, 64, F32)
    clean = m.route(x, 4)
    bad = x.clone()
    bad[5, 9], bad[17, 3] = float("nan"), float("inf")
    r = m.route(bad, 4)
    keep = [i for i in range(40) if i not in (5, 17)]
    for name in ("experts", "weights", "lse"):
        assert torch.equal(getattr(r, name)[keep], getattr(clean, name)[keep])
    assert r.experts[5, 0].item() == 9 and torch.isnan(r.lse[5]) and torch.isnan(r.weights[5]).any()
    assert r.experts[17, 0].item() == 3 and r.lse[17].item() == float("inf")


def test_no_tokens_and_leading_axes():
    m = mok()
    x = torch.empty(0, 16, device="cuda")
    r = m.route(x, 4, balance=True)
    assert r.experts.shape == (0, 4) and r.counts.tolist() == [0] * 16 and r.mean_score.tolist() == [0.0] * 16
    assert m.route_backward(torch.empty(0, 4, device="cuda"), x, r.experts).shape == (0, 16)
    y = _logits(12, 16, BF16)
    a, b = m.route(y, 3), m.route(y.view(3, 4, 16), 3)
    assert b.experts.shape == (3, 4, 3) and b.lse.shape == (3, 4) and torch.equal(a.weights, b.weights.view(12, 3))
    c = m.route(y[2].clone(), 3, balance=True)
    assert c.experts.shape == (3,) and c.lse.shape == () and torch.equal(c.weights, a.weights[2]) and c.counts.sum().item() == 3
    assert torch.equal(m.route_backward(c.weights, y[2].clone(), c.experts), m.route_backward(a.weights, y, a.experts)[2])


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score,normalize,losses", [("softmax", True, False), ("softmax", False, True), ("softmax", True, True),
                                                    ("sigmoid", True, True), ("sigmoid", False, False)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward(T, E, k, score, normalize, losses, dtype):
    m = mok()
    x = _logits(T, E, dtype, seed=1)
    g = torch.Generator("cuda").manual_seed(T + E)
    experts = m.route(x, k).experts
    dw = torch.randn(T, k, device="cuda", generator=g)
    d_lse = torch.randn(T, device="cuda", generator=g) if losses else None
    d_mean = torch.randn(E, device="cuda", generator=g) if losses else None
    d = m.route_backward(dw, x, experts, score=score, normalize=normalize, scale=1.5, d_lse=d_lse, d_mean_score=d_mean)
    assert d.dtype == dtype
    l64 = x.double().requires_grad_(True)
    s = _scores(l64, score)
    w = s.gather(1, experts)
    w = (w / w.sum(1, keepdim=True) if normalize else w) * 1.5
    loss = (w * dw.double()).sum()
    if losses:
        loss = loss + (torch.logsumexp(l64, 1) * d_lse.double()).sum() + (s.mean(0) * d_mean.double()).sum()
    ref, = torch.autograd.grad(loss, l64)
    # the terms' sizes: differences of them carry their errors
    size = 1.5 * dw.abs().max().item() * 2 * torch.zeros_like(ref).scatter_(1, experts, w.detach() / 1.5)
    p = torch.softmax(x.double(), 1)
    if score == "softmax":
        size = size + p * 1.5 * 2 * dw.abs().max().item()
    if losses:
        size = size + p * d_lse.double().abs()[:, None] + s.detach() * 2 * d_mean.abs().max().item() / T
    bound = 4 * _rel(x) * size + 1e-30
    if dtype == BF16:
        bound = bound + 2.0 ** -8 * ref.abs()
    _close(d, ref, bound, "d_logits")


def test_gradient_against_differences():
    m = mok()
    from mixture_experts_layer_mok_gb300.autograd import route

    for score, normalize in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        x = _logits(5, 24, F32, seed=3, std=1.0).requires_grad_(True)
        r = route(x, 4, score=score, normalize=normalize, balance=True)
        cw, cl, cm = (torch.randn(s, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
                      for s in (r.weights.shape, r.lse.shape, r.mean_score.shape))
        ((r.weights * cw).sum() + (r.lse * cl).sum() + (r.mean_score * cm).sum()).backward()

        def f(l64):
            s = _scores(l64, score)
            w = s.gather(1, r.experts)
            w = w / w.sum(1, keepdim=True) if normalize else w
            return (w * cw).sum() + (torch.logsumexp(l64, 1) * cl).sum() + (s.mean(0) * cm).sum()

        h, base = 1e-5, x.detach().double()
        num = torch.zeros_like(base)
        for i in range(5):
            for j in range(24):
                e = torch.zeros_like(base)
                e[i, j] = h
                num[i, j] = (f(base + e) - f(base - e)) / (2 * h)
        # differences: h^2 of a third derivative of order 10; the kernel: 1e-5 of terms of order 3
        assert (x.grad.double() - num).abs().max().item() <= 5e-5
    assert m is not None


def test_backward_ignores_ids_outside_and_sums_repeated_ones():
    m = mok()
    x = _logits(4, 16, F32)
    dw = torch.ones(4, 3, device="cuda")
    ids = torch.tensor([[1, -1, 99], [2, 2, 3], [-5, 16, 1 << 40], [0, 1, 2]], device="cuda")
    d = m.route_backward(dw, x, ids, score="sigmoid", normalize=False)
    s = torch.sigmoid(x.double())
    ref = torch.zeros_like(s)
    for t, row in enumerate(ids.tolist()):
        for e in row:
            if 0 <= e < 16:
                ref[t, e] += s[t, e] * (1 - s[t, e])
    _close(d, ref, 64 * U * ref, "ids")


def test_refusals():
    m = mok()
    x = _logits(8, 16, F32)
    r = m.route(x, 2)
    for call in (lambda: m.route(x, 0), lambda: m.route(x, 17), lambda: m.route(x, 2, score="top"), lambda: m.route(x.half(), 2),
                 lambda: m.route(x[:, ::2], 2), lambda: m.route(x, 2, bias=torch.zeros(8, device="cuda")),
                 lambda: m.route(x, 2, bias=torch.zeros(16, device="cuda", dtype=BF16)), lambda: m.route(x.new_zeros(2, 1025), 2),
                 lambda: m.route(x.new_zeros(2, 100), 65), lambda: m.route_backward(r.weights[:, :1].contiguous(), x, r.experts),
                 lambda: m.route_backward(r.weights.double(), x, r.experts), lambda: m.route_backward(r.weights, x, r.experts.int()),
                 lambda: m.route_backward(r.weights, x, r.experts, d_lse=torch.zeros(7, device="cuda")),
                 lambda: m.route_backward(r.weights, x, r.experts, d_mean_score=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for scale in (float("nan"), float("inf")):
        with pytest.raises(m.MokError):
            m.route(x, 2, scale=scale)
    with pytest.raises(m.MokError):                     # a view that begins between 16 bytes
        m.route(torch.zeros(8 * 16 + 1, device="cuda")[1:].view(8, 16), 2)


def test_streams_and_graph():
    m = mok()
    x = _logits(513, 128, F32)
    ref = m.route(x, 8, balance=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = m.route(x, 8, balance=True, stream=side)
    side.synchronize()
    assert torch.equal(r.weights, ref.weights) and torch.equal(r.mean_score, ref.mean_score)
    buf = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.route(buf, 8, balance=True)
        d = m.route_backward(out.weights, buf, out.experts)
    for seed in (5, 6):
        new = _logits(513, 128, F32, seed=seed)
        buf.copy_(new)
        graph.replay()
        want = m.route(new, 8, balance=True)
        assert torch.equal(out.experts, want.experts) and torch.equal(out.counts, want.counts)
        assert torch.equal(out.mean_score, want.mean_score)
        assert torch.equal(d, m.route_backward(want.weights, new, want.experts))


def test_many_tokens_of_many_experts():
    """Logits beyond 2^31 elements: the last rows are where 32-bit offsets would not reach."""
    m = mok()
    T, E = (1 << 21) + 77, 1024
    x = torch.zeros(T, E, dtype=BF16, device="cuda")
    x[:, 5] = 1.0
    x[-3:] = _logits(3, E, BF16)
    r = m.route(x, 4)
    ref = m.route(x[-3:].clone(), 4)
    assert torch.equal(r.experts[-3:], ref.experts) and torch.equal(r.weights[-3:], ref.weights)
    assert (r.experts[:-3, 0] == 5).all() and (r.experts[:-3, 1] == 0).all()
    d = m.route_backward(r.weights, x, r.experts)
    assert torch.equal(d[-3:], m.route_backward(ref.weights, x[-3:].clone(), ref.experts))
