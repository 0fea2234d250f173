"""The operators together: their autograd faces against a plain fp32 model on
the same weights, the layer on codes that came quantised, and the training
example."""
import os
import sys

import pytest
import torch

from mixture_experts_layer_mok_gb300 import inputs as gen
from tests.gpu_util import BF16_TOL, mok, oracle_fwd_bwd, rel_l2, weights_of

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("xt,rt", [(BF16, None), (BF16, BF16), (BF16, F32), (F32, None), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("use", ["both", "y", "h"])
def test_norm_gradients_match_autograd_in_64_bits(xt, rt, use):
    """bf16 roundings of y's gradient path: 2^-8 per value, a few 1e-3 in norm."""
    mok()
    from mixture_experts_layer_mok_gb300.autograd import rms_norm

    g = torch.Generator().manual_seed(1)
    x = torch.randn(37, 96, generator=g).to(xt)
    r = None if rt is None else torch.randn(37, 96, generator=g).to(rt)
    w = (1 + 0.2 * torch.randn(96, generator=g)).to(BF16)
    cy, ch = torch.randn(37, 96, generator=g).to(BF16), torch.randn(37, 96, generator=g).to(BF16)
    dev = [None if t is None else t.cuda().requires_grad_(True) for t in (x, r, w)]
    y, h = rms_norm(dev[0], dev[2], dev[1], eps=1e-5)
    ref = [None if t is None else t.double().requires_grad_(True) for t in (x, r, w)]
    h64 = ref[0] + (0.0 if r is None else ref[1])
    y64 = h64 / (h64.square().mean(-1, keepdim=True) + 1e-5).sqrt() * ref[2]
    loss = loss64 = 0.0
    if use in ("both", "y"):
        loss, loss64 = loss + (y.float() * cy.cuda().float()).sum(), loss64 + (y64 * cy.double()).sum()
    if use in ("both", "h"):
        loss, loss64 = loss + (h.float() * ch.cuda().float()).sum(), loss64 + (h64 * ch.double()).sum()
    loss.backward()
    loss64.backward()
    for got, want in zip(dev, ref):
        if got is None or want.grad is None:
            continue
        assert got.grad.dtype == got.dtype and rel_l2(got.grad, want.grad) < 6e-3


@pytest.mark.parametrize("act,out", [("none", BF16), ("gelu", BF16), ("silu", F32)])
def test_linear_gradients_match_autograd_in_64_bits(act, out):
    mok()
    from mixture_experts_layer_mok_gb300.autograd import linear
    from tests.test_gpu_linear import act64

    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(3, 50, 136, generator=g).to(BF16), (0.1 * torch.randn(72, 136, generator=g)).to(BF16)
    b, r = torch.randn(72, generator=g).to(BF16), torch.randn(3, 50, 72, generator=g).to(BF16)
    c = torch.randn(3, 50, 72, generator=g)
    dev = [t.cuda().requires_grad_(True) for t in (x, w, b, r)]
    y = linear(*dev[:3], activation=act, residual=dev[3], out_dtype=out)
    (y.float() * c.cuda()).sum().backward()
    ref = [t.double().requires_grad_(True) for t in (x, w, b, r)]
    y64 = act64(ref[0] @ ref[1].t() + ref[2], act) + ref[3]
    (y64 * c.double()).sum().backward()
    assert y.dtype == out and rel_l2(y, y64) < 4e-3
    for got, want in zip(dev, ref):   # dy, z, dz and the gradients are each rounded to bf16
        assert got.grad.dtype == BF16 and rel_l2(got.grad, want.grad) < 1e-2
    x2 = x.cuda()                     # no gradient asked for x: none computed, none kept
    y = linear(x2, dev[1], activation=act)
    y.float().sum().backward()
    assert x2.grad is None


@pytest.mark.parametrize("mode", ["mxfp8", "mxfp8_full"])
@pytest.mark.parametrize("shape", [(200, 256, 384, 5, 3, 256), (333, 128, 128, 16, 4, 0)])
@pytest.mark.parametrize("ring", [0, 128])
def test_layer_on_codes_equals_the_layer_that_quantises(mode, shape, ring):
    """The codes of mxfp8_quantize(x) handed in give every bit of the forward
    and of the backward that quantising inside gives."""
    m = mok()
    T, H, I, E, k, I_s = shape
    inp = gen.make_layer_inputs(T, H, I, E, k, I_s, seed=3)
    g = inp.to("cuda")
    sched = m.schedule(g.top_experts, E, 0.5)
    need = int(sched.arrays()["cnt"].max())
    ring = ring and (need + 127) // 128 * 128
    w = weights_of(g, mode)
    y0, c0 = m.forward(g.x, g.router_w, sched, w, mode=mode, macrobatch=ring)
    g0 = m.backward(g.dy, g.x, g.router_w, sched, c0, w, macrobatch=ring)
    y1, c1 = m.forward(g.x, g.router_w, sched, w, mode=mode, macrobatch=ring, x_mx=m.mxfp8_quantize(g.x))
    g1 = m.backward(g.dy, g.x, g.router_w, sched, c1, w, macrobatch=ring)
    assert c0.status() == 0 and c1.status() == 0
    assert torch.equal(y0, y1) and all(torch.equal(g0[n], g1[n]) for n in g0)


def test_layer_on_the_norms_codes():
    """The oracle on the values that the norm's codes stand for (which quantise
    to themselves): the layer's usual bound."""
    m = mok()
    T, H, I, E, k, I_s = 200, 256, 384, 5, 3, 256
    inp = gen.make_layer_inputs(T, H, I, E, k, I_s, seed=5)
    n = m.rms_norm(inp.x.cuda(), torch.ones(H, dtype=BF16, device="cuda"), mxfp8=True)
    g = inp.to("cuda")
    sched = m.schedule(g.top_experts, E, 0.5)
    y, ctx = m.forward(n.y, g.router_w, sched, weights_of(g, "mxfp8"), mode="mxfp8", x_mx=n.mx)
    assert ctx.status() == 0
    inp.x = m.mxfp8_dequantize(*n.mx).cpu()
    assert rel_l2(y, oracle_fwd_bwd(inp, "mxfp8")[0]) <= BF16_TOL
    with pytest.raises(ValueError):
        m.forward(g.x, g.router_w, sched, weights_of(g), x_mx=n.mx)
    with pytest.raises(ValueError):
        m.forward(g.x, g.router_w, sched, weights_of(g, "mxfp8"), mode="mxfp8", x_mx=(n.mx[0][:4], n.mx[1]))


@pytest.mark.parametrize("mode,state", [("bf16", "fp32"), ("mxfp8", "mxfp8"), ("mxfp8_full", "fp32")])
def test_training_example_learns_and_repeats(mode, state):
    mok()
    import train_block

    losses = train_block.train(steps=25, T=256, H=128, I=128, E=8, k=2, I_s=128, mode=mode, state=state, seed=1)
    assert all(v == v for v in losses)
    assert sum(losses[-3:]) / 3 < 0.8 * sum(losses[:3]) / 3, losses
    assert mok().linear_status() == 0


def test_eight_bit_states_train_like_32_bit_ones():
    """The same run with either kind of state ends at about the same loss."""
    mok()
    import train_block

    kw = dict(steps=40, T=256, H=128, I=128, E=8, k=2, I_s=0, seed=2)
    a, b = train_block.train(state="fp32", **kw), train_block.train(state="mxfp8", **kw)
    end_a, end_b = sum(a[-5:]) / 5, sum(b[-5:]) / 5
    assert abs(end_a - end_b) < 0.15 * sum(a[:3]) / 3, (end_a, end_b)


def test_calls_in_a_cuda_graph():
    """A captured sequence (norm, a token's and a batch's projections, their
    gradients, a step) replays with new inputs in the same buffers."""
    m = mok()
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    x, r, wn, w1, w2 = rand(300, 512), rand(300, 512), rand(512), rand(1024, 512), rand(64, 1024)
    p = torch.randn(1000, generator=g, device="cuda")
    opt = m.AdamW([p], lr=0.0, weight_decay=0.0, state="mxfp8")
    gp = torch.ones(1000, device="cuda")

    def work():
        n = m.rms_norm(x, wn, residual=r, mxfp8=True)
        y, z = m.linear(n.y, w1, activation="gelu", save_z=True)
        one, _ = m.linear(y[:1], w2)
        d = m.linear_backward(y, n.y, w1, z=z, activation="gelu", bias=True)
        b = m.rms_norm_backward(d["dx"], n.h, wn, n.rstd, d_h=r)
        opt.step([gp])
        return [n.y, n.mx[0], y, one, d["d_weight"], d["d_bias"], b["dx"], b["d_weight"]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # warm-up outside the capture
        work()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for _ in range(2):
        x.copy_(rand(300, 512))
        r.copy_(rand(300, 512))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert m.linear_status() == 0


def test_gradients_at_odd_addresses():
    """Rows of 17 behind a row of another tensor: the concatenation's backward
    hands the norm a contiguous gradient that begins at an odd address."""
    mok()
    from mixture_experts_layer_mok_gb300.autograd import rms_norm

    g = torch.Generator().manual_seed(4)
    x, r, w, top = (torch.randn(*s, generator=g).to(BF16).cuda() for s in ((3, 17), (3, 17), (17,), (1, 17)))
    c = torch.randn(4, 17, generator=g).to(BF16).cuda()

    def grads(join):
        leaves = [t.clone().requires_grad_() for t in (x, w, r)]
        y, h = rms_norm(leaves[0], leaves[1], leaves[2])
        if join:
            y, h = torch.cat([top, y]) * c, torch.cat([top, h]) * c
        else:
            y, h = y * c[1:], h * c[1:]
        (y.float().sum() + h.float().sum()).backward()
        return [t.grad for t in leaves]

    assert all(torch.equal(a, b) for a, b in zip(grads(True), grads(False)))
