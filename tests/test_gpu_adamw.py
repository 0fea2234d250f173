"""The AdamW step with 32-bit and MXFP8 states against a 64-bit restatement.

Error bounds: an fp32 result is a handful of roundings of 2^-24 of the terms
it adds; the step itself (m over a root) a dozen, below 2e-6 of its size."""
import numpy as np
import pytest
import torch

from tests.gpu_util import mok

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -22
HYPER = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
LENGTHS = [1, 7, 8, 31, 32, 33, 100, 2047, 2048, 2049, 4096, 10000, 65537]


def _grid_values(codes):
    x = codes.astype(np.int64)
    e, f = (x >> 3) & 15, (x & 7).astype(np.float64)
    mag = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    return np.where(x >= 128, -mag, mag)


def _decode(codes, scales):
    return _grid_values(codes) * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32)[:codes.size]


def _random_bits(n, seed, step, index):
    low = 0xFFFFFFFF
    key = (seed * 0x9E3779B1 + step * 0xB504F333 + index * 0xBB67AE85) & low
    h = ((np.arange(n, dtype=np.uint64) + np.uint64(key)) * np.uint64(0x9E3779B1)) & np.uint64(low)
    h ^= h >> np.uint64(15)
    h = (h * np.uint64(0xB504F333)) & np.uint64(low)
    return (h ^ (h >> np.uint64(16))).astype(np.int64)


def _tensors(lengths, pt, seed):
    g = torch.Generator().manual_seed(seed)
    return [(0.05 * torch.randn(n, generator=g)).to(pt) for n in lengths]


def _step64(p, m, v, g, step, h):
    b1, b2 = h["betas"]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    upd = (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + h["eps"])
    return p * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * upd, m, v, upd


def _np(t):
    return t.detach().double().cpu().numpy().reshape(-1)


@pytest.mark.parametrize("pt,gt,master", [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", False),
                                          ("bf16", "f32", False), ("bf16", "bf16", True), ("bf16", "f32", True)])
def test_fp32_states(pt, gt, master):
    m = mok()
    T = {"bf16": BF16, "f32": F32}
    params = [p.cuda() for p in _tensors(LENGTHS, T[pt], 1)]
    opt = m.AdamW(params, master=master, **HYPER)
    scale = torch.full((1,), 0.5, device="cuda")
    for step in range(1, 4):
        grads = [(g * 0.02).to(T[gt]).cuda() for g in _tensors(LENGTHS, F32, 100 + step)]
        before = [[_np(t) for t in (params[i] if not master else opt.buffers["masters"][i], opt.buffers["m"][i],
                                    opt.buffers["v"][i])] for i in range(len(params))]
        opt.step(grads, grad_scale=scale)
        for i, (p0, m0, v0) in enumerate(before):
            g = 0.5 * _np(grads[i])
            p1, m1, v1, upd = _step64(p0, m0, v0, g, step, HYPER)
            assert (np.abs(_np(opt.buffers["m"][i]) - m1) <= E * (np.abs(m0) + np.abs(g)) + 1e-30).all()
            assert (np.abs(_np(opt.buffers["v"][i]) - v1) <= E * v1 + 1e-37).all()
            # cancellation in m shows in the update: its error is relative to m's terms
            size = HYPER["lr"] * 2e-6 * (np.abs(upd) + (np.abs(m0) + np.abs(g)) / np.maximum(np.sqrt(v1), 1e-12))
            full = opt.buffers["masters"][i] if master else params[i]
            bound = 2 * E * np.abs(p0) + size + (2.0 ** -8 * np.abs(p1) if pt == "bf16" and not master else 0.0)
            assert (np.abs(_np(full) - p1) <= bound).all(), (step, i)
            if master:
                assert torch.equal(params[i], full.to(BF16))


@pytest.mark.parametrize("pt,gt,master", [("f32", "f32", False), ("bf16", "bf16", False), ("bf16", "bf16", True),
                                          ("bf16", "f32", True)])
def test_mxfp8_states(pt, gt, master):
    """Parameters as with 32-bit states (the update uses what is not yet
    rounded); what is kept is the documented neighbour on the grid, except
    where the random bits fall within fp32's error of the threshold."""
    m = mok()
    T = {"bf16": BF16, "f32": F32}
    params = [p.cuda() for p in _tensors(LENGTHS, T[pt], 1)]
    seed = 77
    opt = m.AdamW(params, state="mxfp8", master=master, seed=seed, **HYPER)
    close_calls = total = 0
    for step in range(1, 5):
        grads = [(g * 0.02).to(T[gt]).cuda() for g in _tensors(LENGTHS, F32, 200 + step)]
        grads[6].zero_()
        before = []
        for i in range(len(params)):
            k = [opt.buffers[n][i].cpu().numpy() for n in ("m", "m_scale", "r", "r_scale")]
            before.append((_np(opt.buffers["masters"][i] if master else params[i]), _decode(k[0], k[1]),
                           _decode(k[2], k[3]) ** 2))
        opt.step(grads)
        for i, (p0, m0, v0) in enumerate(before):
            g = _np(grads[i])
            p1, m1, v1, upd = _step64(p0, m0, v0, g, step, HYPER)
            size = HYPER["lr"] * 2e-6 * (np.abs(upd) + (np.abs(m0) + np.abs(g)) / np.maximum(np.sqrt(v1), 1e-12))
            full = opt.buffers["masters"][i] if master else params[i]
            bound = 2 * E * np.abs(p0) + size + (2.0 ** -8 * np.abs(p1) if pt == "bf16" and not master else 0.0)
            assert (np.abs(_np(full) - p1) <= bound).all(), (step, i)
            bits = _random_bits(g.size, seed, step, i)
            for name, val, rnd, slack in (("m", m1, bits >> 16, 4 * E * (np.abs(m0) + np.abs(g))),
                                          ("r", np.sqrt(v1), bits & 0xFFFF, 4 * E * np.sqrt(v1))):
                codes = opt.buffers[name][i].cpu().numpy()
                scales = opt.buffers[name + "_scale"][i].cpu().numpy()
                pad = np.zeros(-val.size % 32)
                amax = np.abs(np.concatenate([val, pad])).reshape(-1, 32).max(1)
                with np.errstate(divide="ignore"):
                    s = np.where(amax > 0, np.ceil(np.log2(np.where(amax > 0, amax, 1.0) / 448.0)), 0.0)
                near = amax > 0
                near &= np.abs(amax / (448 * 2.0 ** np.round(np.log2(np.where(amax > 0, amax, 1) / 448))) - 1) < 1e-5
                assert ((scales.astype(np.float64) - 127 == s) | near).all(), (step, i, name)
                unit = np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32)[:val.size]
                a = np.abs(val) / unit
                got = np.abs(_grid_values(codes))
                e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
                gap = 2.0 ** (e - 3)
                t = a / gap + rnd / 65536.0
                want = np.floor(t) * gap
                if name == "r":
                    want = np.where((val > 0) & (want == 0), 2.0 ** -9, want)
                unsure = np.abs(t - np.round(t)) < 2.0 ** -16 + slack / unit / gap
                off = got != want
                assert not (off & ~unsure).any(), (step, i, name, np.nonzero(off & ~unsure)[0][:5])
                assert (np.abs(got - a) <= gap * (1 + 1e-5) + slack / unit).all()
                assert ((_grid_values(codes) * np.sign(val) >= 0) | (np.abs(val) <= slack)).all()
                close_calls += int(off.sum())
                total += val.size
    assert close_calls <= 1e-3 * total + 3


def _kept32(x, rand16, keep_positive):
    """The codes and scales of fp32 x (whole blocks): E4M3 neighbours chosen by 16 random bits."""
    b = x.reshape(-1, 32)
    mant, e = np.frexp(np.abs(b).max(1))
    s = np.where(mant <= 0.875, e - 9, e - 8).clip(-127, 127)
    s = np.where(mant == 0, 0, s)
    y = np.ldexp(b, -s[:, None]).astype(np.float32)
    off = np.where(np.abs(y) < np.float32(2.0 ** -6), np.float32(2.0 ** -6), np.float32(0))
    bits = (np.abs(y) + off).astype(np.float32).view(np.uint32) + (rand16.reshape(-1, 32).astype(np.uint32) << np.uint32(4))
    q = (bits & np.uint32(0xFFF00000)).view(np.float32) - off
    if keep_positive:
        q = np.where((y > 0) & (q == 0), np.float32(2.0 ** -9), q)
    return np.copysign(q, y).reshape(-1), s


@pytest.mark.parametrize("seed", [5, 6])
def test_mxfp8_states_are_those_of_separately_rounded_operations(seed):
    """m, v and sqrt(v) are each operation rounded once to fp32, so that every
    element falls on the same side of its random bits as in a restatement of
    that kind: no code differs, over millions of elements."""
    n = 1 << 21
    (p,), b1, b2 = _tensors([n], F32, seed), *HYPER["betas"]
    opt = mok().AdamW([p.cuda()], state="mxfp8", seed=seed, **HYPER)
    f = np.float32
    for step in range(1, 4):
        g = (_tensors([n], F32, 10 * seed + step)[0] * 0.02)
        kept = {k: opt.buffers[k][0].cpu().numpy() for k in ("m", "m_scale", "r", "r_scale")}
        m0 = _decode(kept["m"], kept["m_scale"]).astype(f)
        r0 = _decode(kept["r"], kept["r_scale"]).astype(f)
        opt.step([g.cuda()])
        g = g.numpy()
        m1 = f(b1) * m0 + f(1 - b1) * g
        r1 = np.sqrt(f(b2) * (r0 * r0) + f(1 - b2) * g * g)
        assert m1.dtype == r1.dtype == f
        bits = _random_bits(n, seed, step, 0)
        for name, x, rand16 in (("m", m1, bits >> 16), ("r", r1, bits & 0xFFFF)):
            want, s = _kept32(x, rand16, name == "r")
            assert np.array_equal(opt.buffers[name + "_scale"][0].cpu().numpy(), s + 127), (step, name)
            got = _grid_values(opt.buffers[name][0].cpu().numpy())
            assert np.array_equal(got, want.astype(np.float64)), (step, name, int((got != want).sum()))


def test_rounding_is_right_on_average():
    """Steps with a zero gradient shrink r by sqrt(b2) = 0.05% each, far below
    the grid's spacing: after 200 of them the mean has shrunk as it should.
    The mean of n = 65536 values, each a product of unbiased roundings of at
    most 12%, has a deviation of about 0.12 sqrt(200 / 12 n) < 0.2%; 5 of them."""
    m = mok()
    n = 65536
    p = torch.zeros(n, device="cuda")
    opt = m.AdamW([p], lr=0.0, betas=(0.9, 0.999), weight_decay=0.0, state="mxfp8", seed=5)
    opt.step([torch.rand(n, generator=torch.Generator().manual_seed(0)).cuda() + 0.5])
    first = m.mxfp8_dequantize(opt.buffers["r"][0], opt.buffers["r_scale"][0]).double().mean().item()
    zero = torch.zeros(n, device="cuda")
    for _ in range(200):
        opt.step([zero])
    last = m.mxfp8_dequantize(opt.buffers["r"][0], opt.buffers["r_scale"][0]).double().mean().item()
    # E[r^2] decays by b2 exactly; E[r] is a little more, the variance being r's own: stay inside 3%
    assert abs(last / first / 0.999 ** 100 - 1.0) < 0.03, (first, last)


def test_missing_gradients_empty_tensors_and_two_gradient_types():
    m = mok()
    ps = [torch.ones(n, device="cuda") for n in (40, 0, 64, 33)] + [torch.ones(70, dtype=BF16, device="cuda")]
    opt = m.AdamW(ps, lr=0.1)
    gs = [torch.ones(40, device="cuda"), torch.ones(0, device="cuda"), None,
          torch.ones(33, dtype=BF16, device="cuda"), torch.ones(70, dtype=BF16, device="cuda")]
    opt.step(gs)
    assert bool((ps[2] == 1).all()) and bool((opt.buffers["m"][2] == 0).all())
    for i in (0, 3, 4):
        assert (ps[i].float() - (1 - 0.1 * 0.01 - 0.1)).abs().max() < 4e-3, i
    gs[2] = torch.ones(64, device="cuda")
    opt.step(gs)
    assert bool((ps[2] < 1).all())
    for p, g in zip(ps, gs):
        p.grad = g.to(p.dtype)
    opt.step()
    assert opt.step_count == 3


def test_many_tensors_span_launches_and_reproduce():
    m = mok()
    lengths = [(i * 37) % 900 + 1 for i in range(1000)]

    def run(state):
        ps = [p.cuda() for p in _tensors(lengths, F32, 3)]
        opt = m.AdamW(ps, state=state, seed=9, **HYPER)
        for k in range(2):
            opt.step([g.cuda() for g in _tensors(lengths, F32, 50 + k)])
        return ps, opt

    one, _ = run("fp32")
    for i in (0, 399, 400, 401, 799, 800, 999):      # tensor i alone
        p = _tensors(lengths, F32, 3)[i].cuda()
        opt = m.AdamW([p], **HYPER)
        for k in range(2):
            opt.step([_tensors(lengths, F32, 50 + k)[i].cuda()])
        assert torch.equal(p, one[i]), i
    (a, oa), (b, ob) = run("mxfp8"), run("mxfp8")
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    for name in oa.buffers:
        assert all(torch.equal(x, y) for x, y in zip(oa.buffers[name], ob.buffers[name]))


@pytest.mark.parametrize("state,master", [("fp32", False), ("mxfp8", True)])
def test_state_round_trip_continues_the_run(state, master):
    m = mok()
    pt = BF16 if master else F32

    def fresh():
        ps = [p.cuda() for p in _tensors([300, 64], pt, 3)]
        return ps, m.AdamW(ps, state=state, master=master, seed=4, **HYPER)

    gs = [[g.cuda() for g in _tensors([300, 64], F32, 60 + k)] for k in range(4)]
    ps, opt = fresh()
    for k in range(4):
        opt.step(gs[k])
    qs, half = fresh()
    half.step(gs[0])
    half.step(gs[1])
    rs, rest = fresh()
    for r, q in zip(rs, qs):
        r.copy_(q)
    rest.load_state_dict(half.state_dict())
    rest.step(gs[2])
    rest.step(gs[3])
    assert all(torch.equal(a, b) for a, b in zip(ps, rs))
    with pytest.raises(ValueError):
        m.AdamW(rs, state="mxfp8" if state == "fp32" else "fp32").load_state_dict(half.state_dict())


def test_a_nan_gradient_stays_in_its_block():
    m = mok()
    p = torch.ones(256, device="cuda")
    opt = m.AdamW([p], state="mxfp8")
    g = torch.ones(256, device="cuda")
    g[40] = float("nan")
    opt.step([g])
    assert bool(p[40].isnan()) and not bool(p[:40].isnan().any()) and not bool(p[41:].isnan().any())
    r = m.mxfp8_dequantize(opt.buffers["r"][0], opt.buffers["r_scale"][0])
    assert not bool(r[:32].isnan().any()) and not bool(r[64:].isnan().any())


def test_a_backward_notices_the_step():
    m = mok()
    w = torch.nn.Parameter(torch.ones(64, device="cuda"))
    x = torch.ones(64, device="cuda", requires_grad=True)
    loss = (w * w * x).sum()
    m.AdamW([w]).step([torch.ones(64, device="cuda")])
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        loss.backward()


def test_refusals():
    m = mok()
    p = torch.zeros(64, device="cuda")
    with pytest.raises(ValueError):
        m.AdamW([p.cpu()])
    with pytest.raises(ValueError):
        m.AdamW([p.half()])
    with pytest.raises(ValueError):
        m.AdamW([torch.zeros(8, 8, device="cuda").t()])
    with pytest.raises(ValueError):
        m.AdamW([p], state="int4")
    with pytest.raises(ValueError):
        m.AdamW([p], buffers={"m": [p]})
    with pytest.raises(ValueError):
        m.AdamW([p], buffers={"m": [p[:8]], "v": [p]})
    opt = m.AdamW([p])
    for bad in ([], [p[:8]], [p.half()], [p.cpu()]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(ValueError):
        opt.step([p], grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(m.MokError):
        m.AdamW([p], betas=(1.0, 0.9)).step([p.clone()])
    with pytest.raises(m.MokError):
        opt.step([p.clone()], lr=float("inf"))
    with pytest.raises(m.MokError):
        m.AdamW([torch.zeros(65, device="cuda")[1:]]).step([p])
    assert opt.step_count == 0 and bool((p == 0).all())


def _graph_of(step):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    return graph


@pytest.mark.parametrize("state,master", [("fp32", False), ("mxfp8", False), ("mxfp8", True), ("fp32", True)])
@pytest.mark.parametrize("warm", [0, 2])
def test_a_captured_step_replays_the_step_that_is_due(state, master, warm):
    """Replays, steps called in between, and changes of the learning rate, the
    count, the seed and the state: every bit as in an optimiser that is never
    captured."""
    m = mok()
    pt = BF16 if master else F32
    lengths = [300, 2048, 33]

    def fresh(**kw):
        ps = [p.cuda() for p in _tensors(lengths, pt, 3)] + [torch.ones(70, device="cuda")]
        return ps, m.AdamW(ps, state=state, master=master, **{**HYPER, "seed": 4, **kw})

    (ps, opt), (qs, twin) = fresh(), fresh()
    gs = [torch.empty(n, device="cuda") for n in lengths + [70]]
    gs[1] = gs[1].to(BF16)                      # two gradient types: several launches a step
    scale = torch.ones(1, device="cuda")
    draws = iter(range(1000, 2000))

    def both(one, **kw):
        for t, r in zip(gs, _tensors(lengths + [70], F32, next(draws))):
            t.copy_(0.02 * r)
        one()
        twin.step([t.clone() for t in gs], grad_scale=scale, **kw)
        assert opt.step_count == twin.step_count
        for a, b in zip(ps, qs):
            assert torch.equal(a, b)
        for name in opt.buffers:
            assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(opt.buffers[name], twin.buffers[name]))

    call = lambda: opt.step(gs, grad_scale=scale)  # noqa: E731
    for _ in range(warm):
        both(call)
    graph = _graph_of(call)
    assert opt.step_count == warm               # nothing ran yet
    for _ in range(3):
        both(graph.replay)
    both(call)
    opt.lr = twin.lr = 3e-3
    both(graph.replay)
    both(call)
    fixed = _graph_of(lambda: opt.step(gs, grad_scale=scale, lr=0.1))
    both(fixed.replay, lr=0.1)
    both(graph.replay)
    assert opt.lr == 3e-3
    other = fresh(seed=2 ** 63 + 9, step=7)[1]
    other.step([torch.ones_like(p) for p in other.params])
    for o in (opt, twin):
        o.load_state_dict(other.state_dict())
    assert opt.step_count == 8 and opt.seed == 2 ** 63 + 9
    both(graph.replay)
    both(call)
    assert opt.state_dict()["step"] == 10
    with pytest.raises(ValueError):
        opt.lr = float("nan")


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("which", ["gradient", "parameter"])
def test_a_refused_step_moves_nothing(which, captured):
    """Two launches, the second of which is refused: a retry must not step the
    first group twice."""
    m = mok()
    odd = torch.ones(65, device="cuda")[1:]
    ps = [torch.ones(64, dtype=BF16, device="cuda"), torch.ones(64, device="cuda")]
    good = [torch.ones(64, dtype=BF16, device="cuda"), torch.ones(64, device="cuda")]
    opt = m.AdamW(ps, lr=0.1)
    if captured:
        _graph_of(lambda: opt.step(good))
    if which == "parameter":
        ps[1] = odd
        opt = m.AdamW(ps, lr=0.1)
    version = [p._version for p in ps]
    with pytest.raises(m.MokError):
        opt.step(good if which == "parameter" else [good[0], odd])
    torch.cuda.synchronize()
    assert all(bool((p == 1).all()) for p in ps) and opt.step_count == 0
    assert all(bool((b == 0).all()) for name in ("m", "v") for b in opt.buffers[name])
    assert [p._version for p in ps] == version
    if which == "gradient":
        opt.step(good)
        assert opt.step_count == 1 and all(bool((p < 1).all()) for p in ps)


def test_a_backward_does_not_mind_parameters_that_stayed():
    """A parameter without a gradient is left alone, by its version too; of two
    types, so that each launch's own are told apart."""
    m = mok()
    for dtype in (F32, BF16):
        kept, moved = (torch.nn.Parameter(torch.ones(64, device="cuda", dtype=dtype)) for _ in range(2))
        x = torch.ones(64, device="cuda", dtype=dtype, requires_grad=True)
        loss = (kept * kept * x).sum()
        before = moved._version
        m.AdamW([kept, moved, torch.ones(8, device="cuda")]).step([None, torch.ones_like(moved), None])
        loss.backward()
        assert moved._version > before and bool((kept == 1).all()) and bool((x.grad == 1).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), 3e38])
@pytest.mark.parametrize("at", [0, 40, 63, 255, 259])
def test_a_gradient_that_is_not_finite_stays_in_its_element(bad, at):
    """32-bit states hold such a value in one element.  So do MXFP8 states, as
    NaN: every other element, its block's own among them, is to the bit what it
    is in a run where that element's gradient is zero, in the step and in the
    one after.  (3e38 has an infinite square and an m that is finite: it stays
    m's, and sets the scale of its block of m as any value does.)"""
    m = mok()
    n = 260
    g = torch.rand(n, generator=torch.Generator().manual_seed(at)) + 0.5

    def run(value):
        p = torch.ones(n, device="cuda")
        opt = m.AdamW([p], state="mxfp8", seed=3)
        for k in range(2):
            gk = (1.0 + k) * g
            gk[at] = value if k == 0 else gk[at] * 0
            opt.step([gk.cuda()])
            kept = {name: opt.buffers[name][0].cpu().numpy().copy() for name in ("m", "m_scale", "r", "r_scale")}
            yield p.cpu().clone(), kept

    others = np.arange(n) != at
    block = np.arange(n) // 32 == at // 32
    for (p, kept), (p0, kept0) in zip(run(bad), run(0.0)):
        assert not np.isfinite(p[at].item()) or bad == 3e38
        names = ("m", "r") if bad != 3e38 else ("r",)
        for name in names:
            value = _decode(kept[name], kept[name + "_scale"])
            assert (kept[name][at] & 127) == 127            # E4M3's NaN
            assert np.array_equal(value[others], _decode(kept0[name], kept0[name + "_scale"])[others]), name
            assert np.array_equal(kept[name + "_scale"], kept0[name + "_scale"]), name
        if bad == 3e38:
            assert np.array_equal(kept["m"][~block], kept0["m"][~block]) and (kept["m"][at] & 127) != 127
        assert torch.equal(p[others & ~block] if bad == 3e38 else p[others], p0[others & ~block] if bad == 3e38 else p0[others])
