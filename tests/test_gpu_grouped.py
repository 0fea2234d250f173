"""The projections grouped by expert, and their backward, against 64-bit
restatements; the error bounds are those derived in ``test_gpu_linear`` (the
same products and epilogue)."""
import numpy as np
import pytest
import torch

from tests.gpu_util import mok
from tests.test_gpu_linear import U, _f, act64, slope64

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
T = {"bf16": BF16, "f32": F32}


def _within(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert not torch.isnan(err).any(), what
    worst = (err / bound.clamp(min=1e-30)).max().item() if err.numel() else 0.0
    assert worst <= 1.0, (what, worst)


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _rand(g, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _counts(c):
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def _ragged(M, E, seed, tail=0):
    rng = np.random.RandomState(seed)
    share = np.exp(rng.randn(E))
    if E > 3:
        share[rng.randint(E)] = 0.0
    return rng.multinomial(M - tail, share / share.sum()).tolist()


def _slices(counts):
    at = 0
    for e, c in enumerate(counts):
        yield e, slice(at, at + c)
        at += c


# (counts, rows behind, N, K): one row, empty groups, groups around the tiles' edges, odd widths, K shorter than a block
CASES = [
    ([1], 0, 8, 8), ([0, 1, 0], 0, 8, 64), ([0, 0, 0], 5, 16, 72), ([3, 0, 2], 1, 136, 72), ([31, 32, 33], 0, 128, 128),
    ([64, 65, 1, 127, 128, 129], 3, 200, 264), ([255, 256, 257], 0, 256, 512), ([511, 1, 513], 7, 264, 136),
    ([1000], 0, 1032, 1032), ([700, 0, 1500, 2, 0, 300], 11, 712, 520), (_ragged(512, 256, 1), 0, 256, 768),
    (_ragged(1999, 12, 2, 37), 37, 1416, 2056), (_ragged(9001, 20, 3), 0, 520, 712), ([1] * 1024, 0, 64, 64),
    (_ragged(300, 1000, 4), 0, 72, 200), ([20000], 0, 256, 256),
]


def _forward64(x, w, b, counts, act):
    M, N = x.shape[0], w.shape[1]
    z, size = torch.zeros(M, N, dtype=F64, device="cuda"), torch.zeros(M, N, dtype=F64, device="cuda")
    for e, r in _slices(counts):
        z[r], size[r] = x[r].double() @ w[e].double().t(), x[r].double().abs() @ w[e].double().abs().t()
        if b is not None:
            z[r] += b[e].double()
            size[r] += b[e].double().abs()
    return z, act64(z, act), size


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("act,bias,out,save_z", [("none", None, "bf16", False), ("gelu", "bf16", "bf16", True),
                                                 ("silu", "f32", "bf16", False), ("relu", "f32", "f32", True),
                                                 ("gelu_tanh", "bf16", "f32", False)])
def test_forward(case, act, bias, out, save_z):
    m = mok()
    counts, tail, N, K = CASES[case]
    E, M = len(counts), sum(counts) + tail
    g = _gen(case)
    x, w = _rand(g, M, K), _rand(g, E, N, K, std=K ** -0.5)
    x[M - tail:] = float("nan")               # rows of no group are not computed with
    b = None if bias is None else _rand(g, E, N, dtype=T[bias])
    call = lambda: m.grouped_linear(x, w, _counts(counts), bias=b, activation=act, out_dtype=T[out], save_z=save_z)  # noqa: E731
    y, z = call()
    assert m.linear_status() == 0
    z64, y64, size = _forward64(x, w, b, counts, act)
    fz = _f(K) * size
    fy = 1.13 * fz + 4e-6 * (z64.abs() + y64.abs())
    _within(y, y64, fy + (U * y64.abs() if out == "bf16" else 0.0), "y")
    assert (y[M - tail:] == 0).all()
    if save_z:
        _within(z, z64, fz + U * z64.abs(), "z")
        assert (z[M - tail:] == 0).all()
    else:
        assert z is None
    again, _ = call()
    assert torch.equal(again, y)


@pytest.mark.parametrize("counts", [[63], [64], [127], [128], [129], [191], [192], [255], [256], [0, 257], [320, 130], [64] * 39,
                                    [256] * 76 + [200], [256] * 80 + [1, 129], [130] * 19])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N", [256, 264])
def test_few_tiles(counts, out, N):
    """A last round of few tiles, which are cut by rows: each count around the parts' 64."""
    m = mok()
    E, M, K = len(counts), sum(counts) + 3, 136
    g = _gen(M + N)
    x, w, b = _rand(g, M, K), _rand(g, E, N, K, std=K ** -0.5), _rand(g, E, N, dtype=F32)
    x[M - 3:] = float("nan")
    y, _ = m.grouped_linear(x, w, _counts(counts), bias=b, out_dtype=T[out])
    assert m.linear_status() == 0
    _, y64, size = _forward64(x, w, b, counts, "none")
    _within(y, y64, 1.13 * _f(K) * size + 4e-6 * 2 * y64.abs() + (U * y64.abs() if out == "bf16" else 0.0), "y")
    assert (y[M - 3:] == 0).all()


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("act,bias,dyt", [("none", False, "bf16"), ("none", True, "bf16"), ("gelu", True, "bf16"),
                                          ("silu", True, "f32"), ("none", True, "f32"), ("relu", False, "bf16")])
def test_backward(case, act, bias, dyt):
    m = mok()
    counts, tail, N, K = CASES[case]
    E, M = len(counts), sum(counts) + tail
    g = _gen(100 + case)
    x, w, dy = _rand(g, M, K), _rand(g, E, N, K, std=K ** -0.5), _rand(g, M, N, dtype=T[dyt])
    z = _rand(g, M, N, std=1.5) if act != "none" else None
    for t in (x, dy, z):
        if t is not None:
            t[M - tail:] = float("nan")
    call = lambda **kw: m.grouped_linear_backward(dy, x, w, _counts(counts), z=z, activation=act, bias=bias, **kw)  # noqa: E731
    out = call()
    assert m.linear_status() == 0
    assert set(out) == {"dx", "d_weight"} | ({"d_bias"} if bias else set())
    assert (out["dx"][M - tail:] == 0).all()
    rounded = U if act != "none" or dyt == "f32" else 0.0
    for e, r in _slices(counts):
        dz, slope_err = dy[r].double(), torch.zeros_like(dy[r], dtype=F64)
        if act != "none":
            # at 0 itself relu's slope is 0, by definition here, where the clamp's derivative is 1
            dz = dz * ((z[r] > 0).double() if act == "relu" else slope64(z[r].double(), act))
            slope_err = 4e-6 * dy[r].double().abs() * (1 + z[r].double().abs())
        term = rounded * dz.abs() + slope_err
        wd, xd, n = w[e].double(), x[r].double(), counts[e]
        if n == 0:
            assert (out["d_weight"][e] == 0).all() and (not bias or (out["d_bias"][e] == 0).all())
            continue
        for got, ref, size, extra, k in ((out["dx"][r], dz @ wd, dz.abs() @ wd.abs(), term @ wd.abs(), N),
                                         (out["d_weight"][e], dz.t() @ xd, dz.abs().t() @ xd.abs(), term.t() @ xd.abs(), n)):
            _within(got, ref, _f(k) * size * 1.01 + extra * 1.01 + U * ref.abs(), (e, k))
        if bias:
            _within(out["d_bias"][e], dz.sum(0), (n / 8 + 64) * 2.0 ** -24 * dz.abs().sum(0) + slope_err.sum(0) + 1e-30, "d_bias")
    again = call()
    assert all(torch.equal(again[k], out[k]) for k in out)
    for need in (("dx",), ("d_weight",), ()):
        part = call(need=need)
        assert set(part) == set(need) | ({"d_bias"} if bias else set())
        assert all(torch.equal(part[k], out[k]) for k in part)


def test_neighbours_do_not_leak():
    """A group's results depend on its own rows alone: NaN in every other group's rows, weights and gradients."""
    m = mok()
    counts, N, K = [70, 1, 129, 40, 300], 136, 200
    g = _gen(7)
    M = sum(counts)
    x, w, dy = _rand(g, M, K), _rand(g, 5, N, K), _rand(g, M, N)
    y, _ = m.grouped_linear(x, w, _counts(counts))
    b = m.grouped_linear_backward(dy, x, w, _counts(counts), bias=True)
    for e, r in _slices(counts):
        x2, w2, dy2 = torch.full_like(x, float("nan")), torch.full_like(w, float("nan")), torch.full_like(dy, float("nan"))
        x2[r], w2[e], dy2[r] = x[r], w[e], dy[r]
        assert torch.equal(m.grouped_linear(x2, w2, _counts(counts))[0][r], y[r])
        b2 = m.grouped_linear_backward(dy2, x2, w2, _counts(counts), bias=True)
        assert torch.equal(b2["dx"][r], b["dx"][r]) and torch.equal(b2["d_weight"][e], b["d_weight"][e])
        assert torch.equal(b2["d_bias"][e], b["d_bias"][e])


def test_one_group_is_the_plain_projection():
    """Close to ``linear`` (the sums' order differs): each within its bound of the same value."""
    m = mok()
    g = _gen(8)
    x, w = _rand(g, 777, 520), _rand(g, 1, 264, 520, std=520 ** -0.5)
    y, _ = m.grouped_linear(x, w, _counts([777]), out_dtype=F32)
    ref, _ = m.linear(x, w[0], out_dtype=F32)
    size = x.double().abs() @ w[0].double().abs().t()
    _within(y, ref.double(), 2 * _f(520) * size, "y")


def test_no_rows():
    m = mok()
    x, w = torch.empty(0, 64, dtype=BF16, device="cuda"), torch.ones(3, 32, 64, dtype=BF16, device="cuda")
    c = _counts([0, 0, 0])
    y, z = m.grouped_linear(x, w, c, save_z=True)
    assert y.shape == (0, 32) and z.shape == (0, 32)
    out = m.grouped_linear_backward(torch.empty(0, 32, dtype=BF16, device="cuda"), x, w, c, bias=True)
    assert out["dx"].shape == (0, 64) and (out["d_weight"] == 0).all() and (out["d_bias"] == 0).all()


def test_bad_counts_are_bounded_and_reported():
    """Counts below 0 and beyond the rows: clamped on the device, and told by the status."""
    m = mok()
    from mixture_experts_layer_mok_gb300 import _lib

    g = _gen(9)
    x, w, dy = _rand(g, 100, 64), _rand(g, 4, 32, 64), _rand(g, 100, 32)
    assert m.linear_status() == 0
    for bad, good in (([40, -3, 30, 10], [40, 0, 30, 10]), ([60, 60, 5, 0], [60, 40, 0, 0]),
                      ([2 ** 31 - 1] * 4, [100, 0, 0, 0]), ([-2 ** 31] * 4, [0, 0, 0, 0])):
        y, _ = m.grouped_linear(x, w, _counts(bad))
        assert m.linear_status() == _lib.MOK_ERR_INDEX and m.linear_status() == 0
        assert torch.equal(y, m.grouped_linear(x, w, _counts(good))[0])
        out = m.grouped_linear_backward(dy, x, w, _counts(bad), bias=True)
        assert m.linear_status() == _lib.MOK_ERR_INDEX
        ref = m.grouped_linear_backward(dy, x, w, _counts(good), bias=True)
        assert all(torch.equal(out[k], ref[k]) for k in out) and m.linear_status() == 0


def test_streams_graph_and_workspaces():
    """Two captured backwards replayed with other counts, each with its own workspace, on two streams at a time."""
    m = mok()
    g = _gen(10)
    E, N, K, M = 6, 264, 328, 500
    sides = [torch.cuda.Stream() for _ in range(2)]
    bufs, graphs, outs = [], [], []
    for s in sides:
        x, w, dy, c = _rand(g, M, K), _rand(g, E, N, K), _rand(g, M, N), _counts([10] * E)
        z = _rand(g, M, N)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            y, _ = m.grouped_linear(x, w, c, activation="silu")
            out = m.grouped_linear_backward(dy, x, w, c, z=z, activation="silu", bias=True)
        bufs.append((x, w, dy, c, z))
        graphs.append(graph)
        outs.append((y, out))
    for trial in range(3):
        for (x, w, dy, c, z) in bufs:
            c.copy_(_counts(_ragged(M - 3, E, 20 + trial)))
            x.copy_(_rand(g, M, K))
        torch.cuda.synchronize()
        for s, graph in zip(sides, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (x, w, dy, c, z), (y, out) in zip(bufs, outs):
            assert torch.equal(y, m.grouped_linear(x, w, c, activation="silu")[0])
            ref = m.grouped_linear_backward(dy, x, w, c, z=z, activation="silu", bias=True)
            assert all(torch.equal(out[k], ref[k]) for k in ref)
    assert m.linear_status() == 0


def test_gradient_against_differences():
    """A directional derivative of a smooth function of the outputs, in fp32 outputs: bf16 parameters stepped by exact
    powers of two."""
    m = mok()
    from mixture_experts_layer_mok_gb300.autograd import grouped_linear

    g = _gen(11)
    counts, N, K = [9, 0, 14, 5], 24, 16
    x, w = _rand(g, 30, K), _rand(g, 4, N, K, std=0.3)
    b = _rand(g, 4, N, dtype=F32)
    cot = _rand(g, 30, N)
    leaves = [t.clone().requires_grad_(True) for t in (x, w, b)]
    y = grouped_linear(leaves[0], leaves[1], _counts(counts), leaves[2], "gelu_tanh", F32)
    y.backward(cot.float())

    def f(x64, w64, b64):
        total = 0.0
        for e, r in _slices(counts):
            total = total + (act64(x64[r] @ w64[e].t() + b64[e], "gelu_tanh") * cot[r].double()).sum()
        return total

    base = [t.double() for t in (x, w, b)]
    for i in range(3):
        d = _rand(g, *base[i].shape, dtype=F64)
        h = 1e-5
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + h * d, base[i] - h * d
        num = (f(*up) - f(*down)) / (2 * h)
        got = (leaves[i].grad.double() * d).sum()
        # dz and the gradients are each rounded to bf16 (U of every term; z too, through the slope, of order U): the terms'
        # sizes, with slopes up to 1.13 and slopes of slopes up to 1.2
        size = 0.0
        for e, r in _slices(counts):
            dz = 1.13 * cot[r].double().abs() * (1 + base[0][r].abs() @ base[1][e].abs().t() + base[2][e].abs())
            dd = d[r].abs() if i == 0 else d[e].abs()
            size = size + (((dz @ base[1][e].abs()) * dd).sum() if i == 0 else ((dz.t() @ base[0][r].abs()) * dd).sum() if i == 1
                           else (dz.sum(0) * dd).sum())
        assert (got - num).abs() <= 3 * U * size, i


def test_long_outputs():
    """Outputs beyond 2^31 elements: a group at the end of a long batch, whose offsets pass 32 bits."""
    m = mok()
    g = _gen(12)
    M, N, K, last = 1 << 20, 2304, 64, 321
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    x[-last:] = _rand(g, last, K)
    w = _rand(g, 2, N, K)
    y, _ = m.grouped_linear(x, w, _counts([M - last, last]))
    assert torch.equal(y[-last:], m.grouped_linear(x[-last:].clone(), w[1:].clone(), _counts([last]))[0])
    assert (y[:-last] == 0).all()
    dy = torch.zeros_like(y)
    dy[-last:] = _rand(g, last, N)
    out = m.grouped_linear_backward(dy, x, w, _counts([M - last, last]), bias=True)
    ref = m.grouped_linear_backward(dy[-last:].clone(), x[-last:].clone(), w[1:].clone(), _counts([last]), bias=True)
    assert torch.equal(out["dx"][-last:], ref["dx"]) and (out["dx"][:-last] == 0).all()
    assert torch.equal(out["d_weight"][1:], ref["d_weight"]) and (out["d_weight"][0] == 0).all()
    total = dy[-last:].double().sum(0)
    _within(out["d_bias"][1], total, (last / 8 + 64) * 2.0 ** -24 * dy[-last:].double().abs().sum(0), "d_bias")
    assert m.linear_status() == 0


def test_refusals():
    m = mok()
    x, w, c = torch.ones(4, 64, dtype=BF16, device="cuda"), torch.ones(3, 32, 64, dtype=BF16, device="cuda"), _counts([1, 2, 1])
    for kw in (dict(activation="swish"), dict(out_dtype=torch.float16), dict(bias=torch.ones(32, device="cuda")),
               dict(bias=torch.ones(3, 32, device="cuda", dtype=torch.float16))):
        with pytest.raises(ValueError):
            m.grouped_linear(x, w, c, **kw)
    for a in ((x[:, :32], w, c), (x[:, ::2], w[:, :, :32].contiguous(), c), (x, w[0], c), (x, w.transpose(1, 2), c), (x, w, c.long()),
              (x, w, c[:2]), (x.float(), w, c), (x, w, c.cpu()), (x, torch.ones(3, 12, 64, dtype=BF16, device="cuda"), c),
              (x.view(2, 2, 64), w, c)):
        with pytest.raises(ValueError):
            m.grouped_linear(*a)
    dy = torch.ones(4, 32, dtype=BF16, device="cuda")
    for kw in (dict(activation="gelu"), dict(need=("dw",)), dict(activation="gelu", z=dy[:2])):
        with pytest.raises(ValueError):
            m.grouped_linear_backward(dy, x, w, c, **kw)
    with pytest.raises(m.MokError):           # 16-byte alignment: a view that begins between
        m.grouped_linear(torch.ones(4 * 64 + 4, dtype=BF16, device="cuda")[4:].view(4, 64), w, c)


def test_as_many_rows_as_there_can_be():
    """2^31 - 513 rows of 8: tiles, chunks and offsets at the end of 32 bits.  Rows
    of small integers among zeros, so that every result is exact in bf16, and NaN
    behind the last expert's rows."""
    m = mok()
    M, tail, first = (1 << 31) - 513, 5, 7
    last = M - tail
    spans = [(0, 300), (last // 2 - 300, last // 2 + 300), (last - 3000, last)]
    g = torch.Generator("cuda").manual_seed(0)
    ints = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").to(BF16)  # noqa: E731
    counts = torch.tensor([first, last - first], dtype=torch.int32, device="cuda")
    w = ints(2, 8, 8)
    each = w[(torch.cat([torch.arange(a, b) for a, b in spans]) >= first).long().cuda()].double()   # each kept row's weight

    def rows():
        t = torch.zeros(M, 8, dtype=BF16, device="cuda")
        for a, b in spans:
            t[a:b] = ints(b - a, 8)
        t[last:] = float("nan")
        return t, torch.cat([t[a:b] for a, b in spans]).double()

    def check(y, ref):
        assert torch.equal(torch.cat([y[a:b] for a, b in spans]).double(), ref)
        for a, b in spans:
            y[a:b] = 0
        assert not any((y[i:i + (1 << 27)] != 0).any().item() for i in range(0, M, 1 << 27))

    x, kept = rows()
    y, _ = m.grouped_linear(x, w, counts)
    check(y, torch.einsum("rk,rnk->rn", kept, each))
    del y
    z, kept = rows()                 # its own gradient too: ReLU passes what is above 0
    got = m.grouped_linear_backward(z, x, w, counts, z=z, activation="relu", bias=True, need=("dx",))
    dz = kept.clamp(min=0)
    check(got["dx"], torch.einsum("rn,rnk->rk", dz, each))
    assert torch.equal(got["d_bias"].double(), torch.stack([dz[:first].sum(0), dz[first:].sum(0)]))
    assert m.linear_status() == 0
    del x, z, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("counts", [[136], [136] * 3, [200], [208], [224], [232, 200, 8], [256] * 76 + [200], [0, 136, 0, 224]])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_parts_that_leave_few_rows(counts, out):
    """Tiles of a last round whose parts, in steps of 32 rows, leave 8 or 16 for the last."""
    test_few_tiles(counts, out, 264)
