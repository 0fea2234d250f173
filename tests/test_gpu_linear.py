"""The dense projection with bias, activation and residual, and its backward,
against 64-bit restatements on the CPU.

Error bounds, from the arithmetic: products of bf16 values are exact in fp32;
the tensor core adds them in steps of 16, each step good to 2^-23 of the terms
seen so far, so a sum over K is within (K/16 + 8) 2^-23 of the sum of its
terms' sizes (written S).  An activation's slope is at most 1.13 and its own
error below 4e-6 of |z|.  Rounding to bf16 adds 2^-8 (U) of the value.  In the
backward dz is rounded to bf16 before the products: U of each term more."""
import pytest
import torch

from tests.gpu_util import mok

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -8
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _f(K):
    return (K / 16 + 8) * 2.0 ** -23


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def slope64(z, act):
    z = z.clone().requires_grad_(True)
    return torch.autograd.grad(act64(z, act).sum(), z)[0] if act != "none" else torch.ones_like(z)


def _rand(g, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _within(got, ref, bound, what):
    err = (got.double().cpu() - ref).abs()
    assert not torch.isnan(err).any(), what
    worst = (err / bound.clamp(min=1e-30)).max().item() if err.numel() else 0.0
    assert worst <= 1.0, (what, worst)


# one token to many, N and K at and around the tiles' edges, K shorter than a
# block, products for the split kernel (1 to 8 CTAs) and for the pair kernel
SHAPES = [(1, 8, 8), (1, 128, 64), (1, 7168, 2048), (2, 136, 72), (3, 1000, 1032), (8, 256, 4096), (15, 264, 520),
          (16, 128, 7168), (17, 120, 200), (32, 2048, 512), (33, 384, 136), (63, 64, 64), (64, 1416, 2056),
          (65, 72, 1000), (100, 8, 16), (127, 520, 264), (128, 128, 128), (129, 136, 8), (257, 256, 7168),
          (1003, 1416, 2056), (4096, 256, 1024), (2500, 2056, 72), (2561, 2304, 520), (19500, 200, 136)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act,bias,res,out,save_z", [("none", None, None, "bf16", False), ("gelu", "bf16", None, "bf16", True),
                                                     ("silu", None, "bf16", "bf16", False),
                                                     ("relu", "f32", "f32", "f32", True),
                                                     ("gelu_tanh", "f32", "bf16", "f32", False)])
def test_forward(M, N, K, act, bias, res, out, save_z):
    m = mok()
    T = {"bf16": BF16, "f32": F32}
    g = torch.Generator().manual_seed(M + 3 * N + 7 * K)
    x, w = _rand(g, M, K), _rand(g, N, K, std=K ** -0.5)
    b = None if bias is None else _rand(g, N, dtype=T[bias])
    r = None if res is None else _rand(g, M, N, dtype=T[res])
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    y, z = m.linear(c(x), c(w), bias=c(b), activation=act, residual=c(r), out_dtype=T[out], save_z=save_z)
    assert m.linear_status() == 0
    z64 = x.double() @ w.double().t()
    size = x.double().abs() @ w.double().abs().t()
    if b is not None:
        z64 = z64 + b.double()
        size = size + b.double().abs()
    y64 = act64(z64, act) + (0.0 if r is None else r.double())
    fz = _f(K) * size
    fy = 1.13 * fz + 4e-6 * (z64.abs() + y64.abs())
    _within(y, y64, fy + (U * y64.abs() if out == "bf16" else 0.0), "y")
    if save_z:
        _within(z, z64, fz + U * z64.abs(), "z")
    else:
        assert z is None
    again, _ = m.linear(c(x), c(w), bias=c(b), activation=act, residual=c(r), out_dtype=T[out], save_z=save_z)
    assert torch.equal(again, y)


@pytest.mark.parametrize("M,N,K", SHAPES + [(2048, 2504, 2304), (5000, 1032, 1096)])
@pytest.mark.parametrize("act,bias,dyt", [("none", False, "bf16"), ("none", True, "bf16"), ("gelu", True, "bf16"),
                                          ("silu", True, "f32"), ("none", True, "f32")])
def test_backward(M, N, K, act, bias, dyt):
    m = mok()
    g = torch.Generator().manual_seed(M + 3 * N + 7 * K + 1)
    x, w, dy = _rand(g, M, K), _rand(g, N, K, std=K ** -0.5), _rand(g, M, N, dtype=BF16 if dyt == "bf16" else F32)
    z = _rand(g, M, N, std=1.5) if act != "none" else None
    out = m.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z=None if z is None else z.cuda(), activation=act, bias=bias)
    assert m.linear_status() == 0
    dz = dy.double()
    slope_err = torch.zeros_like(dz)
    if act != "none":
        dz = dz * slope64(z.double(), act)
        slope_err = 4e-6 * dy.double().abs() * (1 + z.double().abs())
    rounded = U if act != "none" or dyt == "f32" else 0.0
    term = rounded * dz.abs() + slope_err
    wd, xd = w.double(), x.double()
    for key, ref, size, extra, k in (("dx", dz @ wd, dz.abs() @ wd.abs(), term @ wd.abs(), N),
                                     ("d_weight", dz.t() @ xd, dz.abs().t() @ xd.abs(), term.t() @ xd.abs(), M)):
        _within(out[key], ref, _f(k) * size * 1.01 + extra * 1.01 + U * ref.abs(), key)
        if M > 1:   # roundings of 2^-9 at random, of dz and of the result, each about 1.7e-3 in norm
            assert torch.linalg.norm(out[key].double().cpu() - ref) <= 4e-3 * torch.linalg.norm(ref), key
    if bias:
        _within(out["d_bias"], dz.sum(0), (M / 8 + 64) * 2.0 ** -24 * dz.abs().sum(0) + slope_err.sum(0), "d_bias")
    else:
        assert "d_bias" not in out
    again = m.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z=None if z is None else z.cuda(), activation=act, bias=bias)
    assert all(torch.equal(again[k], out[k]) for k in out)


@pytest.mark.parametrize("act", ACTS)
def test_slopes_against_differences(act):
    """dz through the kernel (dx with a one-hot weight) against central
    differences of the 64-bit activation; bf16 rounding of dz and dx: 2 U."""
    m = mok()
    z = torch.linspace(-8, 8, 2048).to(BF16).view(256, 8)
    z = torch.where(z.abs() < 1e-3, torch.full_like(z, 0.5), z)      # away from relu's corner
    eye = torch.eye(8, dtype=BF16).cuda()
    out = m.linear_backward(torch.ones(256, 8, dtype=BF16, device="cuda"), torch.zeros(256, 8, dtype=BF16, device="cuda"),
                            eye, z=z.cuda(), activation=act, bias=True)
    h = 1e-6
    num = (act64(z.double() + h, act) - act64(z.double() - h, act)) / (2 * h)
    _within(out["dx"], num, 2 * U * num.abs() + 1e-5, "slope")
    _within(out["d_bias"], num.sum(0), torch.full((8,), 256 * 1e-5), "sum")


def test_gradient_against_differences():
    """The whole operator: central differences of the 64-bit forward in x, W
    and b at the kernel's inputs.  dz and the gradients are rounded to bf16."""
    m = mok()
    M, N, K = 5, 16, 24
    g = torch.Generator().manual_seed(4)
    x, w, b, dy = _rand(g, M, K), _rand(g, N, K, std=0.3), _rand(g, N, dtype=F32), _rand(g, M, N)
    y, z = m.linear(x.cuda(), w.cuda(), bias=b.cuda(), activation="gelu", save_z=True)
    out = m.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z=z, activation="gelu", bias=True)

    def loss(x64, w64, b64):
        return (dy.double() * act64(x64 @ w64.t() + b64, "gelu")).sum().item()

    args = [x.double(), w.double(), b.double()]
    for i, key in enumerate(("dx", "d_weight", "d_bias")):
        num = torch.zeros_like(args[i])
        flat = num.view(-1)
        for j in range(flat.numel()):
            hi, lo = [a.clone() for a in args], [a.clone() for a in args]
            hi[i].view(-1)[j] += 1e-5
            lo[i].view(-1)[j] -= 1e-5
            flat[j] = (loss(*hi) - loss(*lo)) / 2e-5
        # z itself was rounded for the backward: U |z| times a curvature below 0.8
        assert torch.linalg.norm(out[key].double().cpu() - num) <= 1.5e-2 * torch.linalg.norm(num), key


@pytest.mark.parametrize("K", [776, 1536, 1600, 4096])
@pytest.mark.parametrize("act,bias,res,save_z", [("none", None, None, False), ("gelu", F32, BF16, True)])
def test_32_bit_outputs_do_not_lose_with_the_length(K, act, bias, res, save_z):
    """A 2-norm bound that does not grow with K: at most 48 truncating additions
    in a row, each of half of 2^-23 of the sum so far on average, whose size
    over them averages two thirds of its last: 48/2 2^-23 2/3, below 2^-19; one
    row with an infinity beside it."""
    M, N = 2500, 2056
    g = torch.Generator().manual_seed(K)
    x, w = _rand(g, M, K), _rand(g, N, K, std=K ** -0.5)
    x[7, K - 1] = float("inf")
    b = None if bias is None else _rand(g, N, dtype=bias, std=0.1)
    r = None if res is None else _rand(g, M, N, dtype=res)
    y, z = mok().linear(x.cuda(), w.cuda(), bias=None if b is None else b.cuda(), activation=act,
                        residual=None if r is None else r.cuda(), out_dtype=F32, save_z=save_z)
    z64 = x.double().cuda() @ w.double().cuda().T
    z64 = z64 if b is None else z64 + b.double().cuda()
    y64 = act64(z64, act)
    y64 = y64 if r is None else y64 + r.double().cuda()
    rows = torch.arange(M, device="cuda") != 7
    assert ((y[rows].double() - y64[rows]).norm() / y64[rows].norm()).item() <= 2.0 ** -19
    assert torch.isinf(z64[7]).all() and not torch.isfinite(y[7]).all()
    if save_z:
        assert ((z[rows].double() - z64[rows]).norm() / z64[rows].norm()).item() <= 2.0 ** -9
    again, _ = mok().linear(x.cuda(), w.cuda(), bias=None if b is None else b.cuda(), activation=act,
                            residual=None if r is None else r.cuda(), out_dtype=F32, save_z=save_z)
    assert torch.equal(again[rows], y[rows])


@pytest.mark.parametrize("M,N,K", [(3, 136, 200), (300, 264, 136), (2600, 2048, 72)])
def test_infinities_and_nan_stay_in_their_rows(M, N, K):
    m = mok()
    g = torch.Generator().manual_seed(8)
    x, w, r = _rand(g, M, K), _rand(g, N, K, std=K ** -0.5), _rand(g, M, N)
    clean, _ = m.linear(x.cuda(), w.cuda(), residual=r.cuda(), activation="relu")
    x[1, K - 1] = float("nan")
    w[N - 1, 0] = float("inf")
    r[2, 0] = float("-inf")
    y, _ = m.linear(x.cuda(), w.cuda(), residual=r.cuda(), activation="relu")
    keep = torch.ones(M, N, dtype=torch.bool)
    keep[1], keep[:, N - 1], keep[2, 0] = False, False, False
    assert torch.equal(y.cpu()[keep], clean.cpu()[keep])
    assert bool(y[1].isnan().all()) and y[2, 0].item() == float("-inf") and not bool(torch.isfinite(y[0, N - 1])) \
        or bool(x[0, 0] < 0)


def test_empty_leading_axes_and_partial_gradients():
    m = mok()
    g = torch.Generator().manual_seed(2)
    x, w, dy = _rand(g, 2, 3, 64).cuda(), _rand(g, 40, 64).cuda(), _rand(g, 2, 3, 40).cuda()
    y, _ = m.linear(x, w)
    assert y.shape == (2, 3, 40) and torch.equal(y.view(6, 40), m.linear(x.view(6, 64), w)[0])
    out = m.linear_backward(dy, x, w, bias=True)
    assert out["dx"].shape == x.shape
    only = m.linear_backward(dy, x, w, need=("d_weight",))
    assert set(only) == {"d_weight"} and torch.equal(only["d_weight"], out["d_weight"])
    only = m.linear_backward(dy, x, w, need=("dx",))
    assert set(only) == {"dx"} and torch.equal(only["dx"], out["dx"])
    y0, z0 = m.linear(x[:0], w, save_z=True)
    assert y0.shape == (0, 3, 40) and z0.shape == (0, 3, 40)
    e = m.linear_backward(dy[:0], x[:0], w, bias=True)
    assert bool((e["d_weight"] == 0).all()) and bool((e["d_bias"] == 0).all()) and e["dx"].shape == (0, 3, 64)


def test_output_past_32_bit_offsets():
    """An output of 2^31 + elements: its last rows equal those computed alone."""
    m = mok()
    M, N, K = 270000, 8192, 64
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, generator=g, device="cuda", dtype=BF16)
    w = torch.randn(N, K, generator=g, device="cuda", dtype=BF16)
    y, _ = m.linear(x, w)
    last, _ = m.linear(x[-2048:].clone(), w)
    assert torch.equal(y[-2048:], last)
    assert m.linear_status() == 0


@pytest.mark.parametrize("M,N,K", [(1, 40000, 264), (3, 20000, 72), (100, 19600, 64), (19600, 64, 136), (20000, 8, 64),
                                   (9000, 120, 72)])
def test_one_long_side(M, N, K):
    """Outputs with one side narrower than a CTA's tile and the other long, whichever kernel takes them."""
    m = mok()
    g = torch.Generator().manual_seed(M)
    x, w, b, r = _rand(g, M, K), _rand(g, N, K, std=K ** -0.5), _rand(g, N), _rand(g, M, N)
    y, _ = m.linear(x.cuda(), w.cuda(), bias=b.cuda(), residual=r.cuda())
    y64 = x.double() @ w.double().t() + b.double() + r.double()
    size = x.double().abs() @ w.double().abs().t() + b.double().abs() + r.double().abs()
    _within(y, y64, _f(K) * size + U * y64.abs(), "y")
    dy = _rand(g, M, N)
    out = m.linear_backward(dy.cuda(), x.cuda(), w.cuda(), bias=True)
    for key, a, c, k in (("dx", dy, w, N), ("d_weight", dy.t(), x, M)):
        ref = a.double() @ c.double()
        _within(out[key], ref, _f(k) * (a.double().abs() @ c.double().abs()) * 1.01 + U * ref.abs(), key)
    assert m.linear_status() == 0


def test_another_stream_gives_the_same():
    m = mok()
    g = torch.Generator().manual_seed(2)
    x, w, dy = _rand(g, 700, 512).cuda(), _rand(g, 1024, 512).cuda(), _rand(g, 700, 1024).cuda()
    y, z = m.linear(x, w, activation="silu", save_z=True)
    out = m.linear_backward(dy, x, w, z=z, activation="silu", bias=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2, z2 = m.linear(x, w, activation="silu", save_z=True, stream=s)
    out2 = m.linear_backward(dy, x, w, z=z2, activation="silu", bias=True, stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(z, z2) and all(torch.equal(out[k], out2[k]) for k in out)


def test_refusals():
    m = mok()
    x, w = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.zeros(32, 64, dtype=BF16, device="cuda")
    dy = torch.zeros(4, 32, dtype=BF16, device="cuda")
    bad = [lambda: m.linear(x.float(), w), lambda: m.linear(x.cpu(), w), lambda: m.linear(x, w.t()),
           lambda: m.linear(x[:, :56], w), lambda: m.linear(x, w[:30].contiguous()),
           lambda: m.linear(x, w, activation="tanh"), lambda: m.linear(x, w, out_dtype=torch.float16),
           lambda: m.linear(x, w, bias=torch.zeros(31, device="cuda")), lambda: m.linear(x, w, residual=x),
           lambda: m.linear(x[:, ::2], w[:, :32].contiguous()),
           lambda: m.linear_backward(dy, x, w, activation="gelu"), lambda: m.linear_backward(dy[:2], x, w),
           lambda: m.linear_backward(dy, x, w, need=("db",))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"case {i} was taken")
    odd = torch.zeros(4 * 64 + 1, dtype=BF16, device="cuda")[1:].view(4, 64)     # not 16-byte aligned
    with pytest.raises(m.MokError):
        m.linear(odd, w)
    with pytest.raises(m.MokError):
        m.linear_backward(dy, odd, w)


@pytest.mark.parametrize("K", [1600, 4096, 16384])
@pytest.mark.parametrize("M,N", [(1, 40000), (20, 40000), (60, 40000), (100, 40000), (128, 264), (1800, 1800), (4096, 256),
                                 (1003, 1416), (40000, 64)])
def test_32_bit_outputs_do_not_lose_with_the_length_in_any_kernel(M, N, K):
    """The bound of the test above, whichever kernel takes the product and
    however many CTAs share its K: a token or a few beside a large weight (each
    tile width, K whole), fewer tiles than the GPU has pairs (K whole and
    split), a narrow weight."""
    g = torch.Generator(device="cuda").manual_seed(K + M)
    x = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    w = (torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).to(BF16)
    b = torch.randn(N, generator=g, device="cuda")
    r = torch.randn(M, N, generator=g, device="cuda").to(BF16)
    y, z = mok().linear(x, w, bias=b, residual=r, activation="silu", out_dtype=F32, save_z=True)
    plain, _ = mok().linear(x, w, out_dtype=F32)
    z64 = x.double() @ w.double().T
    assert ((plain.double() - z64).norm() / z64.norm()).item() <= 2.0 ** -19
    z64 += b.double()
    y64 = act64(z64, "silu") + r.double()
    assert ((y.double() - y64).norm() / y64.norm()).item() <= 2.0 ** -19
    assert ((z.double() - z64).norm() / z64.norm()).item() <= 2.0 ** -9
    again, _ = mok().linear(x, w, bias=b, residual=r, activation="silu", out_dtype=F32, save_z=True)
    assert torch.equal(again, y) and mok().linear_status() == 0


@pytest.mark.parametrize("M,N,K", [(3, 136, 200), (300, 264, 136), (300, 264, 2056), (2600, 2048, 72), (2600, 2048, 2056)])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", [BF16, F32])
def test_infinities_and_nan_arrive(M, N, K, act, out):
    """A NaN in a row of x is in all of that row's outputs, an infinite weight
    in its column with x's sign, an infinite residual in its element; nowhere
    else."""
    m = mok()
    g = torch.Generator().manual_seed(8)
    x, w, r = _rand(g, M, K), _rand(g, N, K, std=K ** -0.5), _rand(g, M, N)
    assert bool((x[:, 0] != 0).all())
    clean, _ = m.linear(x.cuda(), w.cuda(), residual=r.cuda(), activation=act, out_dtype=out)
    x[1, K - 1] = float("nan")
    w[N - 1, 0] = float("inf")
    r[2, 0] = float("-inf")
    y, z = m.linear(x.cuda(), w.cuda(), residual=r.cuda(), activation=act, out_dtype=out, save_z=True)
    y, z, clean = y.cpu(), z.cpu(), clean.cpu()
    keep = torch.ones(M, N, dtype=torch.bool)
    keep[1], keep[:, N - 1], keep[2, 0] = False, False, False
    assert torch.equal(y[keep], clean[keep])
    assert bool(y[1].isnan().all()) and bool(z[1].isnan().all())
    assert y[2, 0].item() == float("-inf") and bool(z[2, 0].isfinite())
    rows = torch.arange(M) != 1
    up, down = rows & (x[:, 0] > 0), rows & (x[:, 0] < 0)
    assert bool((z[up, N - 1] == float("inf")).all()) and bool((z[down, N - 1] == float("-inf")).all())
    assert bool((y[up, N - 1] == float("inf")).all())
    if act == "none":
        assert bool((y[down, N - 1] == float("-inf")).all())
    elif act == "relu":
        assert torch.equal(y[down, N - 1], r[down, N - 1].to(out))
    else:   # their limit is 0, their formula -inf times 0
        assert not bool(y[down, N - 1].isinf().any())
    assert m.linear_status() == 0


@pytest.mark.parametrize("M,N,K", [(1, 7168, 264), (3, 136, 200), (100, 19600, 64), (300, 264, 136), (300, 264, 2056),
                                   (1003, 1416, 2056), (2600, 2056, 72), (2600, 2056, 1032)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_output_may_be_the_residual(M, N, K, dtype):
    """y in the residual's place, through the C ABI: every bit as apart."""
    m = mok()
    from mixture_experts_layer_mok_gb300 import _lib

    g = torch.Generator().manual_seed(M)
    x, w, r = _rand(g, M, K).cuda(), _rand(g, N, K, std=K ** -0.5).cuda(), _rand(g, M, N, dtype=dtype).cuda()
    want, _ = m.linear(x, w, residual=r, activation="gelu", out_dtype=dtype)
    t = _lib.MOK_DTYPE_F32 if dtype == F32 else _lib.MOK_DTYPE_BF16
    s = torch.cuda.current_stream().cuda_stream
    st = _lib.load().mok_linear(x.data_ptr(), w.data_ptr(), None, 0, r.data_ptr(), t, _lib.ACTIVATIONS["gelu"], M, N, K,
                                r.data_ptr(), t, None, s)
    assert st == 0 and torch.equal(r, want) and m.linear_status() == 0


def test_gelu_over_its_range():
    """In 32 bits, from a bias alone: within 4e-7 (its values reach 12: half of
    2^-21 of rounding) and, for negative z, within 4e-3 of the value down to -6."""
    N = 1 << 18
    z = torch.linspace(-12, 12, N, device="cuda")
    x, w = torch.zeros(1, 8, device="cuda", dtype=BF16), torch.zeros(N, 8, device="cuda", dtype=BF16)
    y = mok().linear(x, w, bias=z, activation="gelu", out_dtype=F32)[0][0].double()
    ref = act64(z.double(), "gelu")
    err = (y - ref).abs()
    assert bool((err <= 4e-7 + 2.0 ** -24 * ref.abs()).all())
    tail = (z < 0) & (z > -6)
    assert bool((err[tail] <= 4e-3 * ref[tail].abs()).all())


def test_first_calls_from_several_threads():
    """The launch parameters that are looked up once, first needed by threads at
    the same time (a fresh process: nothing is looked up yet)."""
    import os
    import subprocess
    import sys

    mok()
    code = """
import threading, torch
import mixture_experts_layer_mok_gb300 as m
xs = [torch.randn(M, 512, device="cuda").bfloat16() for M in (1, 300, 9000)]
w = torch.randn(2560, 512, device="cuda").bfloat16()
out, gate = {}, threading.Barrier(8)
def work(i):
    gate.wait()
    out[i] = [m.linear(x, w, activation="silu", stream=torch.cuda.Stream())[0] for x in xs]
ts = [threading.Thread(target=work, args=(i,)) for i in range(8)]
[t.start() for t in ts]; [t.join() for t in ts]
torch.cuda.synchronize()
want = [m.linear(x, w, activation="silu")[0] for x in xs]
assert len(out) == 8 and all(torch.equal(a, b) for o in out.values() for a, b in zip(o, want))
assert m.linear_status() == 0
print("ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip() == "ok", p.stderr[-2000:]
