"""The norm with the residual's addition (bf16 and MXFP8 outputs), its
backward and the MXFP8 reader, against 64-bit restatements.

Error bounds, from the arithmetic: a bf16 result is one rounding (2^-8 of its
value at most, written U) of an fp32 value; fp32 sums over a row take at most
about 50 roundings in sequence and the reciprocal root two, below 8e-6 in all
(written F); an E4M3 value is within half a spacing of what it stands for
(2^-4 of the value, or 2^-10 of the block's scale near zero)."""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import mok

pytestmark = pytest.mark.gpu
U, F = 2.0 ** -8, 8e-6
BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}

ROWS_H = [(1, 7168), (1, 1), (3, 8), (5, 32), (7, 40), (33, 256), (4, 264), (9, 512), (6, 520), (2, 1024), (3, 1032),
          (130, 2048), (2, 2056), (3, 4096), (2, 4104), (2, 8192), (2, 8200), (1, 32768), (3, 17), (2, 1001),
          (2, 4095), (2, 4097), (1, 32767), (700, 96), (1300, 64), (2500, 24), (1217, 640)]


def _inputs(rows, H, xt, rt, wt, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 7 + H)
    x = torch.randn(rows, H, generator=g).to(TYPES[xt])
    r = None if rt == "none" else (3.0 * torch.randn(rows, H, generator=g)).to(TYPES[rt])
    w = (1.0 + 0.3 * torch.randn(H, generator=g)).to(TYPES[wt])
    return x, r, w


def _ref(x, r, w, eps):
    h = x.double() + (0.0 if r is None else r.double())
    rstd = 1.0 / torch.sqrt((h * h).mean(-1) + eps)
    return h, rstd, h * rstd[:, None] * w.double()


def _cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def _close(got, ref, bound, what):
    err = (got.double().cpu() - ref).abs()
    worst = (err - bound).max().item() if err.numel() else 0.0
    assert not worst > 0.0 and not torch.isnan(err).any(), (what, worst)


@pytest.mark.parametrize("rows,H", ROWS_H)
@pytest.mark.parametrize("xt,rt,wt", [("bf16", "none", "bf16"), ("bf16", "bf16", "f32"), ("bf16", "f32", "bf16"),
                                      ("f32", "none", "f32"), ("f32", "bf16", "bf16"), ("f32", "f32", "bf16")])
def test_forward(rows, H, xt, rt, wt):
    m = mok()
    x, r, w = _inputs(rows, H, xt, rt, wt)
    h, rstd, y = _ref(x, r, w, 1e-5)
    gx, gr, gw = _cuda(x, r, w)
    mx = H % 32 == 0
    out = m.rms_norm(gx, gw, residual=gr, eps=1e-5, bf16=True, mxfp8=mx)
    _close(out.rstd, rstd, F * rstd, "rstd")
    _close(out.y, y, (U + F) * y.abs(), "y")
    if r is None:
        assert out.h is gx
    else:
        want = (x.float() + r.float()).to(r.dtype)
        assert torch.equal(out.h.cpu(), want)
    if mx:
        codes, scales = out.mx
        dec = m.mxfp8_dequantize(codes, scales).double().cpu()
        s = torch.pow(2.0, scales.cpu().double() - 127.0).repeat_interleave(32, -1).reshape(y.shape)
        _close(dec, y, torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s) * (1 + 1e-5) + F * y.abs(), "mxfp8")
        amax = y.reshape(rows, -1, 32).abs().amax(-1)
        s = s.reshape(rows, -1, 32)[..., 0]
        assert bool((amax <= 448 * s * (1 + F)).all()) and bool((amax > 224 * s * (1 - F)).all())
        only = m.rms_norm(gx, gw, residual=gr, eps=1e-5, bf16=False, mxfp8=True)   # the same codes alone
        assert only.y is None and torch.equal(only.mx[0], codes) and torch.equal(only.mx[1], scales)


def test_leading_axes_empty_rows_and_in_place_values():
    m = mok()
    x, r, w = _cuda(*_inputs(12, 64, "bf16", "bf16", "bf16"))
    flat = m.rms_norm(x, w, residual=r, mxfp8=True)
    cube = m.rms_norm(x.view(3, 4, 64), w, residual=r.view(3, 4, 64), mxfp8=True)
    assert cube.y.shape == (3, 4, 64) and cube.rstd.shape == (3, 4) and cube.mx[1].shape == (3, 4, 2)
    assert torch.equal(cube.y.view(12, 64), flat.y) and torch.equal(cube.mx[0].view(12, 64), flat.mx[0])
    none = m.rms_norm(x[:0], w, residual=r[:0], mxfp8=True)
    assert none.y.shape == (0, 64) and none.mx[1].shape == (0, 2)
    g = m.rms_norm_backward(x[:0], r[:0], w, none.rstd)
    assert g["dx"].shape == (0, 64) and bool((g["d_weight"] == 0).all())


def test_rows_of_zeros_infinities_and_nan_stay_in_their_row():
    m = mok()
    x, r, w = _inputs(6, 256, "bf16", "bf16", "bf16")
    clean = m.rms_norm(*_cuda(x, w), residual=r.cuda(), mxfp8=True)
    x[1], r[1] = 0.0, 0.0
    x[2, 5] = float("nan")
    x[4, 200] = float("inf")
    out = m.rms_norm(*_cuda(x, w), residual=r.cuda(), eps=1e-6, mxfp8=True)
    torch.cuda.synchronize()
    assert bool((out.y[1] == 0).all()) and bool((out.mx[0][1] == 0).all()) and bool((out.mx[1][1] == 127).all())
    assert abs(out.rstd[1].item() - 1e3) < 1e-2
    assert bool(out.y[2].isnan().all()) and bool(out.y[4, 200].isnan()) and bool((out.y[4, :200] == 0).all())
    for row in (0, 3, 5):
        assert torch.equal(out.y[row], clean.y[row]) and torch.equal(out.mx[0][row], clean.mx[0][row])


@pytest.mark.parametrize("rows,H", ROWS_H)
@pytest.mark.parametrize("ht,wt,with_dh", [("bf16", "bf16", True), ("f32", "f32", True), ("f32", "bf16", False),
                                           ("bf16", "f32", False)])
def test_backward(rows, H, ht, wt, with_dh):
    m = mok()
    h, dh, w = _inputs(rows, H, ht, ht, wt, seed=3)
    dy = _inputs(rows, H, "bf16", "none", "bf16", seed=5)[0]
    rstd = _ref(h, None, w, 1e-6)[1].float()
    r = rstd.double()[:, None]
    xhat, g = h.double() * r, dy.double() * w.double()
    mean_abs = (g * xhat).abs().mean(-1, keepdim=True)
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if with_dh:
        dx = dx + dh.double()
    dw = (dy.double() * xhat).sum(0)
    a = _cuda(dy, h, w, rstd, dh if with_dh else None)
    out = m.rms_norm_backward(*a[:4], d_h=a[4], bf16_dx=True)
    size = r * (g.abs() + xhat.abs() * mean_abs) + (dh.double().abs() if with_dh else 0.0)
    _close(out["dx"], dx, F * size + (U * dx.abs() if ht == "bf16" else 0.0), "dx")
    if ht == "f32":
        assert torch.equal(out["dx_bf16"], out["dx"].to(BF16))
    # up to rows / 608 + 19 + 32 terms in sequence
    _close(out["d_weight"], dw, F * (dy.double() * xhat).abs().sum(0) + 1e-30, "d_weight")
    again = m.rms_norm_backward(*a[:4], d_h=a[4])
    assert torch.equal(again["dx"], out["dx"]) and torch.equal(again["d_weight"], out["d_weight"])


def test_backward_against_differences():
    """Central differences of the 64-bit forward: their own error is of the
    order of step^2 = 1e-8."""
    m = mok()
    rows, H, step = 3, 40, 1e-4
    x, r, w = _inputs(rows, H, "f32", "f32", "f32", seed=9)
    dy = _inputs(rows, H, "bf16", "none", "bf16", seed=10)[0]
    out = m.rms_norm(*_cuda(x, w), residual=r.cuda(), eps=1e-5)
    g = m.rms_norm_backward(dy.cuda(), out.h, w.cuda(), out.rstd)

    def loss(x64, w64):
        h = x64 + r.double()
        return (dy.double() * h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-5) * w64).sum()

    x64, w64 = x.double(), w.double()
    num_x, num_w = torch.zeros_like(x64), torch.zeros_like(w64)
    for i in range(rows):
        for j in range(H):
            d = torch.zeros_like(x64)
            d[i, j] = step
            num_x[i, j] = (loss(x64 + d, w64) - loss(x64 - d, w64)) / (2 * step)
    for j in range(H):
        d = torch.zeros_like(w64)
        d[j] = step
        num_w[j] = (loss(x64, w64 + d) - loss(x64, w64 - d)) / (2 * step)
    assert (g["dx"].double().cpu() - num_x).abs().max() < 1e-5 * num_x.abs().max()
    assert (g["d_weight"].double().cpu() - num_w).abs().max() < 1e-5 * num_w.abs().max()


def test_more_elements_than_32_bits_of_bytes():
    """Rows whose byte offsets pass 2^32."""
    m = mok()
    rows, H = 270000, 8192
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    x = torch.zeros(rows, H, dtype=BF16, device="cuda")
    x[-1] = torch.arange(H, device="cuda").to(BF16) / H - 0.4
    w = torch.ones(H, dtype=BF16, device="cuda")
    out = m.rms_norm(x, w, bf16=True, mxfp8=True)
    one = m.rms_norm(x[-1:].clone(), w, bf16=True, mxfp8=True)
    assert torch.equal(out.y[-1:], one.y) and torch.equal(out.mx[0][-1:], one.mx[0])
    assert torch.equal(out.mx[1][-1:], one.mx[1]) and bool((out.y[-2] == 0).all())
    g = m.rms_norm_backward(x, x, w, out.rstd)
    g1 = m.rms_norm_backward(x[-1:].clone(), x[-1:].clone(), w, one.rstd)
    assert torch.equal(g["dx"][-1:], g1["dx"])


@pytest.mark.parametrize("shape", [(1, 1), (1, 31), (1, 100), (1, 4097), (3, 32), (5, 96), (17, 7168)])
def test_dequantize_every_code_and_tail(shape):
    m = mok()
    rng = np.random.default_rng(shape[1])
    rows, K = shape
    codes = rng.integers(0, 256, size=shape, dtype=np.uint8)
    codes[(codes & 127) == 127] = 5                      # NaN codes apart
    scales = rng.integers(90, 160, size=(rows, (K + 31) // 32), dtype=np.uint8)
    got = m.mxfp8_dequantize(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()).double().cpu().numpy()
    x = codes.astype(np.int64)
    e, f = (x >> 3) & 15, (x & 7).astype(np.float64)
    mag = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    want = np.where(x >= 128, -mag, mag) * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, axis=1)[:, :K]
    assert np.array_equal(got, want)


def test_dequantize_inverts_the_quantiser():
    m = mok()
    x = (torch.randn(37, 320, generator=torch.Generator().manual_seed(1)) * 3).to(BF16)
    codes, scales = m.mxfp8_quantize(x.cuda())
    got = m.mxfp8_dequantize(codes, scales).double().cpu().numpy()
    assert np.array_equal(got, oracle.mxfp8_roundtrip(x.double().numpy()))


def test_another_stream_gives_the_same():
    m = mok()
    x, r, w = _cuda(*_inputs(512, 2048, "bf16", "bf16", "bf16"))
    here = m.rms_norm(x, w, residual=r, mxfp8=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    there = m.rms_norm(x, w, residual=r, mxfp8=True, stream=s)
    g = m.rms_norm_backward(x, there.h, w, there.rstd, d_h=r, stream=s)
    s.synchronize()
    assert torch.equal(there.y, here.y) and torch.equal(there.mx[0], here.mx[0])
    assert torch.equal(g["dx"], m.rms_norm_backward(x, here.h, w, here.rstd, d_h=r)["dx"])


def test_refusals():
    m = mok()
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    rstd = torch.ones(4, device="cuda")
    bad = [lambda: m.rms_norm(x.cpu(), w), lambda: m.rms_norm(x.half(), w), lambda: m.rms_norm(x.t(), w),
           lambda: m.rms_norm(x, w[:32]), lambda: m.rms_norm(x, w, residual=x[:2]),
           lambda: m.rms_norm(x, w, bf16=False), lambda: m.rms_norm(x[:, :40].contiguous(), w[:40], mxfp8=True),
           lambda: m.rms_norm_backward(x, x, w, rstd[:3]), lambda: m.rms_norm_backward(x.float(), x, w, rstd),
           lambda: m.rms_norm_backward(x, x, w, rstd, d_h=x.float()), lambda: m.mxfp8_dequantize(x, x),
           lambda: m.mxfp8_dequantize(x.to(torch.uint8), torch.zeros(4, 3, dtype=torch.uint8, device="cuda"))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"case {i} was taken")
    wide = torch.zeros(1, 32776, dtype=BF16, device="cuda")
    with pytest.raises(m.MokError):
        m.rms_norm(wide, wide[0])
    with pytest.raises(m.MokError):
        m.rms_norm(x, w, eps=float("nan"))
    odd = torch.zeros(65, dtype=BF16, device="cuda")[1:]      # not 16-byte aligned
    with pytest.raises(m.MokError):
        m.rms_norm(x, odd)
    with pytest.raises(m.MokError):                            # K % 32 != 0 over several rows
        m.mxfp8_dequantize(torch.zeros(2, 40, dtype=torch.uint8, device="cuda"),
                           torch.zeros(2, 2, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("scale", [1e17, 1e13, 1e11, 1e-11, 1e-15, 1e-18])
@pytest.mark.parametrize("rows,H", [(40, 256), (9, 512), (130, 2048), (64, 4096), (2, 8200), (3, 16384), (2, 17), (2, 4097)])
@pytest.mark.parametrize("ht", ["bf16", "f32"])
def test_backward_of_rows_of_any_size(rows, H, ht, scale):
    """Rows over the range that the forward takes (their squares fit 32 bits),
    eps = 0 where they are small: the usual bound."""
    m = mok()
    h, dh, w = _inputs(rows, H, ht, ht, "bf16", seed=13)
    h = (h.double() * scale).to(TYPES[ht])
    dy = _inputs(rows, H, "bf16", "none", "bf16", seed=15)[0]
    out = m.rms_norm(h.cuda(), w.cuda(), eps=0.0 if scale < 1 else 1e-6)
    _close(out.rstd, _ref(h, None, w, 0.0)[1], F * _ref(h, None, w, 0.0)[1], "rstd")
    rstd = out.rstd.cpu()
    r = rstd.double()[:, None]
    dh = (dh.double() / scale).to(TYPES[ht])
    xhat, g = h.double() * r, dy.double() * w.double()
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True)) + dh.double()
    got = m.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), out.rstd, d_h=dh.cuda())
    size = r * (g.abs() + xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True)) + dh.double().abs()
    _close(got["dx"], dx, F * size + (U * dx.abs() if ht == "bf16" else 0.0), "dx")
    _close(got["d_weight"], (dy.double() * xhat).sum(0), F * (dy.double() * xhat).abs().sum(0) + 1e-30, "d_weight")


@pytest.mark.parametrize("rows,H", [(7, 40), (33, 256), (9, 512), (130, 2048), (3, 4104), (2, 8200), (2, 17), (2, 4097)])
@pytest.mark.parametrize("with_dh", [True, False])
def test_backward_in_fp32_of_a_bf16_stream(rows, H, with_dh):
    """dx_f32 is the value that dx is the rounding of."""
    m = mok()
    h, dh, w = _inputs(rows, H, "bf16", "bf16", "bf16", seed=23)
    dy = _inputs(rows, H, "bf16", "none", "bf16", seed=25)[0]
    rstd = _ref(h, None, w, 1e-6)[1].float()
    a = _cuda(dy, h, w, rstd, dh if with_dh else None)
    out = m.rms_norm_backward(*a[:4], d_h=a[4], f32_dx=True)
    plain = m.rms_norm_backward(*a[:4], d_h=a[4], bf16_dx=True)
    assert set(plain) == {"dx", "d_weight"} and out["dx_f32"].dtype == F32
    assert torch.equal(out["dx_f32"].to(BF16), out["dx"]) and torch.equal(out["dx"], plain["dx"])
    r = rstd.double()[:, None]
    xhat, g = h.double() * r, dy.double() * w.double()
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True)) + (dh.double() if with_dh else 0.0)
    size = r * (g.abs() + xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True)) + (dh.double().abs() if with_dh else 0.0)
    _close(out["dx_f32"], dx, F * size, "dx_f32")


def test_an_fp32_x_beside_a_bf16_stream_gets_an_unrounded_gradient():
    """Under autograd the gradient of x is fp32, as x is: within fp32's error of
    the 64-bit gradient at the stream as it was stored, where the stream's own
    gradient is rounded to bf16."""
    mok()
    from mixture_experts_layer_mok_gb300.autograd import rms_norm

    x, r, w = _inputs(37, 96, "f32", "bf16", "bf16", seed=31)
    dy, dh = (_inputs(37, 96, "bf16", "none", "bf16", seed=s)[0] for s in (33, 35))
    gx, gr, gw = (t.cuda().requires_grad_() for t in (x, r, w))
    y, h = rms_norm(gx, gw, gr, eps=1e-5)
    torch.autograd.backward([y, h], [dy.cuda(), dh.cuda()])
    rstd = _ref(x, r, w, 1e-5)[1][:, None]
    xhat, g = h.detach().double().cpu() * rstd, dy.double() * w.double()
    dx = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True)) + dh.double()
    size = rstd * (g.abs() + xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True)) + dh.double().abs()
    assert gx.grad.dtype == F32 and gr.grad.dtype == BF16
    _close(gx.grad, dx, F * size, "dx")
    assert torch.equal(gx.grad.to(BF16), gr.grad)


IN_PLACE = [(7, 40), (33, 256), (9, 512), (1300, 64), (130, 2048), (1217, 640), (3, 4104), (700, 8200), (2, 32768), (2, 17), (2, 4097)]


def _ptr(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("rows,H", IN_PLACE)
@pytest.mark.parametrize("xt,rt,place", [("bf16", "bf16", "residual"), ("bf16", "f32", "residual"), ("f32", "f32", "x"),
                                         ("bf16", "bf16", "x")])
def test_the_stream_may_be_written_in_place(rows, H, xt, rt, place):
    """h in the residual's or x's place, through the C ABI: every bit as apart."""
    m = mok()
    from mixture_experts_layer_mok_gb300 import _lib

    x, r, w = _cuda(*_inputs(rows, H, xt, rt, "bf16", seed=41))
    want = m.rms_norm(x, w, residual=r, eps=1e-5)
    h = r if place == "residual" else x
    y, rstd = torch.empty_like(want.y), torch.empty_like(want.rstd)
    code = {"bf16": _lib.MOK_DTYPE_BF16, "f32": _lib.MOK_DTYPE_F32}
    st = _lib.load().mok_rms_norm(_ptr(x), code[xt], _ptr(r), code[rt], _ptr(w), 0, rows, H, 1e-5, _ptr(h), _ptr(y), None, None,
                                  _ptr(rstd), torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(h, want.h) and torch.equal(y, want.y) and torch.equal(rstd, want.rstd)


@pytest.mark.parametrize("rows,H", IN_PLACE)
@pytest.mark.parametrize("ht", ["bf16", "f32"])
def test_the_streams_gradient_may_be_written_in_place(rows, H, ht):
    """dx in dh's place, through the C ABI: every bit as apart."""
    m = mok()
    from mixture_experts_layer_mok_gb300 import _lib

    h, dh, w = _cuda(*_inputs(rows, H, ht, ht, "bf16", seed=43))
    dy = _inputs(rows, H, "bf16", "none", "bf16", seed=45)[0].cuda()
    rstd = torch.rsqrt(h.float().square().mean(-1) + 1e-6)
    want = m.rms_norm_backward(dy, h, w, rstd, d_h=dh, bf16_dx=True)
    lib = _lib.load()
    n = lib.mok_rms_norm_bwd_workspace_bytes(rows, H)
    ws, dw = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(want["d_weight"])
    d16 = torch.empty_like(want["dx_bf16"]) if ht == "f32" else None
    st = lib.mok_rms_norm_bwd(_ptr(dy), _ptr(h), int(ht == "f32"), _ptr(w), 0, _ptr(rstd), _ptr(dh), rows, H, _ptr(dh), _ptr(d16),
                              _ptr(dw), _ptr(ws), n, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(dh, want["dx"]) and torch.equal(dw, want["d_weight"])
    assert d16 is None or torch.equal(d16, want["dx_bf16"])
