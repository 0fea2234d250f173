"""4-bit weights: the quantiser, the layout and the reader exactly, the products
against 64-bit restatements.

Error bounds: the weights' integers times bf16 activations are exact in fp32;
a sum over K is a chain of K / 16 tensor-core steps (each good to 2^-23 of the
terms so far), K / group scalings and 8 parts: within (K / 16 + K / group + 16)
2^-23 of the terms' sizes.  A rounding to bf16 adds 2^-8 of the value, an
activation 4e-6 and its slope, up to 1.13."""
import pytest
import torch

from tests.gpu_util import mok
from tests.test_gpu_linear import U, act64

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
T = {"bf16": BF16, "f32": F32}


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _rand(g, *shape, dtype=BF16, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _weight(g, lead, N, K, group, zeros):
    """Codes and scales as they come from elsewhere, and the values in 64 bits."""
    codes = torch.randint(0, 256, (*lead, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(*lead, N, K // group, generator=g, device="cuda") + 0.5).div(K ** 0.5).to(BF16)
    zero = torch.randint(0, 16, scales.shape, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(*lead, N, K).double()
    q = q - (8.0 if zero is None else zero.double().repeat_interleave(group, -1))
    return codes, scales, zero, q * scales.double().repeat_interleave(group, -1)


@pytest.mark.parametrize("lead,N,K,group", [((), 1, 32, 32), ((), 16, 128, 128), ((), 7, 192, 64), ((), 100, 96, 32), ((3,), 17, 320, 64),
                                            ((2,), 33, 256, 32), ((), 130, 384, 128), ((5,), 8, 2048, 128)])
@pytest.mark.parametrize("zeros", [False, True])
def test_pack_and_dequantize_are_exact(lead, N, K, group, zeros):
    m = mok()
    codes, scales, zero, values = _weight(_gen(N + K), lead, N, K, group, zeros)
    w = m.int4_pack(codes, scales, zero)
    assert w.shape == (*lead, N, K) and w.group == group
    assert torch.equal(m.int4_dequantize(w), values.to(F32).to(BF16))   # 5 bits x 8 bits: exact in fp32, rounded once


@pytest.mark.parametrize("lead,N,K,group", [((), 1, 32, 32), ((), 24, 128, 128), ((), 7, 192, 64), ((3,), 17, 320, 32), ((2,), 50, 1024, 64)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_rounds_to_nearest(lead, N, K, group, zeros, dtype):
    m = mok()
    g = _gen(N * K)
    w = _rand(g, *lead, N, K, dtype=dtype, std=0.05)
    w[..., 0, :group] = 0.0                       # a group of nothing
    if N > 1:
        w[..., 1, :group] = w[..., 1, :group].abs() + 0.5   # all of one sign, far from 0
    got = m.int4_quantize(w, group, zeros)
    v = w.float().cpu().reshape(*lead, N, K // group, group)
    lo, hi = v.amin(-1).clamp(max=0.0), v.amax(-1).clamp(min=0.0)
    scale = (((hi - lo) / 15.0) if zeros else torch.maximum(-lo, hi) / 7.0).to(BF16)
    s = scale.float()
    on = s > 0
    safe = torch.where(on, s, torch.ones_like(s))
    zero = torch.where(on, torch.round(-lo / safe).clamp(0, 15), torch.zeros_like(s)) if zeros else torch.full_like(s, 8.0)
    q = torch.where(on[..., None], (torch.round(v / safe[..., None]) + zero[..., None]).clamp(0, 15), zero[..., None])
    value = ((q - zero[..., None]) * s[..., None]).to(BF16).reshape(*lead, N, K)
    assert torch.equal(m.int4_dequantize(got).cpu(), value)
    packed = q.reshape(*lead, N, K).to(torch.uint8)
    ref = m.int4_pack((packed[..., 0::2] | packed[..., 1::2] << 4).contiguous().cuda(), scale.cuda(),
                      zero.to(torch.uint8).cuda() if zeros else None)
    assert torch.equal(m.int4_dequantize(ref), m.int4_dequantize(got))
    # off by half a step at most, and a bf16 scale's rounding of the furthest value
    step = s.double().repeat_interleave(group, -1).reshape(*lead, N, K)
    assert ((w.double().cpu() - value.double()).abs() <= 0.5 * step + 2.0 ** -7 * w.double().cpu().abs() + step * 2.0 ** -4).all()


def _bound(K, group, size):
    return (K / 16 + K / group + 16) * 2.0 ** -23 * size


def _check(y, z64, size, act, K, group, out):
    y64 = act64(z64, act)
    bound = 1.13 * _bound(K, group, size) + 4e-6 * (z64.abs() + y64.abs()) + (U * y64.abs() if out == BF16 else 0.0)
    err = (y.double() - y64).abs()
    assert not torch.isnan(err).any()
    worst = (err / bound.clamp(min=1e-30)).max().item() if err.numel() else 0.0
    assert worst <= 1.0, worst


ONE = [(1, 8, 32, 32), (1, 7168, 2048, 128), (1, 1000, 4096, 64), (2, 17, 96, 32), (3, 1, 128, 64), (7, 264, 160, 32), (8, 513, 1024, 128),
       (9, 40, 384, 128), (16, 2056, 512, 64), (17, 136, 7168, 128), (31, 33, 224, 32), (32, 4096, 256, 128), (33, 100, 640, 64),
       (64, 520, 1152, 128), (100, 24, 192, 64), (1000, 72, 320, 32)]
# rows of w enough for the variant whose warps share x, and many rows of both
WIDE = [(1, 39169, 96, 32), (5, 39168, 640, 128), (1, 77824, 96, 32), (6, 78001, 320, 64), (3, 77840, 256, 128), (8, 80000, 160, 32),
        (130, 4200, 2048, 128), (9, 30001, 320, 64), (33, 8200, 1056, 32), (20, 1100, 8192, 128), (64, 520, 16384, 32), (12, 41000, 192, 64), (16, 39200, 1024, 32), (31, 40007, 704, 64), (33, 30000, 128, 128),
        (64, 39168, 256, 64)]


@pytest.mark.parametrize("rows,N,K,group", ONE + WIDE)
@pytest.mark.parametrize("zeros,bias,act,out", [(False, None, "none", BF16), (True, F32, "gelu", F32), (True, BF16, "silu", BF16),
                                                (False, F32, "relu", F32), (False, None, "gelu_tanh", BF16)])
def test_one_matrix(rows, N, K, group, zeros, bias, act, out):
    m = mok()
    g = _gen(rows + N + K)
    codes, scales, zero, values = _weight(g, (), N, K, group, zeros)
    w = m.int4_pack(codes, scales, zero)
    x = _rand(g, rows, K)
    b = None if bias is None else _rand(g, N, dtype=bias)
    y = m.int4_linear(x, w, bias=b, activation=act, out_dtype=out)
    assert y.dtype == out and y.shape == (rows, N)
    z = x.double() @ values.t() + (0.0 if b is None else b.double())
    size = x.double().abs() @ (values.abs() + scales.double().repeat_interleave(group, -1)).t() + (0.0 if b is None else b.double().abs())
    _check(y, z, size, act, K, group, out)
    assert torch.equal(m.int4_linear(x, w, bias=b, activation=act, out_dtype=out), y)


EXPERTS = [(1, 1, 2, 8, 32, 32), (1, 8, 256, 72, 256, 32), (3, 2, 5, 40, 384, 128), (16, 6, 64, 136, 320, 64), (64, 8, 128, 24, 256, 128),
           (40, 3, 4, 100, 512, 64), (200, 1, 2, 520, 128, 128), (1, 6, 8, 2056, 2048, 128), (4, 4, 8, 72, 256, 64), (12, 8, 9, 33, 320, 32),
           (30, 8, 40, 136, 192, 64), (100, 8, 100, 17, 256, 128)]


@pytest.mark.parametrize("rows,k,E,N,K,group", EXPERTS)
@pytest.mark.parametrize("zeros,bias,act,out", [(False, None, "none", BF16), (True, F32, "silu", F32), (True, BF16, "gelu", BF16)])
def test_experts(rows, k, E, N, K, group, zeros, bias, act, out):
    m = mok()
    g = _gen(rows + N + K + E)
    codes, scales, zero, values = _weight(g, (E,), N, K, group, zeros)
    w = m.int4_pack(codes, scales, zero)
    x = _rand(g, rows, K)
    ids = torch.rand(rows, E, generator=g, device="cuda").topk(k, 1).indices.contiguous()
    if rows > 2:
        ids[1] = ids[0, 0]                     # one expert for all of a token's choices
        ids[2, -1] = -1                        # and none
    b = None if bias is None else _rand(g, E, N, dtype=bias)
    y = m.int4_linear(x, w, bias=b, activation=act, experts=ids, out_dtype=out)
    assert y.shape == (rows, k, N) and m.linear_status() == 0
    z, size = torch.zeros(rows, k, N, dtype=F64, device="cuda"), torch.zeros(rows, k, N, dtype=F64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        z[t, j] = x[t].double() @ values[e].t() + (0.0 if b is None else b[e].double())
        size[t, j] = x[t].double().abs() @ (values[e].abs() + scales[e].double().repeat_interleave(group, -1)).t() + (
            0.0 if b is None else b[e].double().abs())
    _check(y, z, size, act, K, group, out)
    assert (y[ids == -1] == 0).all()
    each = x[:, None].expand(rows, k, K).contiguous()      # a row of x for each choice: the same sums
    assert torch.equal(m.int4_linear(each, w, bias=b, activation=act, experts=ids, out_dtype=out), y)


@pytest.mark.parametrize("rows", [1, 3, 30])
def test_ids_out_of_range_give_zeros_and_the_status(rows):
    m = mok()
    from mixture_experts_layer_mok_gb300 import _lib

    g = _gen(3)
    codes, scales, zero, values = _weight(g, (4,), 24, 128, 64, False)
    w = m.int4_pack(codes, scales, zero)
    x = _rand(g, rows, 128)
    ids = torch.tensor([[0, 4], [-7, 1], [1 << 40, 2]] * 10, device="cuda")[:rows].contiguous()
    y = m.int4_linear(x, w, experts=ids)
    assert m.linear_status() == _lib.MOK_ERR_INDEX and m.linear_status() == 0
    ok = (ids >= 0) & (ids < 4)
    assert (y[~ok] == 0).all()
    clean = m.int4_linear(x, w, experts=torch.where(ok, ids, torch.full_like(ids, -1)))
    assert torch.equal(clean, y) and m.linear_status() == 0


def test_no_rows_nan_rows_and_shapes():
    m = mok()
    g = _gen(4)
    codes, scales, zero, values = _weight(g, (), 40, 256, 128, True)
    w = m.int4_pack(codes, scales, zero)
    assert m.int4_linear(torch.empty(0, 256, dtype=BF16, device="cuda"), w).shape == (0, 40)
    x = _rand(g, 6, 256)
    y = m.int4_linear(x, w)
    bad = x.clone()
    bad[2, 5], bad[4, 7] = float("nan"), float("inf")
    r = m.int4_linear(bad, w)
    keep = [0, 1, 3, 5]
    assert torch.equal(r[keep], y[keep]) and torch.isnan(r[2]).all() and not torch.isfinite(r[4]).any()
    assert torch.equal(m.int4_linear(x.view(2, 3, 256), w).view(6, 40), y)
    assert torch.equal(m.int4_linear(x[0], w), m.int4_linear(x[:1].clone(), w)[0])
    codes, scales, zero, values = _weight(g, (3,), 40, 256, 128, True)
    w3 = m.int4_pack(codes, scales, zero)
    one = m.int4_linear(x[0].clone(), w3, experts=torch.tensor([2, 0], device="cuda"))
    assert one.shape == (2, 40)
    assert torch.equal(one, m.int4_linear(x[:1].clone(), w3, experts=torch.tensor([[2, 0]], device="cuda"))[0])


def test_streams_and_graph():
    m = mok()
    g = _gen(5)
    codes, scales, zero, values = _weight(g, (8,), 136, 512, 64, True)
    w = m.int4_pack(codes, scales, zero)
    x, ids = _rand(g, 2, 512), torch.tensor([[0, 1], [2, 3]], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = m.int4_linear(x, w, experts=ids, stream=side)
    side.synchronize()
    assert torch.equal(y, m.int4_linear(x, w, experts=ids))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.int4_linear(x, w, experts=ids, activation="silu")
    for seed in range(3):
        x.copy_(_rand(g, 2, 512))
        ids.copy_(torch.randint(0, 8, (2, 2), generator=g, device="cuda"))
        graph.replay()
        assert torch.equal(out, m.int4_linear(x, w, experts=ids, activation="silu"))


def test_large_weight():
    """Codes beyond 2^31 bytes: the last expert's offsets pass 32 bits."""
    m = mok()
    g = _gen(6)
    E, N, K = 160, 4096, 8192
    codes = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    codes[-1] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.full((E, N, K // 128), 2.0 ** -6, dtype=BF16, device="cuda")
    w = m.int4_pack(codes, scales)
    x = _rand(g, 1, K)
    y = m.int4_linear(x, w, experts=torch.tensor([[E - 1, 0]], device="cuda"))
    one = m.int4_pack(codes[-1].clone(), scales[-1].clone())
    v = m.int4_dequantize(one).double()      # (codes times a power of two: exact in bf16)
    ref = (x.double() @ v.t())[0]
    size = (x.double().abs() @ (v.abs() + 2.0 ** -6).t())[0]
    assert ((y[0, 0].double() - ref).abs() <= U * ref.abs() + _bound(K, 128, size)).all()
    zero = x.double().sum() * -8 * 2.0 ** -6
    assert (y[0, 1].double() - zero).abs().max() <= U * zero.abs() + _bound(K, 128, x.double().abs().sum() * 0.125)
    assert torch.equal(m.int4_dequantize(w)[-1], m.int4_dequantize(one))


def test_refusals():
    m = mok()
    g = _gen(7)
    codes, scales, zero, values = _weight(g, (), 16, 128, 64, True)
    w = m.int4_pack(codes, scales, zero)
    x, ids = _rand(g, 2, 128), torch.zeros(2, 1, dtype=torch.int64, device="cuda")
    for call in (lambda: m.int4_pack(codes, scales[:, :1].expand(16, 3).contiguous()), lambda: m.int4_pack(codes, scales.float()),
                 lambda: m.int4_pack(codes, scales, zero[:8]), lambda: m.int4_pack(codes[:, ::2], scales),
                 lambda: m.int4_pack(codes[0], scales[0]), lambda: m.int4_quantize(x, 48), lambda: m.int4_quantize(x[:, :96].contiguous(), 64),
                 lambda: m.int4_quantize(x.half(), 64), lambda: m.int4_linear(x[:, :64].contiguous(), w), lambda: m.int4_linear(x, values),
                 lambda: m.int4_linear(x, w, experts=ids), lambda: m.int4_linear(x, w, activation="swish"),
                 lambda: m.int4_linear(x, w, out_dtype=torch.float16), lambda: m.int4_linear(x.float(), w),
                 lambda: m.int4_linear(x, w, bias=torch.ones(8, device="cuda")), lambda: m.int4_linear(x.cpu(), w),
                 lambda: m.int4_linear(torch.zeros(70000, 128, dtype=BF16, device="cuda"), w)):
        with pytest.raises(ValueError):
            call()
    codes, scales, zero, values = _weight(g, (2,), 16, 128, 64, False)
    w = m.int4_pack(codes, scales)
    for call in (lambda: m.int4_linear(x, w), lambda: m.int4_linear(x, w, experts=ids[:1]), lambda: m.int4_linear(x, w, experts=ids.int()),
                 lambda: m.int4_linear(x, w, experts=ids, bias=torch.ones(16, device="cuda"))):
        with pytest.raises(ValueError):
            call()
