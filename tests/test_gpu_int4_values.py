"""4-bit weights of values at the ends of their types: what is not finite, ranges
beyond the largest number, and zeros with more than four bits."""
import pytest
import torch

from tests.gpu_util import mok

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _weights(lead, N, K, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*lead, N, K, generator=g, device="cuda") * 0.05).to(dtype)


@pytest.mark.parametrize("lead,N,K,group", [((), 3, 32, 32), ((), 24, 384, 128), ((3,), 17, 320, 64), ((2,), 33, 224, 32)])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_group_with_a_value_that_is_not_finite_is_nan(lead, N, K, group, zeros, dtype):
    m = mok()
    w = _weights(lead, N, K, dtype, N + K)
    clean = m.int4_dequantize(m.int4_quantize(w, group, zeros))
    inf, nan = float("inf"), float("nan")
    rows = w.view(-1, K)
    at = [(0, 0, nan), (1, K - 1, inf), (2, group // 2, -inf)]
    if N > 16:
        at += [(16, K - group, -nan), (N - 1, 7, nan), (N - 1, 8, inf)]
    hit = torch.zeros(rows.shape[0], K // group, dtype=torch.bool, device="cuda")
    for r, k, v in at:
        rows[r, k] = v
        hit[r, k // group] = True
    rows[-1, K - group:] = nan                       # nothing else in the group
    hit[-1, -1] = True
    got = m.int4_dequantize(m.int4_quantize(w, group, zeros))
    hit = hit.repeat_interleave(group, -1).view(w.shape)
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("rows,N,K", [(1, 100, 512), (30, 100, 512), (5, 39200, 96), (20, 8200, 1056)])
@pytest.mark.parametrize("zeros", [False, True])
def test_products_show_it_in_that_row_alone(rows, N, K, zeros):
    m = mok()
    w = _weights((), N, K, BF16, 1)
    x = _weights((), rows, K, BF16, 2)
    clean = m.int4_linear(x, m.int4_quantize(w, 32, zeros))
    w[N // 2, K // 2] = float("nan")
    y = m.int4_linear(x, m.int4_quantize(w, 32, zeros))
    assert torch.isnan(y[:, N // 2]).all()
    y[:, N // 2] = clean[:, N // 2]
    assert torch.equal(y, clean)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_range_beyond_the_largest_number(group, dtype):
    """lo and hi of 3e38 each: hi - lo is not a number of 32 bits, a fifteenth of it is."""
    m = mok()
    g = torch.Generator("cuda").manual_seed(0)
    w = ((torch.rand(40, 256, generator=g, device="cuda") * 2 - 1) * 3e38).to(dtype)
    w[:, ::32], w[:, 1::32] = 3e38, -3e38
    v = w.double().view(40, -1, group)
    scale = ((v.amax(-1) - v.amin(-1)) / 15).float().to(BF16).double()
    got = m.int4_dequantize(m.int4_quantize(w, group, True)).double().view_as(v)
    # half a step for the value and half a step for the zero, a scale off by 2^-8 of itself over 15 steps, and bf16 values
    assert ((got - v).abs() <= scale[..., None] * (1 + 15 * 2.0 ** -8) + v.abs() * 2.0 ** -7).all()


def test_zeros_count_by_their_low_four_bits():
    m = mok()
    g = torch.Generator("cuda").manual_seed(0)
    codes = torch.randint(0, 256, (3, 20, 80), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(3, 20, 5, generator=g, device="cuda") + 0.5).to(BF16)
    zeros = torch.randint(0, 256, (3, 20, 5), generator=g, device="cuda", dtype=torch.uint8)
    assert torch.equal(m.int4_dequantize(m.int4_pack(codes, scales, zeros)), m.int4_dequantize(m.int4_pack(codes, scales, zeros & 15)))


@pytest.mark.parametrize("E,N,K", [(0, 24, 96), (0, 8200, 1056), (3, 40, 160), (66000, 1, 32)])
def test_as_many_rows_as_there_can_be(E, N, K):
    """65535 rows: of one matrix by both kernels, of few experts and of more experts
    than rows.  Rows, codes and scales are whole numbers and powers of two, so that
    the sums are exact."""
    m = mok()
    g = torch.Generator("cuda").manual_seed(N)
    k, rows = 3 if E else 1, 65535
    codes = torch.randint(0, 256, (E, N, K // 2) if E else (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.exp2(torch.randint(-3, 2, codes.shape[:-1] + (K // 32,), generator=g, device="cuda").float()).to(BF16)
    w = m.int4_pack(codes, scales)
    x = torch.randint(-2, 3, (rows // k, K), generator=g, device="cuda").to(BF16)
    values = m.int4_dequantize(w).float()      # (exact: four bits times a power of two)
    if not E:
        assert torch.equal(m.int4_linear(x, w, out_dtype=F32), x.float() @ values.t())
        return
    ids = torch.randint(-1, E, (rows // k, k), generator=g, device="cuda")
    y = m.int4_linear(x, w, experts=ids, out_dtype=F32)
    ref = torch.einsum("tknc,tc->tkn", values[ids.clamp(min=0)], x.float()) * (ids >= 0)[..., None]
    assert torch.equal(y, ref) and m.linear_status() == 0
