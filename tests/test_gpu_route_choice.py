"""The router's choice where it goes by a selection bias: by the scores' own
errors, where scores meet, and in every way that tokens are dealt to warps."""
import pytest
import torch

from tests.gpu_util import mok

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24


@pytest.mark.parametrize("E,k", [(8, 2), (40, 5), (100, 6), (256, 8), (512, 9), (1000, 12)])
@pytest.mark.parametrize("T", [1, 3000])
def test_softmax_scores_of_a_choice_are_the_exact_ones(E, k, T):
    """Scores of e^-80 and less, whose exponent 80 log2 e a 32-bit product rounds by
    44 u of the result, beside biases that bring their sums to within 64 u of one
    another.  The differences to the largest logit are exact and the sum of all
    exponentials is 1, so that a score has expf's error, 2 u of what is half
    the sum, and the sum with the bias u: two of them are at most 4 u apart from
    where they should be."""
    m = mok()
    g = torch.Generator("cuda").manual_seed(E + T)
    for _ in range(50 if T == 1 else 3):
        x = torch.zeros(E, device="cuda")
        x[1:] = -80 - torch.randint(0, 256, (E - 1,), device="cuda", generator=g) / 256
        s = torch.softmax(x.double(), 0)
        c = 2 * s[1:].max()
        bias = (c - s + c * 64 * U * torch.rand(E, device="cuda", generator=g, dtype=F64)).float()
        bias[0] = -2.0
        by = s + bias.double()
        experts = m.route(x.expand(T, E).contiguous(), k, bias=bias).experts
        assert (experts == experts[0]).all()
        got, top = by[experts[0]], by.topk(k).values
        assert ((top - got) <= 4 * U * c).all(), ((top - got) / c / U).max().item()


# (E, k): every number of lanes and of logits to a lane, few picks and more than lanes or 32
WIDTHS = [(3, 3), (8, 3), (32, 32), (33, 4), (40, 5), (64, 12), (65, 7), (96, 6), (128, 40), (200, 8), (256, 20), (256, 33), (384, 9),
          (512, 64), (777, 12), (1024, 8), (1024, 64)]


def _spread(T, E, seed):
    """Whole numbers from -300 to 300, so that scores saturate or underflow, or
    differ by far more than their errors; masked and equal ones among them."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randint(-300, 301, (T, E), device="cuda", generator=g).float()
    x[torch.rand(T, E, device="cuda", generator=g) < 0.1] = -float("inf")
    x[0] = 7.0
    if T > 2:
        x[1] = -float("inf")
        x[2, E // 2] = float("nan")
    return x


def _logit_order(x, k):
    """Largest logits, NaN before them, lowest index of equal ones."""
    return torch.sort(torch.nan_to_num(x, nan=1e30, neginf=-1e30), dim=1, descending=True, stable=True).indices[:, :k]


@pytest.mark.parametrize("E,k", WIDTHS)
@pytest.mark.parametrize("T", [5, 3000])     # a token to a round of a warp, and several
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_bias_for_all_experts_changes_no_choice(E, k, T, score, dtype):
    m = mok()
    x = _spread(T, E, E + k).to(dtype)       # (up to 300: bf16 rounds beyond 256 to even numbers)
    want = _logit_order(x.float(), k)
    plain = m.route(x, k, score=score)
    assert torch.equal(plain.experts, want)
    for level in (0.0, 0.25, -3.0):
        r = m.route(x, k, score=score, bias=torch.full((E,), level, device="cuda"), balance=True)
        assert torch.equal(r.experts, want)
        assert torch.equal(r.counts.long(), torch.bincount(want.flatten(), minlength=E))


@pytest.mark.parametrize("E,k", WIDTHS)
@pytest.mark.parametrize("T", [5, 3000])
def test_equal_sums_go_by_logit_and_then_by_index(E, k, T):
    """Sigmoids of 20 and more are 1 in 32 bits; biases of three values."""
    m = mok()
    g = torch.Generator("cuda").manual_seed(E * k)
    x = torch.randint(20, 40, (T, E), device="cuda", generator=g).float()
    bias = torch.randint(-1, 2, (E,), device="cuda", generator=g) / 4
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(bias[order], dim=1, descending=True, stable=True).indices)[:, :k]
    r = m.route(x, k, score="sigmoid", bias=bias)
    assert torch.equal(r.experts, order)
    assert (r.weights - 1 / k).abs().max().item() <= 8 * U / k


@pytest.mark.parametrize("E,k", [(8, 8), (40, 38), (96, 32), (96, 40), (200, 64), (1000, 33)])
@pytest.mark.parametrize("T", [3, 2600])
def test_biases_that_open_and_close_experts(E, k, T):
    """+inf before all, -inf behind all but masked logits; each of them in the logits' order."""
    m = mok()
    g = torch.Generator("cuda").manual_seed(E)
    x = torch.randint(20, 40, (T, E), device="cuda", generator=g).float()
    x[:, ::5] = -float("inf")
    bias = torch.zeros(E, device="cuda")
    bias[3::4], bias[1::3] = float("inf"), -float("inf")
    level = torch.where(torch.isinf(x), torch.full_like(x, -2.0), torch.sign(bias).expand_as(x))
    order = torch.sort(torch.nan_to_num(x, neginf=-1.0), dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(level.gather(1, order), dim=1, descending=True, stable=True).indices)[:, :k]
    assert torch.equal(m.route(x, k, score="sigmoid", bias=bias).experts, order)
