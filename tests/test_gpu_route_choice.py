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
