"""The balance loss's scores far from zero, and far below their row's largest:
their relative error does not grow with the distance. In steps U = 2^-24 (E = 2
and fp32 logits, so that sums are one addition and z - max is one rounding, of
an exact difference):
 e^v: the exponential instruction 4 (2^-22), its correction 1: 5.
 s = 1 / (1 + e^-z): 5, the addition 1, the reciprocal 2: 8.
 1 - s = e^-z s: where s is tiny 1 + 2 + 1 = 4; where it is 1, 5 + 3 + 1 = 9.
 p: the score, its sum (as far off as the larger score, and 1), the reciprocal
 2 and the product 1.
"""
import pytest
import torch

from tests import step_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

L = 4096


def relative(z, scoring, slopes):
    """Largest relative error of dlogits, an element 0 of a row, in steps U."""
    import chunked_lm_head_gemm_gb300 as lce
    c = torch.tensor(slopes, device="cuda")
    one = torch.ones((), device="cuda")
    got = lce.balance_backward(z, c, one, scoring).double()
    want = ref.balance_grad(z, c, 1.0, scoring, None)
    return float(((got - want) / want)[:, 0].abs().max()) / ref.U


def uniform(lo, hi, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(L, device="cuda", generator=g) * (hi - lo) + lo


@pytest.mark.parametrize("lo,hi,bound", [(-1, 0, 43), (-25, -15, 34),
                                         (-60, -50, 34), (-67, -57, 34)])
def test_sigmoid_scores_far_below_zero(lo, hi, bound):
    """p 8 + 8 + 4 = 20, slope 9 at most, two products; c - dot = 1 - p has 1
    and p / (1 - p) of p's: p is e^-3 / (1 + e^-3) far below, where it is 2,
    and at most 0.35 around zero, where it is 12."""
    require_gpu()
    z = uniform(lo, hi, 1)
    assert relative(torch.stack([z, z + 3], 1), "sigmoid",
                    [1.0, 0.0]) <= bound


@pytest.mark.parametrize("lo,hi", [(12, 22), (45, 55), (70, 80)])
def test_the_slope_of_sigmoid_scores_far_above_zero(lo, hi):
    """Both scores are 1, but for 2^-17 at most, and off by 1 + 2: p half of
    both, 3, and 1 + 2 + 1: 7; 1 - p, where p is a half, 7 and 1; slope 9, two
    products: 26."""
    require_gpu()
    z = uniform(lo, hi, 2)
    assert relative(torch.stack([z, z + 1], 1), "sigmoid", [1.0, 0.0]) <= 26


@pytest.mark.parametrize("lo,hi", [(-12, -2), (-40, -30), (-70, -60)])
def test_softmax_scores_far_below_the_largest(lo, hi):
    """The other score is 1: p 5 + 1 + 2 + 1, of which e^-2 of p's error comes
    back in the sum and in 1 - p, 1 each and its subtraction 1, one product:
    14."""
    require_gpu()
    z = uniform(lo, hi, 3)
    z = torch.stack([z, torch.zeros_like(z)], 1)
    assert relative(z, "softmax", [1.0, 0.0]) <= 14


@pytest.mark.parametrize("lo,hi,below", [(-18, -10, 65), (-30, -19, 60),
                                         (-50, -40, 40), (-69, -60, 25)])
def test_sigmoid_scores_far_below_a_small_one(lo, hi, below):
    """Scores below fp32's range that are e^-25 and less of the row's sum. The
    logits are multiples of 2^-10, whose differences are exact, so the bound is
    that of scores far below zero (relative to the largest they are 5, not 8,
    and half a step for s = e^z and 1 - s = 1)."""
    require_gpu()
    z = (uniform(lo, hi, 4) * 1024).round() / 1024
    assert relative(torch.stack([z - below, z], 1), "sigmoid",
                    [1.0, 0.0]) <= 34


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_logits_at_the_ends_of_the_range(scoring):
    """The lowest and highest values of fp32 and infinities: each row is what
    float64 gives for it."""
    import math

    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    most = torch.finfo(torch.float32).max
    values = [-math.inf, -most, -0.7 * most, -1e30, -200.0, -88.6, -88.4, 0.0,
              1.0, 87.0, 120.0, 1e30, 0.7 * most]
    if scoring == "sigmoid":
        values += [most, math.inf]
    z = torch.tensor([[a, b] for a in values for b in values], device="cuda")
    experts = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    p, _ = ref.probabilities(z.double(), scoring)
    for row, want in zip(z, p[:, 0].tolist()):
        loss, _, _ = lce.balance_forward(row[None], experts, scoring, 0.5)
        # E / (N K) = 2 times the coefficient; below fp32's range, 0
        assert abs(float(loss) - want) <= 40 * ref.U * want + 1.2e-38, \
            (row.tolist(), float(loss), want)
    c = torch.tensor([1.0, -1.0], device="cuda")
    one = torch.ones((), device="cuda")
    dz = lce.balance_backward(z, c, one, scoring)
    p, d = ref.probabilities(z.double(), scoring)
    want = ref.balance_grad(z, c, 1.0, scoring, None)
    # p, slope and dot each within 30 of themselves
    assert ((dz.double() - want).abs() <=
            60 * ref.U * p * d * (1 + p.sum(1, keepdim=True)) + 1e-37).all()
