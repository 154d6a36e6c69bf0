"""More of the gradient clipping on the GPU: norms that are not finite under an
infinite limit, and layouts against float64."""
import math

import pytest
import torch

from tests import step_ref as ref
from tests.gpu_util import require_gpu
from tests.test_gpu_grads import BF, F32, NORM, make, near

pytestmark = pytest.mark.gpu

SMALL, LARGE = [((1000,), F32), ((77,), BF)], [((700003,), F32), ((64,), BF)]


@pytest.mark.parametrize("shapes", [SMALL, LARGE], ids=["small", "large"])
@pytest.mark.parametrize("in_place", [True, False])
def test_a_norm_that_is_nan_under_no_limit(shapes, in_place):
    """NaN reaches every output whatever the limit."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    g = make(shapes)
    g[0][5] = math.nan
    outs = g if in_place else [torch.zeros_like(t) for t in g]
    norm = lce.clip_grad_norm(g, math.inf, grads_out=None if in_place else outs)
    assert math.isnan(float(norm))
    assert all(torch.isnan(t).all() for t in outs)
    g = make(shapes)
    lce.clip_grads(g, norm, math.inf)
    assert all(torch.isnan(t).all() for t in g)


@pytest.mark.parametrize("bad", [math.inf, -math.inf])
def test_a_norm_that_is_infinite_under_no_limit(bad):
    """Nothing is clipped: the gradients keep their bits."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    g = make(SMALL)
    g[0][5] = bad
    before = [t.clone() for t in g]
    outs = [torch.zeros_like(t) for t in g]
    assert float(lce.clip_grad_norm(g, math.inf, grads_out=outs)) == math.inf
    assert float(lce.clip_grad_norm(g, math.inf)) == math.inf
    for t, o, b in zip(g, outs, before):
        assert torch.equal(t, b) and torch.equal(o, b)


@pytest.mark.parametrize("max_norm", [1.0, 1e9])
def test_layouts_against_float64(max_norm):
    """Transposed and permuted gradients: norm and values as they lie."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    a = make([((30, 50), F32), ((4, 5, 6), BF)], std=3.0)
    before = [t.clone() for t in a]
    norm = lce.clip_grad_norm([a[0].t(), a[1].permute(2, 0, 1)], max_norm)
    want = ref.grad_norm(before)
    assert abs(float(norm) - want) <= want * NORM
    for t, c in zip(a, ref.clip(before, float(norm), max_norm)):
        near(t, c, t.dtype)
