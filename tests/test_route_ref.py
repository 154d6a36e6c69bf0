"""Routing without a GPU: the reference's gradient formulas against central
differences, closed forms, and the refusals of the C ABI and the binding."""
import ctypes

import numpy as np
import pytest
import torch

from tests import sparse_ref as ref


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_formulas_against_differences(scoring, renorm):
    rng = np.random.default_rng(3)
    z = rng.normal(size=(5, 9))
    w, e = ref.route(z, 3, scoring, renormalize=renorm, scale=2.5)
    dw = rng.normal(size=w.shape)
    dz = ref.route_grad(z, e, dw, scoring, renorm, 2.5)
    h = 1e-5
    for i in range(5):
        for j in range(9):
            f = []
            for sgn in (1, -1):
                zz = z[i].copy()
                zz[j] += sgn * h
                f.append((ref.weights_of(zz, e[i], scoring, renorm, 2.5) *
                          dw[i]).sum())
            # truncation h^2 f'''/6 and rounding 2^-53 f / h, both < 1e-9
            assert abs((f[0] - f[1]) / (2 * h) - dz[i, j]) < 1e-8


def test_closed_forms():
    z = np.zeros((1, 6))
    w, e = ref.route(z, 4)
    assert e.tolist() == [[0, 1, 2, 3]] and np.allclose(w, 0.25)
    w, e = ref.route(z, 2, "sigmoid", renormalize=False, scale=3.0,
                     bias=np.array([0, 0, 1.0, 0, 1.0, 0]))
    assert e.tolist() == [[2, 4]] and np.allclose(w, 1.5)
    # two groups of three: the second has the larger pair sum
    z = np.array([[5.0, -9, -9, 2, 2, 2]])
    assert ref.select(z[0], 2, "sigmoid", n_group=2, topk_group=1,
                      group_top=2) == [3, 4]
    assert ref.select(z[0], 2, "sigmoid", n_group=2, topk_group=1,
                      group_top=1) == [0, 1]
    w, e = ref.route(np.full((1, 4), -np.inf), 2)
    assert e.tolist() == [[0, 1]] and (w == 0).all()


@pytest.fixture(scope="module")
def lib():
    import chunked_lm_head_gemm_gb300 as lce
    return lce.load(build_if_missing=True)


def _opts(**kw):
    from chunked_lm_head_gemm_gb300 import _binding as B
    d = dict(scoring=0, top_k=2, n_group=1, topk_group=1, group_top=1,
             renormalize=1, scale=1.0)
    d.update(kw)
    return ctypes.pointer(B.RouteOpts(*d.values()))


BAD = [dict(scoring=2), dict(scoring=-1), dict(top_k=0), dict(top_k=33),
       dict(top_k=9), dict(renormalize=2), dict(scale=float("inf")),
       dict(scale=float("nan"))]
BAD_FORWARD = [dict(n_group=0), dict(n_group=3), dict(n_group=2, topk_group=0),
               dict(n_group=2, topk_group=3),
               dict(n_group=4, topk_group=1, top_k=3),
               dict(n_group=2, group_top=3), dict(n_group=2, group_top=0),
               dict(n_group=8, topk_group=8, group_top=2)]


def test_refusals_before_any_device_call(lib):
    """Every call fails validation first, so no pointer is used."""
    p, null = ctypes.c_void_p(0x1000), ctypes.c_void_p(0)
    odd = ctypes.c_void_p(0x1001)

    def fwd(o, z=p, dt=0, bias=null, L=4, E=8, w=p, e=p):
        return lib.lce_route_forward(z, dt, bias, L, E, o, w, e, null)

    def bwd(o, z=p, dt=0, e=p, dw=p, L=4, E=8, dz=p):
        return lib.lce_route_backward(z, dt, e, dw, L, E, o, dz, null)

    for kw in BAD:
        assert fwd(_opts(**kw)) == 1, kw
        assert bwd(_opts(**kw)) == 1, kw
    for kw in BAD_FORWARD:
        assert fwd(_opts(**kw)) == 1, kw
    ok = _opts()
    for f in (fwd, bwd):
        assert f(None) == 1
        assert f(ok, dt=5) == 2
        assert f(ok, L=-1) == 1 and f(ok, E=0) == 1 and f(ok, E=1025) == 1
        assert f(ok, z=null) == 1 and f(ok, z=odd) == 1
        assert f(ok, e=null) == 1 and f(ok, e=ctypes.c_void_p(0x1002)) == 1
        # nothing to do, whatever the pointers
        assert f(ok, z=null, e=null, L=0) == 0
    assert fwd(ok, w=null) == 1 and fwd(ok, bias=odd) == 1
    assert bwd(ok, dw=null) == 1 and bwd(ok, dz=null) == 1


def test_binding_refusals(lib):
    import chunked_lm_head_gemm_gb300 as lce
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        lce.route_forward(z, 2)
    with pytest.raises(ValueError, match="CUDA"):
        lce.route_backward(z, torch.zeros(4, 2, dtype=torch.int32),
                           torch.zeros(4, 2))
