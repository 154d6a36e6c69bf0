"""The experts' MLP without a GPU: the reference's gradient formulas against
central differences, its agreement with one dense MLP, and refusals."""
import ctypes

import numpy as np
import pytest
import torch

from tests import sparse_ref as ref


def _draw(L=6, H=5, I=4, E=3, K=2, seed=0):
    r = np.random.default_rng(seed)
    e = np.stack([r.permutation(E)[:K] for _ in range(L)])
    e[1, 0] = -1
    e[2] = -1
    return [r.normal(size=s) for s in ((L, H), (E, I, H), (E, I, H),
                                       (E, H, I), (L, K))] + [e]


def test_gradient_formulas_against_differences():
    args = _draw()
    dy = np.random.default_rng(9).normal(size=args[0].shape)
    grads = ref.experts_mlp(*args, dy)[1:]
    h = 1e-5
    for n in range(5):
        flat = args[n].reshape(-1)
        for i in range(flat.size):
            keep = flat[i]
            f = []
            for sgn in (1, -1):
                flat[i] = keep + sgn * h
                f.append((ref.experts_mlp(*args) * dy).sum())
            flat[i] = keep
            # truncation h^2 f'''/6 and rounding 2^-53 |f| / h
            assert abs((f[0] - f[1]) / (2 * h) - grads[n].reshape(-1)[i]) < 1e-7


def test_one_expert_is_the_dense_mlp():
    x, Wg, Wu, Wd, w, e = _draw(E=1, K=1)
    e[:] = 0
    g, u = x @ Wg[0].T, x @ Wu[0].T
    y = (g / (1 + np.exp(-g)) * u) @ Wd[0].T * w
    assert np.allclose(ref.experts_mlp(x, Wg, Wu, Wd, w, e), y, rtol=1e-12)


@pytest.fixture(scope="module")
def lib():
    import chunked_lm_head_gemm_gb300 as lce
    return lce.load(build_if_missing=True)


def test_workspace_size(lib):
    f = lib.lce_experts_workspace_size
    good = dict(L=100, H=64, I=72, E=8, K=2, b=0)
    assert f(*good.values()) > 100 * 2 * (72 * 2 + 64 * 4)
    assert f(*dict(good, b=1).values()) > f(*good.values())
    assert f(*dict(good, L=0).values()) > 0
    for bad in (dict(L=-1), dict(H=12), dict(H=0), dict(I=4), dict(E=0),
                dict(E=1025), dict(K=0), dict(K=33), dict(b=2),
                dict(L=1 << 30)):
        assert f(*dict(good, **bad).values()) == 0, bad


def test_refusals_before_any_device_call(lib):
    """Every call fails validation first, so no pointer is used."""
    p, null = ctypes.c_void_p(0x1000), ctypes.c_void_p(0)
    odd = ctypes.c_void_p(0x1008)

    def fwd(x=p, Wg=p, Wu=p, Wd=p, w=p, dt=0, e=p, L=4, H=8, I=8, E=4, K=2,
            y=p, ws=p, n=1 << 30):
        return lib.lce_experts_forward(x, Wg, Wu, Wd, w, dt, e, L, H, I, E, K,
                                       y, ws, n, null)

    def bwd(x=p, Wg=p, Wu=p, Wd=p, w=p, dt=0, e=p, dy=p, L=4, H=8, I=8, E=4,
            K=2, gdt=0, dx=p, dWg=p, dWu=p, dWd=p, dw=p, ws=p, n=1 << 30):
        return lib.lce_experts_backward(x, Wg, Wu, Wd, w, dt, e, dy, L, H, I,
                                        E, K, gdt, dx, dWg, dWu, dWd, dw, ws,
                                        n, null)

    for f in (fwd, bwd):
        for name in ("x", "Wg", "Wu", "Wd", "w", "e", "ws"):
            assert f(**{name: null}) == 1, name
        for name in ("x", "Wg", "Wu", "Wd", "ws"):
            assert f(**{name: odd}) == 1, name
        assert f(H=12) == 1 and f(I=12) == 1 and f(E=0) == 1 and f(K=33) == 1
        assert f(L=-1) == 1 and f(L=1 << 30) == 1
        assert f(dt=7) == 2
        assert f(n=64) == 3
    assert fwd(y=null) == 1 and fwd(y=odd) == 1
    assert bwd(dy=null) == 1 and bwd(dy=odd) == 1 and bwd(gdt=3) == 2
    assert bwd(dWg=null) == 1 and bwd(dWu=null) == 1
    assert bwd(dx=null, dWg=null, dWu=null, dWd=null, dw=null) == 1
    assert bwd(dx=odd) == 1 and bwd(dWd=odd) == 1
    assert bwd(dw=ctypes.c_void_p(0x1001)) == 1
    assert bwd(dx=null, dWg=null, dWu=null, dWd=null, n=64) == 3
    assert fwd(x=null, w=null, e=null, y=null, L=0) == 0  # nothing to do


def test_binding_refusals(lib):
    import chunked_lm_head_gemm_gb300 as lce
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    W = torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    e = torch.zeros(4, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lce.experts_forward(x, W, W, W, torch.zeros(4, 1), e)
    with pytest.raises(ValueError, match="invalid"):
        lce.experts_workspace_size(4, 12, 8, 2, 1)
