"""The float64 reference of the norms, the balance loss and the clipping: its
gradient formulas against central differences. No GPU."""
import math

import pytest
import torch

from tests import step_ref as ref

STEP = 1e-6


def slope(f, t, i):
    """Central difference of f along element i of t."""
    up, down = t.clone(), t.clone()
    up.view(-1)[i] += STEP
    down.view(-1)[i] -= STEP
    return (f(up) - f(down)) / (2 * STEP)


def gen(*shape, seed):
    return torch.randn(*shape, dtype=torch.float64,
                       generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("H", [1, 2, 7])
def test_norm_gradients(layer, H):
    x, w, b, dy = gen(3, H, seed=1), gen(H, seed=2), gen(H, seed=3), \
        gen(3, H, seed=4)
    b = b if layer else None
    eps = 1e-2

    def loss(x_, w_, b_):
        return float((ref.norm(x_, w_, b_, eps, layer)[0] * dy).sum())

    _, mean, rstd = ref.norm(x, w, b, eps, layer)
    dx, dw, db = ref.norm_grad(x, w, mean, rstd, dy, layer)
    for i in range(x.numel()):
        assert abs(slope(lambda t: loss(t, w, b), x, i) - dx.view(-1)[i]) < 1e-7
    for i in range(H):
        assert abs(slope(lambda t: loss(x, t, b), w, i) - dw[i]) < 1e-7
        if layer:
            assert abs(slope(lambda t: loss(x, w, t), b, i) - db[i]) < 1e-7


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_balance_gradient(scoring):
    L, E, K = 5, 6, 2
    z = gen(L, E, seed=5)
    z[0, 2] = -math.inf
    z[3] = -math.inf
    experts = torch.tensor([[0, 1], [5, -1], [2, 2], [1, 0], [4, 9]])
    mask = torch.tensor([True, True, False, True, True])
    _, counts, slopes = ref.balance(z, experts, scoring, 0.7, mask)
    assert counts.tolist() == [2, 2, 0, 0, 1, 1]
    dz = ref.balance_grad(z, slopes, 1.3, scoring, mask)
    assert not dz[2].any() and not dz[3].any()

    def loss(t):
        return 1.3 * float(ref.balance(t, experts, scoring, 0.7, mask)[0])

    for i in range(L * E):
        if torch.isfinite(z.view(-1)[i]):
            assert abs(slope(loss, z, i) - dz.view(-1)[i]) < 1e-8


def test_even_load_has_no_gradient_and_loss_coef():
    z = gen(4, 4, seed=6)
    experts = torch.tensor([[0], [1], [2], [3]])
    loss, counts, slopes = ref.balance(z, experts, "softmax", 0.5, None)
    assert abs(float(loss) - 0.5) < 1e-15 and not slopes.any()
    assert counts.tolist() == [1, 1, 1, 1]


def test_clip():
    g = [torch.tensor([3.0]), torch.tensor([[4.0]]), torch.zeros(0)]
    assert ref.grad_norm(g) == 5.0
    assert float(ref.clip(g, 5.0, 1.0)[1]) == pytest.approx(0.8, rel=1e-6)
    assert float(ref.clip(g, 5.0, 10.0)[1]) == 4.0
    assert float(ref.clip(g, 5.0, math.inf)[1]) == 4.0
