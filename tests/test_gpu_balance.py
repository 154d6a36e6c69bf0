"""The balance loss, its gradient and the experts' counts on the GPU against
their float64 reference (tests/step_ref.py), with tolerances derived there."""
import math

import pytest
import torch

from tests import step_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SCORES = pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])


def make(L, E, K, dtype, seed=0, masked=0.0, padded=0.0, drop=0.0, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    z = torch.randn(L, E, device="cuda", generator=g) * spread
    experts = torch.topk(z, K, dim=1).indices.int()
    if masked:
        z = z.masked_fill(uniform(L, E) < masked, -math.inf)
    if drop:
        experts = experts.masked_fill(uniform(L, K) < drop, -1)
    mask = uniform(L) >= padded if padded else None
    return z.to(dtype), experts.contiguous(), mask


def check(z, experts, mask, scoring, coef=0.3, dloss=1.7):
    import chunked_lm_head_gemm_gb300 as lce
    L, E = z.shape
    loss, counts, slopes = lce.balance_forward(z, experts, scoring, coef, mask)
    assert lce.get_error() == 0
    want, rcounts, rslopes = ref.balance(z, experts, scoring, coef, mask)
    assert counts.dtype is torch.int32
    assert torch.equal(counts.long(), rcounts)
    assert torch.equal(lce.expert_counts(experts, E, mask), counts)
    # coef reaches the library as fp32, off by at most U of itself, and a
    # slope is rounded once: (1 + U)^2 - 1 < 2.01 U
    assert ((slopes.double() - rslopes).abs() <=
            2.01 * ref.U * rslopes.abs() + 1e-45).all()
    rel = float(ref.balance_rel(z).max()) + ref.sum_bound(L) + 4 * ref.U
    assert abs(float(loss) - float(want)) <= abs(float(want)) * rel
    d = torch.tensor(dloss, device=z.device)
    dz = lce.balance_backward(z, slopes, d, scoring, mask)
    d = float(d)
    rz = ref.balance_grad(z, slopes, d, scoring, mask)
    tol = ref.balance_grad_tolerance(z, slopes, d, scoring, mask, z.dtype)
    off = (dz.double() - rz).abs()
    assert (off <= tol).all(), float((off - tol).max())
    return loss, counts, slopes, dz


SHAPES = [  # L, E, K, dtype
    (1, 1, 1, F32), (1, 128, 8, BF), (2, 3, 2, F32), (7, 5, 5, BF),
    (33, 31, 4, F32), (64, 32, 2, BF), (65, 33, 3, F32), (130, 60, 4, BF),
    (100, 64, 6, F32), (257, 100, 7, BF), (300, 127, 8, F32), (300, 128, 8, F32),
    (513, 129, 1, BF), (40, 250, 32, F32), (170, 256, 8, BF), (170, 256, 8, F32),
    (90, 257, 8, F32), (90, 384, 8, BF), (31, 511, 3, F32), (31, 512, 16, BF),
    (19, 513, 8, F32), (19, 1000, 10, F32), (23, 1024, 32, BF),
    (5003, 128, 8, BF), (20000, 64, 6, F32), (9001, 256, 8, F32)]


@SCORES
@pytest.mark.parametrize("L,E,K,dtype", SHAPES)
def test_shapes(L, E, K, dtype, scoring):
    require_gpu()
    check(*make(L, E, K, dtype, seed=E), scoring)


@SCORES
@pytest.mark.parametrize("L,E,K,dtype", [(9, 8, 2, F32), (1003, 60, 4, BF),
                                         (4099, 128, 8, F32),
                                         (777, 300, 5, BF)])
def test_masks_and_dropped_slots(L, E, K, dtype, scoring):
    require_gpu()
    z, experts, mask = make(L, E, K, dtype, seed=2, masked=0.2, padded=0.3,
                            drop=0.1)
    z[1] = -math.inf  # a row with nothing left
    mask[1] = True
    # what stands behind the mask is not looked at
    off = ~mask
    z[off] = math.nan
    experts[off] = 1 << 30
    clean = torch.where(mask[:, None], z, torch.zeros_like(z))
    safe = torch.where(mask[:, None], experts, torch.zeros_like(experts))
    got = check(clean, safe, mask, scoring)
    import chunked_lm_head_gemm_gb300 as lce
    loss, counts, slopes = lce.balance_forward(z, experts, scoring, 0.3, mask)
    dz = lce.balance_backward(z, slopes, torch.tensor(1.7, device="cuda"),
                              scoring, mask)
    assert lce.get_error() == 0
    for a, b in zip((loss, counts, slopes, dz), got):
        assert torch.equal(a, b)
    assert not dz[off].any() and not dz[1].any()


@SCORES
def test_nobody_takes_part(scoring):
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    z, experts, _ = make(50, 16, 2, F32)
    mask = torch.zeros(50, dtype=torch.bool, device="cuda")
    loss, counts, slopes, dz = check(z, experts, mask, scoring)
    assert float(loss) == 0 and not counts.any() and not dz.any()
    empty = torch.zeros(0, 16, device="cuda")
    none = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    loss, counts, slopes = lce.balance_forward(empty, none, scoring)
    assert float(loss) == 0 and not counts.any() and not slopes.any()
    dz = lce.balance_backward(empty, slopes, torch.ones((), device="cuda"))
    assert dz.shape == (0, 16)
    assert not lce.expert_counts(none, 16).any()


@SCORES
@pytest.mark.parametrize("shift", [-300.0, -90.0, 80.0, 3e4])
def test_far_logits(scoring, shift):
    """Scores keep their ratios far from zero, where sigmoid(z) alone is 0."""
    require_gpu()
    z, experts, _ = make(200, 64, 4, F32, seed=4)
    check(z + shift, experts, None, scoring)


@SCORES
def test_a_row_that_is_not_finite(scoring):
    """NaN stays in its row of the gradient, and reaches the loss."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    z, experts, _ = make(40, 33, 2, F32)
    z[7, 3] = math.nan
    loss, counts, slopes = lce.balance_forward(z, experts, scoring)
    assert math.isnan(float(loss)) and torch.isfinite(slopes).all()
    dz = lce.balance_backward(z, slopes, torch.ones((), device="cuda"),
                              scoring)
    rows = [i for i in range(40) if i != 7]
    assert torch.isnan(dz[7]).all() and torch.isfinite(dz[rows]).all()


def test_one_expert_takes_all():
    require_gpu()
    L, E, K = 3001, 40, 1
    z, _, _ = make(L, E, K, F32)
    experts = torch.full((L, K), 17, dtype=torch.int32, device="cuda")
    loss, counts, _, _ = check(z, experts, None, "softmax")
    assert int(counts[17]) == L


@pytest.mark.parametrize("L,K", [(5, 2), (5000, 8)])
def test_index_out_of_range(L, K):
    import chunked_lm_head_gemm_gb300 as lce
    from chunked_lm_head_gemm_gb300 import _binding as B
    require_gpu()
    z, experts, _ = make(L, 24, K, F32)
    for bad in (24, -2, 2 ** 31 - 1, -2 ** 31):
        e = experts.clone()
        e[L // 2, 1] = bad
        d = experts.clone()
        d[L // 2, 1] = -1
        got = lce.balance_forward(z, e)
        assert lce.get_error() == B.LCE_ERR_EXPERT_RANGE
        want = lce.balance_forward(z, d)
        assert lce.get_error() == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert torch.equal(lce.expert_counts(e, 24), want[1])
        assert lce.get_error() == B.LCE_ERR_EXPERT_RANGE


@pytest.mark.parametrize("L,K", [(1, 1), (64, 8), (513, 32), (40001, 8),
                                 (131072, 8)])
@pytest.mark.parametrize("E", [1, 60, 256, 1024])
def test_counts(L, K, E):
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(L + E)
    e = torch.randint(-1, E, (L, K), device="cuda", generator=g).int()
    mask = torch.rand(L, device="cuda", generator=g) < 0.7
    out = torch.full((E,), -5, dtype=torch.int32, device="cuda")
    for m in (None, mask):
        chosen = e if m is None else e[m]
        want = torch.bincount(chosen[chosen >= 0].long(), minlength=E)
        assert lce.expert_counts(e, E, m, counts_out=out) is out
        assert torch.equal(out.long(), want)
    assert lce.get_error() == 0


@SCORES
@pytest.mark.parametrize("E,dtype", [(64, F32), (128, BF), (61, BF)])
def test_addresses(E, dtype, scoring):
    require_gpu()
    z, experts, mask = make(300, E, 4, dtype, padded=0.2)
    flat = torch.empty(z.numel() + 1, dtype=dtype, device="cuda")
    moved = flat[1:].view(z.shape)
    moved.copy_(z)
    room = torch.zeros(301, dtype=torch.bool, device="cuda")
    room[1:] = mask
    check(moved, experts, room[1:], scoring)


@SCORES
def test_same_bits_again_and_dirty_workspace(scoring):
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    z, experts, mask = make(30011, 96, 6, F32, padded=0.1)
    first = lce.balance_forward(z, experts, scoring, mask=mask)
    ws = torch.full((lce.balance_workspace_size(30011, 96),), 255,
                    dtype=torch.uint8, device="cuda")
    again = lce.balance_forward(z, experts, scoring, mask=mask, workspace=ws)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_autograd_capture_and_streams():
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    z, experts, mask = make(4000, 128, 8, F32, padded=0.2)
    leaf = z.clone().requires_grad_(True)
    loss, counts = lce.balance_loss(leaf, experts, coef=0.02, mask=mask)
    assert not counts.requires_grad
    (2 * loss).backward()
    _, _, slopes = lce.balance_forward(z, experts, coef=0.02, mask=mask)
    two = torch.tensor(2.0, device="cuda")
    want = lce.balance_backward(z, slopes, two, mask=mask)
    assert torch.equal(leaf.grad, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lce.balance_forward(z, experts, coef=0.02, mask=mask)
        dz = lce.balance_backward(z, out[2], two, mask=mask)
        alone = lce.expert_counts(experts, 128, mask)
    for seed in (5, 6):
        nz, ne, nm = make(4000, 128, 8, F32, seed=seed, padded=0.3)
        z.copy_(nz), experts.copy_(ne), mask.copy_(nm)
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            again = lce.balance_forward(z, experts, coef=0.02, mask=mask)
            dagain = lce.balance_backward(z, again[2], two, mask=mask)
        side.synchronize()
        for a, b in zip((*out, dz, alone), (*again, dagain, again[1])):
            assert torch.equal(a, b)


def test_second_derivative_is_refused():
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    z, experts, _ = make(40, 12, 2, F32)
    z.requires_grad_(True)
    loss, _ = lce.balance_loss(z, experts)
    g, = torch.autograd.grad(loss.square(), z, create_graph=True)
    total = g.square().sum() + z.square().sum()
    with pytest.raises(RuntimeError, match="twice"):
        total.backward()


def test_offsets_past_32_bits():
    """Logits behind 2^31 elements: 2.2e9 elements of bf16."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    L, E, K = 2150000, 1024, 1
    z = torch.zeros(L, E, dtype=BF, device="cuda")
    tail, te, _ = make(64, E, K, BF, seed=1)
    z[-64:] = tail
    experts = torch.zeros(L, K, dtype=torch.int32, device="cuda")
    experts[-64:] = te
    mask = torch.zeros(L, dtype=torch.bool, device="cuda")
    mask[-64:] = True
    got = lce.balance_forward(z, experts, mask=mask)
    want = lce.balance_forward(tail, te)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    rel = float(ref.balance_rel(tail).max()) + ref.sum_bound(64)
    assert abs(float(got[0]) - float(want[0])) <= 2 * rel * float(want[0])
    one = torch.ones((), device="cuda")
    dz = lce.balance_backward(z, got[2], one, mask=mask)
    assert torch.equal(dz[-64:], lce.balance_backward(tail, want[2], one))
    assert not dz[:L - 64:1009].any()
