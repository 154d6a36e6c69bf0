"""The norms' parameter gradients over many rows. A thread adds at most 1024
rows in fp32 registers (with up to 1024 blocks); of terms of one sign the k-th
of m additions is off by at most U = 2^-24 of k / m of the sum, together (m + 1)
/ 2 U. A cluster's runs have at most 64 rows and a 128th of all, of 38912 rows
368, and it adds 8 runs to one another where clusters are 14 or more. What
blocks or clusters have is joined to twice that precision and rounded once."""
import pytest
import torch

from tests import step_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("L,H,layer,m", [(38912, 32800, False, 368 + 2 * 8),
                                         (38912, 32801, True, 368 + 2 * 8),
                                         (38912, 65536, False, 368 + 2 * 8),
                                         (600000, 640, True, 1024),
                                         (5000011, 63, False, 1024)])
def test_rows_whose_sums_are_rounded_one_way(L, H, layer, m):
    """Every row adds 1 + 2^-14 - 2^-20 to every column (x = dy = 1, and that
    for rstd): sums from 1024 to 4096 in fp32 would lose 2^-14 of each."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    ones = torch.ones(L, H, dtype=torch.bfloat16, device="cuda")
    v = 1 + 2.0 ** -14 - 2.0 ** -20
    rstd = torch.full((L,), v, device="cuda")
    if layer:
        _, dw, db = lce.layer_norm_backward(ones, None, torch.zeros_like(rstd),
                                            rstd, ones, compute_dx=False)
        assert (db == L).all()  # below 2^24: exact
    else:
        _, dw = lce.rms_norm_backward(ones, None, rstd, ones, compute_dx=False)
    assert lce.get_error() == 0
    off = (dw.double() / (L * v) - 1).abs().max()
    assert off <= ((m + 1) / 2 + 1) * ref.U


@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("H", [16400, 20001])
def test_several_runs_of_rows(H, layer):
    """Rows of clusters in several runs: every gradient against float64, and
    the same bits again."""
    from tests.test_gpu_norm import BF, backward, check, make
    require_gpu()
    x, w, b, dy = make(3001, H, BF, BF, seed=H)
    _, mean, rstd, *grads = check(x, w, b, dy, layer)
    again = backward(x, w, mean, rstd, dy, layer)
    for a, c in zip(grads, again):
        assert (a is None and c is None) or torch.equal(a, c)


@pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])
@pytest.mark.parametrize("L,H", [(3, 16400), (300, 513), (3001, 20001),
                                 (40000, 8200), (2000, 65536), (1500, 65535),
                                 (20000, 1001), (60000, 8192)])
def test_the_workspace_holds_all_slabs(L, H, layer):
    """A workspace of just the stated size, with a mark behind it."""
    import chunked_lm_head_gemm_gb300 as lce
    from tests.test_gpu_norm import BF, backward, make
    require_gpu()
    x, w, _, dy = make(L, H, BF, BF, seed=H)
    rstd = torch.rand(L, device="cuda") + 0.5
    mean = torch.zeros(L, device="cuda") if layer else None
    size = lce.norm_workspace_size(L, H)
    room = torch.full((size + 4096,), 171, dtype=torch.uint8, device="cuda")
    got = backward(x, w, mean, rstd, dy, layer, workspace=room[:size])
    assert (room[size:] == 171).all()
    want = ref.norm_grad(x, w, mean, rstd, dy, layer)
    tol = ref.norm_grad_tolerance(x, w, mean, rstd, dy, layer, BF,
                                  torch.float32)
    for g, v, t in zip(got, want, tol):
        assert g is None or ((g.double() - v).abs() <= t).all()
