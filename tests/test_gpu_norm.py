"""Layer norm and RMS norm on the GPU against their float64 reference
(tests/step_ref.py), with tolerances derived there: forward, and backward from
the statistics that the forward returned."""
import math

import pytest
import torch

from tests import step_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
KINDS = pytest.mark.parametrize("layer", [True, False], ids=["layer", "rms"])


def make(L, H, dtype, pdtype, seed=0, offset=0.0, std=1.0, affine=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    x = (normal(L, H) * std + offset).to(dtype)
    dy = normal(L, H).to(dtype)
    w = (1 + 0.3 * normal(H)).to(pdtype) if affine else None
    b = (0.3 * normal(H)).to(pdtype) if affine else None
    return x, w, b, dy


def forward(x, w, b, eps, layer, **kw):
    import chunked_lm_head_gemm_gb300 as lce
    if layer:
        return lce.layer_norm_forward(x, w, b, eps=eps, **kw)
    y, rstd = lce.rms_norm_forward(x, w, eps=eps, **kw)
    return y, None, rstd


def backward(x, w, mean, rstd, dy, layer, **kw):
    import chunked_lm_head_gemm_gb300 as lce
    if layer:
        return lce.layer_norm_backward(x, w, mean, rstd, dy, **kw)
    kw.pop("compute_dbias", None)
    return *lce.rms_norm_backward(x, w, rstd, dy, **kw), None


def near(got, want, tol):
    off = (got.double() - want).abs()
    assert (off <= tol).all(), float((off - tol).max())


def check(x, w, b, dy, layer, eps=1e-5, grad_dtype=F32):
    if not layer:
        b = None
    y, mean, rstd = forward(x, w, b, eps, layer)
    ry, rmean, rrstd = ref.norm(x, w, b, eps, layer)
    near(y, ry, ref.norm_tolerance(x, w, b, eps, layer, x.dtype))
    A = ref.sum_bound(x.shape[1])
    if layer:
        near(mean, rmean, (A + ref.U) * x.double().abs().mean(1) + 1e-37)
    lost = A * x.double().abs().mean(1) if layer else 0.0
    near(rstd, rrstd, rrstd * (A + 8 * ref.U + (lost * rrstd) ** 2))
    dx, dw, db = backward(x, w, mean, rstd, dy, layer, grad_dtype=grad_dtype)
    want = ref.norm_grad(x, w, mean, rstd, dy, layer)
    tol = ref.norm_grad_tolerance(x, w, mean, rstd, dy, layer, x.dtype,
                                  grad_dtype)
    near(dx, want[0], tol[0])
    near(dw, want[1], tol[1])
    if layer:
        near(db, want[2], tol[2])
    return y, mean, rstd, dx, dw, db


WIDTHS = [1, 2, 3, 7, 8, 31, 32, 33, 64, 100, 127, 128, 129, 255, 256, 264, 384,
          511, 512, 520, 768, 1000, 1001, 1024, 1032, 1536, 2048, 2050, 2056,
          2560, 4096, 4100, 5120, 8192, 8193, 8200, 12288, 16384, 16392, 16401]


@KINDS
@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("dtype,pdtype", [(BF, BF), (BF, F32), (F32, F32),
                                          (F32, BF)],
                         ids=["bf-bf", "bf-f32", "f32-f32", "f32-bf"])
def test_widths(H, dtype, pdtype, layer):
    require_gpu()
    check(*make(37, H, dtype, pdtype, seed=H), layer, grad_dtype=pdtype)


@KINDS
@pytest.mark.parametrize("H", [9001, 12345, 16383, 32768, 32769, 32776, 40001,
                               65535, 65536, 65537, 200000])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf", "f32"])
def test_wide_rows(H, dtype, layer):
    require_gpu()
    check(*make(5, H, dtype, F32, seed=H), layer)


@KINDS
@pytest.mark.parametrize("L", [1, 2, 3, 5, 8, 9, 150, 153, 1000, 4099])
@pytest.mark.parametrize("H,dtype", [(40, BF), (128, BF), (129, F32), (640, F32),
                                     (2048, BF), (4096, BF), (1001, BF)])
def test_row_counts(L, H, dtype, layer):
    require_gpu()
    check(*make(L, H, dtype, F32, seed=L), layer)


@KINDS
@pytest.mark.parametrize("L,H,dtype", [(200003, 128, BF), (100001, 64, F32),
                                       (40000, 1024, BF), (20000, 4096, BF),
                                       (70001, 33, BF), (3000, 16384, BF),
                                       (2000, 9001, F32), (2001, 9003, BF), (700, 40000, BF),
                                       (600, 65536, F32)])
def test_many_rows(L, H, dtype, layer):
    require_gpu()
    check(*make(L, H, dtype, dtype, seed=3), layer, grad_dtype=F32)


@KINDS
@pytest.mark.parametrize("offset,std", [(100.0, 1.0), (-3.0, 0.01),
                                        (0.0, 1e-4), (0.0, 1e4), (0.0, 0.0),
                                        (5.0, 0.0)])
@pytest.mark.parametrize("H,dtype", [(128, F32), (1000, F32), (4096, F32),
                                     (513, BF)])
def test_offsets_and_scales(H, dtype, offset, std, layer):
    """Rows far from zero, tiny, huge, all zero and all alike."""
    require_gpu()
    x, w, b, dy = make(19, H, dtype, F32, seed=7, offset=offset, std=std)
    check(x, w, b, dy, layer)


@KINDS
@pytest.mark.parametrize("H", [128, 1001, 2048])
def test_no_parameters(H, layer):
    require_gpu()
    x, _, _, dy = make(33, H, BF, F32, affine=False)
    check(x, None, None, dy, layer)


def test_bias_or_weight_alone():
    require_gpu()
    x, w, b, dy = make(9, 320, BF, F32)
    check(x, None, b, dy, True)
    check(x, w, None, dy, True)


@KINDS
@pytest.mark.parametrize("H,dtype", [(128, BF), (1024, BF), (4096, F32),
                                     (1001, F32), (40000, BF)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_rows_that_are_not_finite_stay_apart(H, dtype, bad, layer):
    require_gpu()
    x, w, b, dy = make(21, H, dtype, F32)
    clean = forward(x, w, b if layer else None, 1e-5, layer)
    dx_clean = backward(x, w, *clean[1:], dy, layer, compute_dweight=False,
                        compute_dbias=False)[0]
    x[4, H // 2] = bad
    y, mean, rstd = forward(x, w, b if layer else None, 1e-5, layer)
    dx = backward(x, w, mean, rstd, dy, layer, compute_dweight=False,
                  compute_dbias=False)[0]
    rows = [i for i in range(21) if i != 4]
    assert torch.equal(y[rows], clean[0][rows])
    assert torch.equal(dx[rows], dx_clean[rows])
    ry = ref.norm(x[4:5].cpu(), w.cpu(), b.cpu() if layer else None, 1e-5,
                  layer)[0]
    assert torch.equal(torch.isnan(y[4]).cpu(), torch.isnan(ry[0]))


@KINDS
@pytest.mark.parametrize("dtype,H", [(BF, 136), (BF, 2048), (F32, 132),
                                     (F32, 4096), (BF, 999), (BF, 9001),
                                     (F32, 20001), (BF, 9002)])
@pytest.mark.parametrize("shift", [1, 3, 4])
def test_addresses(dtype, H, shift, layer):
    """Tensors that start on their element's alignment alone give the bits of
    aligned ones, or what their tolerance allows."""
    require_gpu()
    L = 11
    x, w, b, dy = make(L, H, dtype, dtype, seed=5)

    def moved(t):
        flat = torch.empty(t.numel() + shift, dtype=t.dtype, device=t.device)
        out = flat[shift:].view(t.shape)
        return out.copy_(t)

    check(moved(x), moved(w), moved(b), moved(dy), layer, grad_dtype=dtype)
    check(x, moved(w), b, moved(dy), layer, grad_dtype=dtype)
    import chunked_lm_head_gemm_gb300 as lce
    y_out = moved(x)
    want = forward(x, w, b if layer else None, 1e-5, layer)[0]
    kw = dict(eps=1e-5, y_out=y_out)
    if layer:
        lce.layer_norm_forward(x, w, b, **kw)
    else:
        lce.rms_norm_forward(x, w, **kw)
    near(y_out, want.double(), 2 * ref.norm_tolerance(
        x, w, b if layer else None, 1e-5, layer, dtype))


@KINDS
@pytest.mark.parametrize("L,H,dtype", [(50, 128, BF), (7, 1001, BF),
                                       (600, 2048, BF), (9, 40000, F32),
                                       (400, 9001, BF), (300, 9002, BF)])
def test_in_place(L, H, dtype, layer):
    """y over x; dx over dy, and over x."""
    require_gpu()
    x, w, b, dy = make(L, H, dtype, F32)
    y, mean, rstd = forward(x, w, b if layer else None, 1e-5, layer)
    x2 = x.clone()
    y2 = forward(x2, w, b if layer else None, 1e-5, layer, y_out=x2)[0]
    assert y2 is x2 and torch.equal(x2, y)
    want = backward(x, w, mean, rstd, dy, layer)
    for which in ("dy", "x"):
        t = dict(x=x.clone(), dy=dy.clone())
        got = backward(t["x"], w, mean, rstd, t["dy"], layer, dx_out=t[which])
        for a, c in zip(got, want):
            assert (a is None and c is None) or torch.equal(a, c)


@KINDS
@pytest.mark.parametrize("L,H", [(300, 128), (300, 4096), (31, 1001),
                                 (6, 40000)])
def test_optional_gradients_keep_their_bits(L, H, layer):
    require_gpu()
    x, w, b, dy = make(L, H, BF, F32)
    _, mean, rstd = forward(x, w, b if layer else None, 1e-5, layer)
    every = backward(x, w, mean, rstd, dy, layer)
    for mask in range(1, 8 if layer else 4):
        want = [bool(mask >> i & 1) for i in range(3)]
        got = backward(x, w, mean, rstd, dy, layer, compute_dx=want[0],
                       compute_dweight=want[1], compute_dbias=want[2])
        for g, e, n in zip(got, every, want):
            assert (g is None) == (not n)
            if n:
                assert torch.equal(g, e)


@KINDS
def test_no_rows(layer):
    require_gpu()
    x, w, b, dy = make(0, 64, BF, F32)
    y, mean, rstd = forward(x, w, b if layer else None, 1e-5, layer)
    assert y.shape == (0, 64)
    dx, dw, db = backward(x, w, mean, rstd, dy, layer)
    assert dx.shape == (0, 64) and not dw.any()
    assert db is None or not db.any()


@KINDS
@pytest.mark.parametrize("L,H,dtype", [(33000, 128, BF), (4000, 4096, BF),
                                       (513, 1001, F32)])
def test_same_bits_again_and_dirty_workspace(L, H, dtype, layer):
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    x, w, b, dy = make(L, H, dtype, F32)
    _, mean, rstd = forward(x, w, b if layer else None, 1e-5, layer)
    first = backward(x, w, mean, rstd, dy, layer)
    ws = torch.full((lce.norm_workspace_size(L, H),), 255, dtype=torch.uint8,
                    device="cuda")
    again = backward(x, w, mean, rstd, dy, layer, workspace=ws)
    for a, c in zip(first, again):
        assert (a is None and c is None) or torch.equal(a, c)


def test_offsets_past_32_bits():
    """Rows behind 2^31 elements: 2.2e9 elements of bf16."""
    require_gpu()
    L, H = 540000, 4096
    x = torch.zeros(L, H, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    tail = torch.randn(100, H, device="cuda", generator=g).to(BF)
    x[-100:] = tail
    w = torch.ones(H, device="cuda")
    y, mean, rstd = forward(x, w, w, 1e-5, True)
    small = forward(tail, w, w, 1e-5, True)
    assert torch.equal(y[-100:], small[0])
    assert torch.equal(mean[-100:], small[1])
    assert (y[:L - 100:5003] == 1).all()
    dy = torch.zeros_like(x)
    dy[-100:] = tail
    dx, dw, db = backward(x, w, mean, rstd, dy, True)
    sdx, sdw, sdb = backward(tail, w, *small[1:], tail, True)
    assert torch.equal(dx[-100:], sdx) and not dx[:L - 100:5003].any()
    B = ref.sum_bound(L)
    near(dw, sdw.double(), 2 * B * (tail.double() ** 2).sum(0) * 3)
    near(db, sdb.double(), 2 * B * tail.double().abs().sum(0))


@KINDS
def test_autograd_and_types(layer):
    """Through the autograd form: gradients in the leaves' types, an upstream
    gradient that is not contiguous, against float64 autograd."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    x, w, b, dy = make(64, 256, F32, F32, seed=9)
    x, w, b = (t.requires_grad_(True) for t in (x, w, b))
    up = dy.t().contiguous().t()
    y = lce.layer_norm(x, w, b) if layer else lce.rms_norm(x, w, 1e-5)
    y.backward(up)
    d = [t.detach().double().requires_grad_(True) for t in (x, w, b)]
    m = d[0].mean(1, keepdim=True) if layer else 0.0
    v = (d[0] - m).square().mean(1, keepdim=True)
    r = (d[0] - m) / torch.sqrt(v + 1e-5) * d[1] + (d[2] if layer else 0.0)
    r.backward(dy.double())
    for t, u in zip((x, w, b)[:3 if layer else 2], d):
        e = (t.grad.double() - u.grad).norm() / u.grad.norm()
        assert e < 1e-6
    with torch.no_grad():
        free = lce.layer_norm(x, w, b) if layer else lce.rms_norm(x, w, 1e-5)
    assert not free.requires_grad and torch.equal(free, y.detach())


def test_frozen_parameters_and_second_derivative():
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    x, w, b, dy = make(16, 64, BF, BF)
    x.requires_grad_(True)
    lce.layer_norm(x, w, b).backward(dy)
    assert x.grad is not None and w.grad is None
    w.requires_grad_(True)
    y = lce.rms_norm(x.detach(), w)
    y.backward(dy)
    assert w.grad.dtype is BF
    z = lce.rms_norm(x, w)
    g, = torch.autograd.grad(z.float().square().sum(), x, create_graph=True)
    loss = g.float().square().sum() + x.float().square().sum()
    with pytest.raises(RuntimeError, match="twice"):
        loss.backward()


@KINDS
def test_capture_and_streams(layer):
    """Forward and backward captured once and replayed on new inputs, and run
    on a stream of their own."""
    require_gpu()
    x, w, b, dy = make(700, 1024, BF, F32)
    b = b if layer else None

    def step():
        y, mean, rstd = forward(x, w, b, 1e-5, layer)
        return (y, *backward(x, w, mean, rstd, dy, layer))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2):
        nx, _, _, ndy = make(700, 1024, BF, F32, seed=seed)
        x.copy_(nx)
        dy.copy_(ndy)
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = step()
        side.synchronize()
        for a, c in zip(out, want):
            assert (a is None and c is None) or torch.equal(a, c)
