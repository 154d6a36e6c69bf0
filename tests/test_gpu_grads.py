"""The global gradient norm and the clipping on the GPU against float64
(tests/step_ref.py). Tolerances: squares are added in fp32 in groups of at
most 32, then in fp64, so the sum is off by at most 33 steps of 2^-24 relative
and the norm, rounded once, by 17.5 of them; an output is one product of a
rounded factor, rounded once."""
import math

import pytest
import torch

from tests import step_ref as ref
from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NORM = 17.5 * ref.U


def make(shapes, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(*s, device="cuda", generator=g) * std).to(t)
            for s, t in shapes]


def near(got, want, dtype):
    tol = want.abs() * (2 * ref.U + ref.half(dtype)) + 1e-45
    if dtype is BF:
        tol = tol + 1e-40  # a result below the normal range
    assert ((got.double() - want).abs() <= tol).all()


def check(grads, max_norm):
    import chunked_lm_head_gemm_gb300 as lce
    before = [g.clone() for g in grads]
    norm = lce.grad_norm(grads)
    want = ref.grad_norm(grads)
    assert norm.dtype is F32 and norm.shape == ()
    assert abs(float(norm) - want) <= want * NORM
    outs = [torch.full_like(g, 7.0) for g in grads]
    again = lce.clip_grad_norm(grads, max_norm, grads_out=outs)
    assert torch.equal(again, norm)
    for g, b in zip(grads, before):
        assert torch.equal(g, b)
    clipped = ref.clip(before, float(norm), max_norm)
    for o, c in zip(outs, clipped):
        near(o, c, o.dtype)
    assert torch.equal(lce.clip_grad_norm(grads, max_norm), norm)
    for g, o in zip(grads, outs):
        assert torch.equal(g, o)
    return norm, outs


SIZES = [1, 2, 3, 7, 8, 9, 31, 64, 255, 1000, 1023, 4096, 4097, 16383, 16384,
         16385, 32768, 50001, 262144, 1000003]


@pytest.mark.parametrize("n", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf", "f32"])
def test_sizes(n, dtype):
    require_gpu()
    check(make([((n,), dtype)], seed=n), 0.5)


@pytest.mark.parametrize("count", [2, 31, 95, 96, 97, 130, 700])
def test_many_tensors(count):
    """Tables that end inside a launch and fill several; shapes and types
    mixed, empty tensors among them."""
    require_gpu()
    shapes = [((1 + 37 * i % 301, 1 + i % 7), BF if i % 3 else F32)
              for i in range(count)]
    shapes[count // 2] = ((0, 5), F32)
    check(make(shapes, seed=count), 3.0)
    check(make([((3, 0), BF)] + shapes + [((0,), F32)], seed=1), 1e9)


def test_large():
    require_gpu()
    check(make([((50_000_001,), BF), ((30_000_000,), F32), ((17,), F32)]), 1.0)


def test_a_tensor_past_32_bits():
    """2^31 + 1000 elements, clipped in place: the last ones too."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    n = 2 ** 31 + 1000
    g = torch.zeros(n, dtype=BF, device="cuda")
    g[-700:] = 3.0
    g[:300] = 4.0
    norm = lce.clip_grad_norm([g], 1.0)
    want = math.sqrt(700 * 9 + 300 * 16)
    assert abs(float(norm) - want) <= want * NORM
    scale = 1.0 / (float(norm) + 1e-6)
    for part, v in ((g[-700:], 3.0), (g[:300], 4.0)):
        off = (part.double() - v * scale).abs().max()
        assert off <= v * scale * (2 * ref.U + ref.half(BF))
    assert not g[300:-700:100003].any()


@pytest.mark.parametrize("max_norm", [0.0, 1e-6, 1.0, 1e30, math.inf])
def test_limits(max_norm):
    """From everything to nothing clipped; a factor of 1 leaves the bits."""
    require_gpu()
    shapes = [((1000,), F32), ((77, 5), BF)]
    _, outs = check(make(shapes, seed=2), max_norm)
    if max_norm > 1e6:
        for o, g in zip(outs, make(shapes, seed=2)):
            assert torch.equal(o, g)
    if max_norm == 0.0:
        assert not any(o.any() for o in outs)


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-16, 1e16, 1e22, 1e30])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf", "f32"])
def test_far_scales(scale, dtype):
    """Squares below and above fp32's range count in full."""
    require_gpu()
    check(make([((100003,), dtype), ((5,), dtype)], std=scale), 0.1 * scale)


def test_mixed_scales():
    require_gpu()
    g = make([((5000,), F32)], std=1e-25) + make([((5000,), F32)], std=1e-2)
    g[0][::7] = 0
    check(g, 1.0)
    g = make([((4096,), F32)], std=1e-25)
    g[0][5::1000] = 1e21
    check(g, 1.0)


def test_zero_gradients():
    require_gpu()
    z = [torch.zeros(70000, device="cuda"), torch.zeros(3, dtype=BF,
                                                        device="cuda")]
    norm, outs = check(z, 1.0)
    assert float(norm) == 0 and not any(o.any() for o in outs)


def test_no_gradients():
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    assert float(lce.grad_norm([])) == 0.0
    assert float(lce.clip_grad_norm([], 1.0)) == 0.0
    e = [torch.zeros(0, device="cuda")]
    assert float(lce.clip_grad_norm(e, 1.0)) == 0.0


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 12345, 99999])
def test_not_finite(bad, at):
    """NaN makes every gradient NaN; infinity makes finite ones 0."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    g = make([((100000,), F32), ((64,), BF)])
    g[0][at] = bad
    norm = lce.clip_grad_norm(g, 1.0)
    if math.isnan(bad):
        assert math.isnan(float(norm))
        assert all(torch.isnan(t).all() for t in g)
    else:
        assert float(norm) == math.inf
        assert math.isnan(float(g[0][at]))
        g[0][at] = 0
        assert not any(t.any() for t in g)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf", "f32"])
@pytest.mark.parametrize("gs,os", [(0, 0), (1, 1), (1, 0), (0, 1), (3, 2),
                                   (5, 13)])
def test_addresses(dtype, gs, os):
    """Gradients and outputs that start anywhere in larger buffers, which keep
    what stands before and behind."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    for n in (1, 5, 17, 4099, 33333):
        src = make([((n + 40,), dtype)], seed=n)[0]
        g = src[gs:gs + n]
        buf = torch.full((n + 40,), 3.0, dtype=dtype, device="cuda")
        o = buf[os:os + n]
        norm = lce.clip_grad_norm([g], 0.25, grads_out=[o])
        want = ref.grad_norm([g])
        assert abs(float(norm) - want) <= want * NORM
        near(o, ref.clip([g], float(norm), 0.25)[0], dtype)
        assert (buf[:os] == 3).all() and (buf[os + n:] == 3).all()


def test_layouts():
    """Transposed and permuted gradients are clipped as they lie."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    a = make([((30, 50), F32), ((4, 5, 6), BF)])
    g = [a[0].t(), a[1].permute(2, 0, 1)]
    want = [t.clone() for t in a]
    lce.clip_grad_norm(want, 1.0)
    norm = lce.clip_grad_norm(g, 1.0)
    assert abs(float(norm) - math.sqrt(1620)) < 200
    for x, y in zip(a, want):
        assert torch.equal(x, y)


def test_shared_norm_and_determinism():
    """The norm may come from elsewhere (a sum over processes); the same
    gradients give the same bits."""
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    g = make([((200003,), BF), ((999,), F32)])
    n = lce.grad_norm(g)
    for _ in range(3):
        assert torch.equal(lce.grad_norm(g), n)
    both = (n.square() * 2).sqrt()
    before = [t.clone() for t in g]
    lce.clip_grads(g, both, 1.0)
    for t, c in zip(g, ref.clip(before, float(both), 1.0)):
        near(t, c, t.dtype)


def test_overlaps_are_refused():
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    t = torch.ones(100, device="cuda")
    u = torch.ones(50, device="cuda")
    for grads, outs in (([t, t], None), ([t[:60], t[50:]], None),
                        ([t, u, t[10:20]], None), ([u], [t[20:70], u][:1]),):
        if outs is None:
            with pytest.raises(lce.LCEError, match="INVALID_ARG"):
                lce.clip_grad_norm(grads, 1.0)
        else:
            lce.clip_grad_norm(grads, 1e9, grads_out=outs)
    with pytest.raises(lce.LCEError, match="INVALID_ARG"):
        lce.clip_grad_norm([t[:50]], 1.0, grads_out=[t[25:75]])
    with pytest.raises(lce.LCEError, match="INVALID_ARG"):
        lce.clip_grad_norm([t[:50], t[50:]], 1.0, grads_out=[t[50:], t[:50]])
    with pytest.raises(lce.LCEError, match="INVALID_ARG"):
        lce.clip_grads([t], t[3], 1.0)
    assert (t == 1).all()
    # beside each other is apart
    lce.clip_grad_norm([t[:50], t[50:]], 1e9)
    assert float(lce.grad_norm([t, t])) == pytest.approx(math.sqrt(200))


def test_capture_and_streams():
    import chunked_lm_head_gemm_gb300 as lce
    require_gpu()
    shapes = [((40000,), BF), ((33, 77), F32), ((5,), F32)] * 40
    g = make(shapes)
    outs = [torch.empty_like(t) for t in g]
    lce.clip_grad_norm(g, 1.0, grads_out=outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = lce.clip_grad_norm(g, 1.0, grads_out=outs)
    for seed in (1, 2):
        for t, s in zip(g, make(shapes, seed=seed, std=seed)):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            mine = [torch.empty_like(t) for t in g]
            n = lce.clip_grad_norm(g, 1.0, grads_out=mine)
        side.synchronize()
        assert torch.equal(n, norm)
        for a, b in zip(outs, mine):
            assert torch.equal(a, b)
