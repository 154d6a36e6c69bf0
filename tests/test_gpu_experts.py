"""The experts' gated MLP on the GPU against its float64 reference.

Tolerances, fixed before the first run: relative Frobenius errors. A rounding
to bf16 is off by at most 2^-8 of the value; y and dx carry two of them that
are independent (a, or dg and du; the result), a bf16 weight gradient two, an
fp32 one one, dweights only its own. The rest is fp32: sums of at most some
thousand products, 2^-24 each way, and the logistic function at 2^-21."""
import math

import numpy as np
import pytest
import torch

from tests import sparse_ref as ref
from tests.gpu_util import PAIRS, cta_pair, rel_fro, require_gpu, to64

pytestmark = pytest.mark.gpu

R = 2.0 ** -8
F32 = 2.0 ** -15
NAMES = ("x", "Wg", "Wu", "Wd", "w", "e")


def draw(dev, L, H, I, E, K, seed=0, wdt=torch.bfloat16, drop=0.0, idx=None):
    g = torch.Generator().manual_seed(seed)
    bf = torch.bfloat16

    def n(*s):
        return torch.randn(*s, generator=g)
    x, dy = n(L, H).to(bf), n(L, H).to(bf)
    Wg, Wu = (n(E, I, H).mul(H ** -0.5).to(bf) for _ in range(2))
    Wd = n(E, H, I).mul(I ** -0.5).to(bf)
    w = torch.rand(L, K, generator=g).to(wdt)
    e = n(L, E).topk(K, dim=1).indices.to(torch.int32)
    if drop:
        e = e.masked_fill(torch.rand(L, K, generator=g) < drop, -1)
    if idx is not None:
        e = idx.to(torch.int32)
    return [t.to(dev) for t in (x, Wg, Wu, Wd, w, e)], dy.to(dev)


def dirty(nbytes, dev):
    """A workspace whose old contents are NaN in every type."""
    return torch.full((nbytes,), 0xff, dtype=torch.uint8, device=dev)


def run(args, dy, grad_dtype=torch.float32):
    import chunked_lm_head_gemm_gb300 as lce
    L, K = args[5].shape
    E, I, H = args[1].shape
    dev = args[0].device
    y = lce.experts_forward(*args, workspace=dirty(
        lce.experts_workspace_size(L, H, I, E, K), dev))
    grads = lce.experts_backward(*args, dy, grad_dtype=grad_dtype,
                                 workspace=dirty(lce.experts_workspace_size(
                                     L, H, I, E, K, True), dev))
    return (y, *grads)


def compare(got, args, dy):
    want = ref.experts_mlp(*[to64(t) if t.is_floating_point() else
                             t.cpu().numpy() for t in args], to64(dy))
    wr = R if args[4].dtype == torch.bfloat16 else F32
    gr = math.sqrt(2) * R if got[2].dtype == torch.bfloat16 else R + F32
    tol = (math.sqrt(2) * R, math.sqrt(2) * R, gr, gr, gr, wr)
    for name, g, r, t in zip(("y", "dx", "dWg", "dWu", "dWd", "dw"), got,
                             want, tol):
        err = rel_fro(to64(g), r)
        assert err <= t + F32, f"{name} rel Frobenius err {err}"


SHAPES = [  # L, H, I, E, K
    (1, 8, 8, 1, 1), (1, 64, 40, 4, 2), (2, 8, 8, 32, 32), (5, 72, 136, 3, 3),
    (64, 128, 64, 1, 1), (65, 64, 128, 2, 1), (130, 128, 256, 16, 4),
    (200, 264, 328, 5, 2), (700, 512, 192, 8, 2), (257, 1000, 424, 10, 2),
    (40, 64, 64, 1024, 4), (3000, 64, 72, 7, 4), (33, 2048, 768, 12, 8)]


@pytest.mark.parametrize("wdt", [torch.bfloat16, torch.float32],
                         ids=["bf16", "f32"])
@pytest.mark.parametrize("L,H,I,E,K", SHAPES)
def test_shapes(L, H, I, E, K, wdt):
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    args, dy = draw(dev, L, H, I, E, K, seed=L + E, wdt=wdt)
    compare(run(args, dy, wdt), args, dy)
    assert lce.get_error() == 0


@pytest.mark.parametrize("pair", PAIRS, ids=lambda v: "pair" if v else "cta")
@pytest.mark.parametrize("L,H,I,E,K", [
    (600, 264, 328, 1, 1), (1100, 136, 72, 2, 1), (2600, 512, 768, 3, 2),
    (4000, 1000, 424, 4, 2), (5000, 72, 8, 9, 4)])
def test_many_rows_to_an_expert(L, H, I, E, K, pair):
    """Enough rows that CTA pairs take the contractions, and the same on
    single CTAs."""
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    args, dy = draw(dev, L, H, I, E, K, seed=L, drop=0.02)
    with cta_pair(pair):
        compare(run(args, dy, torch.bfloat16), args, dy)
        compare(run(args, dy), args, dy)
    assert lce.get_error() == 0


def _indices(kind, L, E, K):
    g = torch.Generator().manual_seed(4)
    e = torch.randint(0, E, (L, K), generator=g)
    if kind == "one_expert":
        e[:] = E - 1
    elif kind == "dropped":
        e[:] = -1
    elif kind == "half_dropped":
        e[::2] = -1
    elif kind == "one_slot":
        e[:] = -1
        e[L // 2, K - 1] = 2
    elif kind == "same_twice":
        e[:, 1] = e[:, 0]
    return e


@pytest.mark.parametrize("L", [4, 300, 4500])
@pytest.mark.parametrize("kind", ["one_expert", "dropped", "half_dropped",
                                  "one_slot", "same_twice"])
def test_uneven_routing(kind, L):
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    args, dy = draw(dev, L, 72, 136, 5, 2, seed=3,
                    idx=_indices(kind, L, 5, 2))
    got = run(args, dy)
    compare(got, args, dy)
    if kind == "dropped":
        assert all((t == 0).all() for t in got)
    assert lce.get_error() == 0


@pytest.mark.parametrize("L", [3, 500])
def test_bad_indices_are_dropped_and_reported(L):
    dev = require_gpu()
    import chunked_lm_head_gemm_gb300 as lce
    from chunked_lm_head_gemm_gb300 import _binding as B
    args, dy = draw(dev, L, 64, 64, 4, 2, seed=5)
    args[5][1, 0], args[5][2, 1] = 4, -2
    y = lce.experts_forward(*args)
    assert lce.get_error() == B.LCE_ERR_EXPERT_RANGE
    got = (y, *lce.experts_backward(*args, dy))
    assert lce.get_error() == B.LCE_ERR_EXPERT_RANGE
    compare(got, args, dy)
    assert lce.get_error() == 0


@pytest.mark.parametrize("L", [2, 200])
def test_not_finite_stays_in_its_place(L):
    """A dropped token's NaN reaches nothing, a kept token's only its own
    row and the gradients of the experts it visits; a NaN weight of a dropped
    slot reaches nothing."""
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    args, dy = draw(dev, L, 64, 72, 6, 2, seed=6)
    e = torch.randint(0, 5, (L, 2), generator=torch.Generator().manual_seed(1))
    e[0] = -1
    e[1] = 5
    args[5] = e.to(torch.int32).to(dev)
    base = run(args, dy)
    x = args[0].clone()
    x[0] = math.nan
    args[4][0] = math.nan
    again = run([x, *args[1:]], dy)
    for a, b in zip(base, again):
        assert torch.equal(a, b)
    x[1, 3] = math.inf
    again = run([x, *args[1:]], dy)
    keep = torch.ones(L, dtype=torch.bool, device=dev)
    keep[1] = False
    for i in (0, 1, 5):
        assert torch.equal(base[i][keep], again[i][keep])
    for i in (2, 3, 4):
        assert torch.equal(base[i][:5], again[i][:5])
    assert not torch.isfinite(again[0][1]).all()
    assert lce.get_error() == 0


def test_infinite_weight_of_an_expert_with_one_row():
    """Infinities come out where the definition has them: the rows that pad
    an expert's single one add none and no NaN."""
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    args, dy = draw(dev, 200, 64, 72, 6, 1, seed=8)
    e = torch.randint(0, 5, (200, 1),
                      generator=torch.Generator().manual_seed(2))
    e[1] = 5
    args[5] = e.to(torch.int32).to(dev)
    args[3][5, 3, 7] = math.inf
    got = run(args, dy)
    with np.errstate(invalid="ignore"):
        want = ref.experts_mlp(*[to64(t) for t in args[:5]],
                               args[5].cpu().numpy(), to64(dy))
    assert np.isinf(want[2][5, 7]).all() and np.isinf(want[3][5, 7]).all()
    for name, a, r in zip(("y", "dx", "dWg", "dWu", "dWd", "dw"), got, want):
        a = to64(a)
        wild = ~np.isfinite(r)
        assert np.array_equal(np.isnan(a), np.isnan(r)), name
        assert np.array_equal(a[wild], r[wild], equal_nan=True), name
    assert lce.get_error() == 0


@pytest.mark.parametrize("L", [1, 7, 600])
def test_same_bits_on_another_stream_and_in_a_graph(L):
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    args, dy = draw(dev, L, 128, 136, 8, 2, seed=7)
    base = run(args, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run(args, dy)
    side.synchronize()
    for a, b in zip(base, other):
        assert torch.equal(a, b)
    ws = dirty(lce.experts_workspace_size(L, 128, 136, 8, 2, True), dev)
    static = [t.clone() for t in args]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lce.experts_forward(*static, workspace=ws)
        grads = lce.experts_backward(*static, dy, workspace=ws)
    args2, _ = draw(dev, L, 128, 136, 8, 2, seed=8)
    for s, t in zip(static, args2):
        s.copy_(t)
    g.replay()
    for a, b in zip((y, *grads), run(args2, dy)):
        assert torch.equal(a, b)
    assert lce.get_error() == 0


def test_optional_gradients():
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    args, dy = draw(dev, 300, 64, 136, 6, 2, seed=9)
    full = lce.experts_backward(*args, dy)
    flags = ("compute_dx", "compute_dWgu", "compute_dWd", "compute_dweights")
    parts = {"compute_dx": (0,), "compute_dWgu": (1, 2), "compute_dWd": (3,),
             "compute_dweights": (4,)}
    for only in flags:
        got = lce.experts_backward(*args, dy, **{f: f == only for f in flags})
        for i in range(5):
            if i in parts[only]:
                assert torch.equal(got[i], full[i])
            else:
                assert got[i] is None
    with pytest.raises(lce.LCEError):
        lce.experts_backward(*args, dy, **{f: False for f in flags})
    assert lce.get_error() == 0


def test_no_tokens():
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    args, dy = draw(dev, 0, 64, 72, 3, 2, idx=torch.empty(0, 2))
    y = lce.experts_forward(*args)
    dx, dWg, dWu, dWd, dw = lce.experts_backward(*args, dy)
    assert y.shape == dx.shape == (0, 64) and dw.shape == (0, 2)
    assert all((t == 0).all() for t in (dWg, dWu, dWd))
    assert lce.get_error() == 0


def test_autograd_layer():
    """Router and experts together, as a layer under autograd: the gradients
    of sum(y dy) equal the explicit calls'."""
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    (x, Wg, Wu, Wd, _, _), dy = draw(dev, 200, 128, 136, 8, 2, seed=10)
    z = torch.randn(200, 8, generator=torch.Generator().manual_seed(3))
    z = z.to(torch.bfloat16).to(dev)
    leaves = [t.clone().requires_grad_(True) for t in (x, Wg, Wu, Wd, z)]
    w, e = lce.route_experts(leaves[4], 2)
    y = lce.experts_mlp(*leaves[:4], w, e)
    y.backward(dy)
    w2, e2 = lce.route_forward(z, 2)
    want = lce.experts_backward(x, Wg, Wu, Wd, w2, e2, dy,
                                grad_dtype=torch.bfloat16)
    for leaf, g in zip(leaves, want):
        assert torch.equal(leaf.grad, g) or leaf is leaves[4]
    assert torch.equal(leaves[4].grad, lce.route_backward(z, e2, want[4]))
    frozen = [t.detach() for t in leaves[1:4]]
    xx = x.clone().requires_grad_(True)
    lce.experts_mlp(xx, *frozen, w2, e2).backward(dy)
    assert torch.equal(xx.grad, want[0])
    with pytest.raises(ValueError, match="contiguous"):
        lce.experts_forward(x.t(), Wg, Wu, Wd, w2, e2)
    assert lce.get_error() == 0


def test_rows_past_32_bit_offsets():
    """Intermediate rows times columns past 2^31: sampled tokens against the
    reference, forward and dx."""
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    L, H, I, E, K = 280000, 2048, 64, 4, 4
    assert L * K * H > 1 << 31
    (x, Wg, Wu, Wd, _, _), _ = draw(dev, 8, H, I, E, K, seed=11)
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(L, H, device=dev, generator=g, dtype=torch.bfloat16)
    w = torch.rand(L, K, device=dev, generator=g)
    e = torch.rand(L, E, device=dev, generator=g).argsort(1).to(torch.int32)
    y = lce.experts_forward(x, Wg, Wu, Wd, w, e)
    dx = lce.experts_backward(x, Wg, Wu, Wd, w, e, x, compute_dWgu=False,
                              compute_dWd=False)[0]
    assert lce.get_error() == 0
    at = torch.tensor([0, 1, 139999, 262143, 262144, L - 2, L - 1], device=dev)
    args = [to64(t) for t in (x[at], Wg, Wu, Wd, w[at])]
    want = ref.experts_mlp(*args, e[at].cpu().numpy(), to64(x[at]))
    assert rel_fro(to64(y[at]), want[0]) <= 2 * R
    assert rel_fro(to64(dx[at]), want[1]) <= 2 * R


def test_layer_captured_with_its_backward():
    """Router, experts and their gradients through autograd inside a captured
    graph; the replay gives the eager gradients' bits. (The eager graph is
    freed first: while one is alive, torch keeps the leaves' accumulation on
    the stream it was built on, and no captured backward may depend on it.)"""
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    (x, Wg, Wu, Wd, _, _), dy = draw(dev, 300, 128, 136, 8, 2, seed=12)
    z = torch.randn(300, 8, device=dev)
    leaves = [t.requires_grad_(True) for t in (x, Wg, Wu, Wd, z)]

    def layer():
        w, e = lce.route_experts(leaves[4], 2)
        return lce.experts_mlp(*leaves[:4], w, e)
    y = layer()
    want = torch.autograd.grad(y, leaves, dy)
    y_want = y.detach()
    del y
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(layer(), leaves, dy)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
        grads = torch.autograd.grad(y, leaves, dy)
    graph.replay()
    assert torch.equal(y, y_want)
    for a, b in zip(grads, want):
        assert torch.equal(a, b)
    assert lce.get_error() == 0


def test_example_step():
    """examples/sparse_mlp_step.py: router, experts and the head's loss train
    together."""
    import importlib.util
    import os
    require_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(
        os.path.abspath(__file__))), "examples", "sparse_mlp_step.py")
    spec = importlib.util.spec_from_file_location("sparse_mlp_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.run(steps=6)
    assert len(losses) == 6 and all(math.isfinite(v) for v in losses)
    assert losses[-1] < losses[0]


def _child(code):
    """Runs `code` in a process of its own, in which no earlier call has
    changed a kernel's limits."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, timeout=300,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("E,L", [(384, 109), (384, 120), (384, 433),
                                 (384, 480), (1024, 40), (1024, 160)])
def test_plans_near_the_default_shared_memory(E, L):
    """Counters of the one-block plan that fit 48 KB alone but not beside the
    kernel's static arrays, as the first call of a process."""
    require_gpu()
    _child("from tests import test_gpu_experts as t\n"
           "import chunked_lm_head_gemm_gb300 as lce\n"
           "dev = t.require_gpu()\n"
           f"args, dy = t.draw(dev, {L}, 64, 8, {E}, 8, seed={L})\n"
           "t.compare(t.run(args, dy), args, dy)\n"
           "assert lce.get_error() == 0\n")


def test_plans_of_different_sizes_from_many_threads():
    """A plan of more shared memory is not refused because another thread
    queues smaller ones."""
    import threading
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    lib, work, refused = lce.load(), [], []
    for L in (128, 64) * 4:
        args, _ = draw(dev, L, 8, 8, 1024, 8, seed=L)
        want = lce.experts_forward(*args)
        ws = dirty(lce.experts_workspace_size(L, 8, 8, 1024, 8), dev)
        y = torch.empty_like(want)
        call = (*(t.data_ptr() for t in args[:5]), 0, args[5].data_ptr(), L, 8,
                8, 1024, 8, y.data_ptr(), ws.data_ptr(), ws.numel(),
                torch.cuda.Stream().cuda_stream)
        work.append((args, ws, want, y, call))
    torch.cuda.synchronize()

    def loop(call):  # the C call alone, so that the threads meet inside it
        for _ in range(2000):
            status = lib.lce_experts_forward(*call)
            if status:
                refused.append(status)
    threads = [threading.Thread(target=loop, args=(w[4],)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, (len(refused), refused[0])
    for _, _, want, y, _ in work:
        assert torch.equal(y, want)
    assert lce.get_error() == 0


def test_second_derivatives_are_refused():
    """The gradients carry no graph of their own: differentiating them again
    is an error, not a missing term."""
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    (x, Wg, Wu, Wd, w, e), _ = draw(dev, 20, 64, 72, 4, 2, seed=13)
    x.requires_grad_(True)
    z = torch.randn(20, 4, device=dev, requires_grad=True)
    for leaf, out in ((x, lce.experts_mlp(x, Wg, Wu, Wd, w, e)),
                      (z, lce.route_experts(z, 2)[0])):
        g, = torch.autograd.grad((out.float() ** 2).sum(), leaf,
                                 create_graph=True)
        loss = (g.float() ** 2).sum() + (leaf.float() ** 2).sum()
        with pytest.raises(RuntimeError, match="twice"):
            loss.backward()
    assert lce.get_error() == 0
