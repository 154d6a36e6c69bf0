"""A run of the operators as a training step has them: RMS norm, router,
route_experts with its balance loss, experts_mlp, residual, layer norm, the
head's loss, backward, clip_grad_norm; its loss and every gradient against the
same step in float64 autograd. Tolerance: along a path some twelve values are
rounded to bf16, each by at most 2^-8 of itself, 4.7e-2 together."""
import importlib.util
import math
import os

import pytest
import torch

from tests.gpu_util import require_gpu

pytestmark = pytest.mark.gpu

STEP = 12 * 2.0 ** -8
L, H, I, E, K, V = 320, 128, 64, 8, 2, 640


def leaves(dev):
    g = torch.Generator(device=dev).manual_seed(11)

    def normal(*shape, std):
        return (torch.randn(*shape, device=dev, generator=g) * std).bfloat16()

    x = normal(L, H, std=1.0)
    labels = torch.randint(0, V, (L,), device=dev, generator=g)
    w = dict(n1=1 + normal(H, std=0.1), Wr=normal(E, H, std=H ** -0.5),
             Wg=normal(E, I, H, std=H ** -0.5),
             Wu=normal(E, I, H, std=H ** -0.5),
             Wd=normal(E, H, I, std=I ** -0.5), n2=1 + normal(H, std=0.1),
             b2=normal(H, std=0.1), head=normal(V, H, std=0.1))
    return x, labels, w


def step(x, labels, w):
    """The step's loss with its graph, and the chosen experts."""
    import chunked_lm_head_gemm_gb300 as lce
    xn = lce.rms_norm(x, w["n1"])
    z = xn @ w["Wr"].t()
    weights, experts = lce.route_experts(z, K)
    aux, counts = lce.balance_loss(z, experts, coef=0.5)
    h = x + lce.experts_mlp(xn, w["Wg"], w["Wu"], w["Wd"], weights, experts)
    h = lce.layer_norm(h, w["n2"], w["b2"])
    return lce.linear_cross_entropy(h, w["head"], labels) + aux, experts, counts


def reference(x, labels, w, experts):
    d = {k: v.detach().double().requires_grad_(True) for k, v in w.items()}
    x = x.double()
    xn = x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-6) * d["n1"]
    z = xn @ d["Wr"].t()
    p = torch.softmax(z, 1)
    e = experts.long()
    s = p.gather(1, e)
    s = s / s.sum(1, keepdim=True)
    counts = torch.bincount(e.flatten(), minlength=E)
    aux = 0.5 * (counts * E / (L * K) * p.mean(0)).sum()
    g = torch.einsum("lh,lkih->lki", xn, d["Wg"][e])
    u = torch.einsum("lh,lkih->lki", xn, d["Wu"][e])
    a = torch.nn.functional.silu(g) * u
    h = x + torch.einsum("lk,lki,lkhi->lh", s, a, d["Wd"][e])
    h = h - h.mean(1, keepdim=True)
    h = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-5)
    h = h * d["n2"] + d["b2"]
    loss = torch.nn.functional.cross_entropy(h @ d["head"].t(), labels)
    (loss + aux).backward()
    total = float((loss + aux).detach())
    return total, {k: v.grad for k, v in d.items()}, counts


def test_a_training_step():
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    x, labels, w = leaves(dev)
    for v in w.values():
        v.requires_grad_(True)
    total, experts, counts = step(x, labels, w)
    total.backward()
    assert lce.get_error() == 0
    want, grads, rcounts = reference(x, labels, w, experts)
    assert torch.equal(counts.long(), rcounts)
    assert abs(float(total.detach()) - want) <= 1e-2 * want
    for k, v in w.items():
        e = (v.grad.double() - grads[k]).norm() / grads[k].norm()
        assert e <= STEP, (k, float(e))
    got = [v.grad for v in w.values()]
    before = [t.clone() for t in got]
    norm = lce.clip_grad_norm(got, 0.01)
    whole = math.sqrt(sum(float(t.square().sum()) for t in grads.values()))
    assert abs(float(norm) - whole) <= STEP * whole
    for t, b in zip(got, before):
        c = b.double() * min(1.0, 0.01 / (float(norm) + 1e-6))
        assert ((t.double() - c).abs() <= c.abs() * 1.01 * 2.0 ** -8).all()


def test_a_training_step_in_a_graph():
    """The step with its backward pass and the clipping, captured once and
    replayed, gives the eager step's bits."""
    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    x, labels, w = leaves(dev)

    def run():
        leaf = {k: v.detach().requires_grad_(True) for k, v in w.items()}
        total, _, counts = step(x, labels, leaf)
        grads = list(torch.autograd.grad(total, list(leaf.values())))
        norm = lce.clip_grad_norm(grads, 0.01)
        return [total.detach(), counts, norm, *grads]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)
    assert lce.get_error() == 0


def test_calls_at_once():
    """The same calls on four streams and threads at a time give the bits of
    one after the other."""
    import threading

    import chunked_lm_head_gemm_gb300 as lce
    dev = require_gpu()
    g = torch.Generator(device=dev).manual_seed(5)
    x = torch.randn(3000, 1000, device=dev, generator=g)
    z = torch.randn(3000, 64, device=dev, generator=g)
    w = torch.rand(1000, device=dev, generator=g)
    e = torch.topk(z, 4, dim=1).indices.int()
    one = torch.ones((), device=dev)

    def calls():
        y, mean, rstd = lce.layer_norm_forward(x, w, w)
        grads = lce.layer_norm_backward(x, w, mean, rstd, y)
        loss, counts, slopes = lce.balance_forward(z, e)
        dz = lce.balance_backward(z, slopes, one)
        outs = [torch.empty_like(t) for t in grads]
        norm = lce.clip_grad_norm(grads, 1.0, grads_out=outs)
        return [y, *grads, loss, counts, dz, norm, *outs]

    want = calls()
    torch.cuda.synchronize()
    got = [None] * 4

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got[i] = calls()
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for out in got:
        for a, b in zip(out, want):
            assert torch.equal(a, b)
    assert lce.get_error() == 0


@pytest.mark.parametrize("kw", [dict(norm="rms", balance=0.01, max_norm=1.0),
                                dict(norm="layer"), dict(max_norm=0.1)])
def test_example_options_run(kw):
    require_gpu()
    path = os.path.join(os.path.dirname(os.path.dirname(
        os.path.abspath(__file__))), "examples", "sparse_mlp_step.py")
    spec = importlib.util.spec_from_file_location("sparse_mlp_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.run(steps=2, **kw)
    assert len(losses) == 2 and all(math.isfinite(v) for v in losses)
