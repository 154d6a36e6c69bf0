"""Routing on the GPU against its float64 reference.

Tolerances, fixed before the first run: the selection is exact. A score is
within 2^-19 of its value (relative), so a renormalised weight is within
3 * 2^-19, and is rounded once to its type (eps / 2). A gradient element is a
product of a score and a difference of terms up to max |u|, each within a few
2^-19: 16 * 2^-19 * score * max |u|, and one rounding."""
import math

import numpy as np
import pytest
import torch

from tests import sparse_ref as ref
from tests.gpu_util import require_gpu, to64

pytestmark = pytest.mark.gpu

SCORE = 2.0 ** -19


def draw(L, E, dtype, seed, masked=0.0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(L, E, generator=g) * spread
    if masked:
        off = torch.rand(L, E, generator=g) < masked
        z = z.masked_fill(off, -math.inf)
    return z.to(dtype)


def check(z, dev, top_k, bias=None, seed=0, **kw):
    """Forward and backward of CPU logits z against the reference."""
    import chunked_lm_head_gemm_gb300 as lce
    zd = z.to(dev)
    bd = None if bias is None else bias.to(dev)
    w, e = lce.route_forward(zd, top_k, bias=bd, **kw)
    rb = None if bias is None else bias.double().numpy()
    rw, re_ = ref.route(to64(z), top_k, bias=rb, **kw)
    assert np.array_equal(e.cpu().numpy(), re_)
    half = torch.finfo(z.dtype).eps / 2
    got = to64(w)
    nan = np.isnan(rw)
    assert np.array_equal(np.isnan(got), nan)
    assert (np.abs(got - rw)[~nan] <=
            (np.abs(rw) * (3 * SCORE + half) + 1e-37)[~nan]).all()
    grad = {k: kw[k] for k in ("scoring", "renormalize", "scale") if k in kw}
    dw = torch.randn(z.shape[0], top_k,
                     generator=torch.Generator().manual_seed(seed + 99))
    dw = dw.to(z.dtype)
    dz = to64(lce.route_backward(zd, e, dw.to(dev), **grad))
    assert lce.get_error() == 0
    scoring = kw.get("scoring", "softmax")
    scale = kw.get("scale", 1.0)
    rz = ref.route_grad(to64(z), re_, to64(dw), scoring,
                        kw.get("renormalize", True), scale)
    for i in range(z.shape[0]):
        if np.isnan(rz[i]).any():
            continue
        s = np.nan_to_num(ref.scores(to64(z[i]), scoring))
        if kw.get("renormalize", True):
            t = s[re_[i]].sum()
            s = s / t if t else s
        u = np.abs(scale * to64(dw[i])).max()
        tol = 16 * SCORE * s * u + np.abs(rz[i]) * half + 1e-37
        assert (np.abs(dz[i] - rz[i]) <= tol).all(), i


SHAPES = [  # L, E, K, dtype, masked
    (1, 1, 1, torch.float32, 0), (1, 128, 8, torch.bfloat16, 0),
    (3, 5, 5, torch.float32, 0.3), (130, 60, 4, torch.bfloat16, 0.2),
    (33, 127, 7, torch.float32, 0), (65, 128, 1, torch.bfloat16, 0),
    (40, 250, 32, torch.float32, 0), (17, 256, 8, torch.bfloat16, 0.1),
    (9, 511, 3, torch.float32, 0), (9, 512, 16, torch.bfloat16, 0),
    (5, 1000, 10, torch.float32, 0.5), (6, 1024, 32, torch.bfloat16, 0)]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("L,E,K,dtype,masked", SHAPES)
def test_shapes(L, E, K, dtype, masked, biased, scoring):
    dev = require_gpu()
    z = draw(L, E, dtype, seed=E + K, masked=masked)
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(1)) \
        if biased else None
    for renorm in (True, False):
        check(z, dev, K, bias=bias, scoring=scoring, renormalize=renorm,
              scale=2.5)


GROUPS = [  # E, K, groups, kept, group_top
    (64, 6, 8, 3, 1), (64, 6, 8, 3, 2), (256, 8, 8, 4, 2), (60, 4, 5, 2, 2),
    (21, 2, 7, 1, 1), (96, 6, 32, 4, 2), (1024, 8, 16, 2, 2), (10, 3, 10, 4, 1),
    (24, 8, 3, 3, 2), (250, 5, 2, 1, 2)]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("E,K,G,kept,top", GROUPS)
def test_groups(E, K, G, kept, top, biased, scoring):
    dev = require_gpu()
    z = draw(37, E, torch.float32, seed=E, masked=0.15)
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(2)) \
        if biased else None
    check(z, dev, K, bias=bias, scoring=scoring, n_group=G, topk_group=kept,
          group_top=top)


@pytest.mark.parametrize("groups", [dict(), dict(n_group=4, topk_group=2,
                                                 group_top=2)],
                         ids=["flat", "groups"])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_keys_closer_than_fp32(scoring, groups):
    """The bias makes every key of a row 1 up to the bias's own rounding, so
    the order is decided by differences near 2^-25 that fp32 scores cannot
    see; and once more with whole rows of equal inputs (exact ties)."""
    dev = require_gpu()
    E = 64
    z = draw(1, E, torch.float32, seed=5)
    bias = torch.from_numpy(1.0 - ref.scores(to64(z[0]), scoring)).float()
    z = z.expand(50, E).contiguous()
    check(z, dev, 8, bias=bias, scoring=scoring, **groups)
    check(torch.zeros(3, E), dev, 8, bias=torch.zeros(E), scoring=scoring,
          **groups)
    z = draw(200, E, torch.bfloat16, seed=6, spread=0.05)  # many equal logits
    check(z, dev, 8, bias=torch.zeros(E), scoring=scoring, **groups)
    check(z, dev, 8, scoring=scoring, **groups)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_rows_that_are_masked_or_not_finite(scoring, renorm):
    dev = require_gpu()
    E, inf, nan = 12, math.inf, math.nan
    z = draw(8, E, torch.float32, seed=7)
    z[0] = -inf                          # nothing left
    z[1, 1:] = -inf                      # one expert left
    z[2] = torch.finfo(torch.float32).min
    z[3, 4] = nan
    z[4, :6] = -inf
    z[5] = -200.0                        # sigmoid scores underflow
    z[6] = 300.0
    z[7, 0], z[7, 1] = -0.0, 0.0
    kw = dict(scoring=scoring, renormalize=renorm)
    check(z, dev, 4, **kw)
    bias = torch.zeros(E)
    bias[3], bias[5], bias[6] = -inf, inf, inf
    check(z, dev, 4, bias=bias, **kw)
    check(z, dev, 4, bias=bias, n_group=3, topk_group=2, group_top=2, **kw)
    check(z, dev, 4, n_group=3, topk_group=2, group_top=2, **kw)


def test_addresses_and_streams():
    """Rows off 16-byte addresses, another stream, and repeated calls give
    the bits of the aligned call; strided logits are refused."""
    dev = require_gpu()
    import chunked_lm_head_gemm_gb300 as lce
    z = draw(300, 64, torch.bfloat16, seed=8).to(dev)
    w, e = lce.route_forward(z, 6)
    dz = lce.route_backward(z, e, w)
    flat = torch.empty(300 * 64 + 1, dtype=z.dtype, device=dev)
    zz = flat[1:].view(300, 64)
    zz.copy_(z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w2, e2 = lce.route_forward(zz, 6)
        dz2 = lce.route_backward(zz, e2, w2)
    side.synchronize()
    assert torch.equal(w, w2) and torch.equal(e, e2) and torch.equal(dz, dz2)
    with pytest.raises(ValueError, match="contiguous"):
        lce.route_forward(z.t(), 6)
    with pytest.raises(lce.LCEError):
        lce.route_forward(z, 65)
    assert lce.get_error() == 0


def test_empty_and_bad_indices():
    dev = require_gpu()
    import chunked_lm_head_gemm_gb300 as lce
    from chunked_lm_head_gemm_gb300 import _binding as B
    w, e = lce.route_forward(torch.empty(0, 16, device=dev), 2)
    assert w.shape == (0, 2) and e.shape == (0, 2)
    z = draw(4, 16, torch.float32, seed=9).to(dev)
    e = torch.tensor([[1, 2], [16, 3], [4, 5], [-7, 6]], dtype=torch.int32,
                     device=dev)
    dw = torch.ones(4, 2, device=dev)
    dz = lce.route_backward(z, e, dw, scoring="sigmoid", renormalize=False)
    assert lce.get_error() == B.LCE_ERR_EXPERT_RANGE
    assert lce.get_error() == 0
    s = ref.scores(to64(z), "sigmoid")
    want = np.zeros((4, 16))
    for i, j in ((0, 1), (0, 2), (1, 3), (2, 4), (2, 5), (3, 6)):
        want[i, j] = s[i, j] * (1 - s[i, j])
    assert np.allclose(to64(dz), want, rtol=1e-5, atol=0)


def test_autograd_and_graph():
    """route_experts under autograd equals the explicit calls; a captured
    forward and backward replays with new logits."""
    dev = require_gpu()
    import chunked_lm_head_gemm_gb300 as lce
    z = draw(64, 32, torch.float32, seed=10).to(dev)
    leaf = z.clone().requires_grad_(True)
    w, e = lce.route_experts(leaf, 4, "sigmoid", scale=2.0)
    dw = torch.randn_like(w)
    w.backward(dw)
    want = lce.route_backward(z, e, dw, "sigmoid", scale=2.0)
    assert torch.equal(leaf.grad, want) and not e.requires_grad
    zs = z.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w2, e2 = lce.route_forward(zs, 4, "sigmoid", scale=2.0)
        dz2 = lce.route_backward(zs, e2, dw, "sigmoid", scale=2.0)
    z3 = draw(64, 32, torch.float32, seed=11).to(dev)
    zs.copy_(z3)
    g.replay()
    w3, e3 = lce.route_forward(z3, 4, "sigmoid", scale=2.0)
    assert torch.equal(w2, w3) and torch.equal(e2, e3)
    assert torch.equal(dz2, lce.route_backward(z3, e3, dw, "sigmoid",
                                               scale=2.0))
    assert lce.get_error() == 0


MANY = [  # E, K, dtype, kwargs, biased
    (128, 8, torch.bfloat16, dict(), False),
    (128, 8, torch.bfloat16, dict(renormalize=False), True),
    (60, 4, torch.float32, dict(scoring="sigmoid"), True),
    (61, 5, torch.bfloat16, dict(scoring="sigmoid", renormalize=False), False),
    (3, 3, torch.float32, dict(), True), (1, 1, torch.float32, dict(), False),
    (512, 8, torch.float32, dict(), True), (511, 1, torch.bfloat16, {}, False),
    (256, 8, torch.float32, dict(scoring="sigmoid", n_group=8, topk_group=4,
                                 group_top=2), True),
    (256, 6, torch.bfloat16, dict(n_group=8, topk_group=3, group_top=1), False),
    (96, 6, torch.float32, dict(n_group=32, topk_group=5, group_top=2), False),
    (105, 7, torch.float32, dict(n_group=7, topk_group=2, group_top=2), True),
    (250, 8, torch.bfloat16, dict(scoring="sigmoid", n_group=2, topk_group=1,
                                  group_top=2), False)]


@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("E,K,dtype,kw,biased", MANY)
def test_many_rows_like_few(E, K, dtype, kw, biased, masked):
    """4099 rows in one call (eight rows to a warp) choose the experts that
    calls on 700 of them choose (a warp to a row, tested above against the
    reference), with the same weights up to the two computations' scores;
    rows that are masked, infinite, NaN or all equal among them."""
    dev = require_gpu()
    import chunked_lm_head_gemm_gb300 as lce
    L, inf = 4099, math.inf
    z = draw(L, E, dtype, seed=E + 1, masked=masked)
    z[5] = -inf
    z[6, : E // 2] = -inf
    z[7, 0] = inf
    z[8, E - 1] = math.nan
    z[9] = 0.25
    z[10] = -200.0
    z[4098] = torch.finfo(dtype).min
    z[4000:4090] = z[4000:4090].round()  # many ties
    z = z.to(dev)
    biases = [None]
    if biased:
        g = torch.Generator().manual_seed(4)
        b = 0.1 * torch.randn(E, generator=g)
        c = b.clone()
        c[0], c[E // 2] = inf, -inf
        flat = 1.0 - torch.from_numpy(ref.scores(
            to64(z[11].cpu()), kw.get("scoring", "softmax"))).float()
        biases = [b.to(dev), torch.zeros(E, device=dev), c.to(dev),
                  torch.nan_to_num(flat).to(dev)]
        z[12:40] = z[11]
    for bias in biases:
        w, e = lce.route_forward(z, K, bias=bias, **kw)
        for i in range(0, L, 700):
            part = z[i:i + 700].contiguous()
            w2, e2 = lce.route_forward(part, K, bias=bias, **kw)
            assert torch.equal(e[i:i + 700], e2)
            a, b = to64(w[i:i + 700]), to64(w2)
            assert np.array_equal(np.isnan(a), np.isnan(b))
            tol = np.abs(b) * (6 * SCORE + torch.finfo(dtype).eps) + 1e-37
            assert (np.nan_to_num(np.abs(a - b)) <= np.nan_to_num(tol)).all()
    assert lce.get_error() == 0


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("E,G,kept", [(32, 8, 2), (12, 6, 3), (96, 32, 5),
                                      (21, 7, 2)])
def test_infinite_biases_in_many_rows(E, G, kept, top, scoring):
    """Experts that an infinite bias forces (or bars), among groups so small
    that all their experts are candidates, in a call of many rows: one forced
    expert, two of one group, three of different groups, some masked."""
    dev = require_gpu()
    inf = math.inf
    z = draw(3001, E, torch.float32, seed=E + top, masked=0.2)
    for forced in ([E - 1], [E - 2, E - 1], [0, E // 2, E - 1]):
        bias = 0.1 * torch.randn(E,
                                 generator=torch.Generator().manual_seed(6))
        bias[forced] = inf
        bias[1] = -inf
        check(z, dev, 4, bias=bias, scoring=scoring, n_group=G,
              topk_group=kept, group_top=top)


HAMMER = r"""
#include <pthread.h>
#include <stdint.h>
typedef int (*route_fn)(const void*, int, const float*, int64_t, int64_t,
                        const void*, void*, int32_t*, void*);
struct call {
  route_fn f;
  const void* logits;
  int64_t L, E;
  const void* opts;
  void *weights, *experts, *stream;
  int64_t times, refused;
};
static void* run(void* p) {
  struct call* c = p;
  for (int64_t i = 0; i < c->times; ++i)
    c->refused += c->f(c->logits, 1, 0, c->L, c->E, c->opts, c->weights,
                       c->experts, c->stream) != 0;
  return 0;
}
void hammer(struct call* calls, int n) {
  pthread_t t[16];
  for (int i = 0; i < n; ++i) pthread_create(&t[i], 0, run, &calls[i]);
  for (int i = 0; i < n; ++i) pthread_join(t[i], 0);
}
"""


def test_group_ranks_of_different_sizes_from_many_threads(tmp_path):
    """A call whose group ranks need more shared memory is not refused
    because another thread queues calls that need less. (Threads of a C
    helper: Python's meet too seldom inside the calls.)"""
    import ctypes
    import subprocess
    dev = require_gpu()
    import chunked_lm_head_gemm_gb300 as lce
    from chunked_lm_head_gemm_gb300 import _binding as B
    (tmp_path / "hammer.c").write_text(HAMMER)
    so = tmp_path / "hammer.so"
    subprocess.run(["gcc", "-O2", "-shared", "-fPIC", "-pthread", "-o", so,
                    tmp_path / "hammer.c"], check=True)

    class Call(ctypes.Structure):
        _fields_ = [(n, ctypes.c_void_p) for n in ("f", "logits")] + [
            (n, ctypes.c_int64) for n in ("L", "E")] + [
            (n, ctypes.c_void_p) for n in ("opts", "weights", "experts",
                                           "stream")] + [
            (n, ctypes.c_int64) for n in ("times", "refused")]
    f = ctypes.cast(lce.load().lce_route_forward, ctypes.c_void_p).value
    keep, calls = [], (Call * 8)()
    for i in range(8):
        E, G = ((1020, 30), (884, 26))[i % 2]
        z = draw(64, E, torch.float32, seed=E).to(dev)
        want = lce.route_forward(z, 8, n_group=G, topk_group=4, group_top=2)
        got = [torch.empty_like(t) for t in want]
        opts = B.RouteOpts(0, 8, G, 4, 2, 1, 1.0)
        stream = torch.cuda.Stream()
        keep.append((z, want, got, opts, stream))
        calls[i] = Call(f, z.data_ptr(), 64, E, ctypes.addressof(opts),
                        got[0].data_ptr(), got[1].data_ptr(),
                        stream.cuda_stream, 10000, 0)
    torch.cuda.synchronize()
    ctypes.CDLL(str(so)).hammer(calls, 8)
    torch.cuda.synchronize()
    assert [c.refused for c in calls] == [0] * 8
    for _, want, got, _, _ in keep:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert lce.get_error() == 0


@pytest.mark.parametrize("E", [512, 1000], ids=["many", "few"])
def test_a_large_score_just_below_the_border(E):
    """Softmax scores with a bias, top 1: two experts whose keys are their
    biases (no score to speak of), 2^-23 apart, and right below them one with
    half the row's mass, whose fp32 key is off by more than that. The row is
    searched for: of 20000, the one whose fp32 score falls furthest short."""
    dev = require_gpu()
    import chunked_lm_head_gemm_gb300 as lce
    L = 20000
    d = torch.linspace(math.log(E) - 0.7, math.log(E) + 0.7, L)
    z = -d[:, None].expand(L, E).contiguous()
    z[:, 0] = 0.0
    z[:, [40, 80]] = -60.0
    w, e = lce.route_forward(z.to(dev), 1, renormalize=False)
    assert (e == 0).all()
    score = 1.0 / (1.0 + (E - 3) * np.exp(-to64(d)) + 2 * math.exp(-60.0))
    short = score - to64(w)[:, 0]
    i = int(short.argmax())
    gap = 1.25e-7
    assert short[i] > 1.02 * gap  # else the row shows nothing
    bias = torch.full((E,), -10.0)
    bias[0], bias[40], bias[80] = -w[i, 0].cpu(), gap, 2.0 ** -40
    assert ref.select(to64(z[i]), 1, bias=bias.double().numpy()) == [0]
    _, e = lce.route_forward(z[i].expand(L, E).contiguous().to(dev), 1,
                             bias=bias.to(dev))
    assert (e == 0).all()
    assert lce.get_error() == 0
