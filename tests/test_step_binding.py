"""What the norms, the balance loss and the clipping refuse, without a GPU: the
Python calls before they reach the C ABI (host tensors that say they are on
one, a library that only records), and the C ABI before it touches a device."""
import ctypes
import math

import pytest
import torch

import chunked_lm_head_gemm_gb300 as lce
from chunked_lm_head_gemm_gb300 import _binding as B

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class OnGpu(torch.Tensor):
    @property
    def is_cuda(self):
        return True


def t(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_size"):
                return 4096
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(B, "load", lambda *a: rec)
    monkeypatch.setattr(B, "_lib", None)
    monkeypatch.setattr(B, "_stream_ptr", lambda device: 0)
    sizes = (B.norm_workspace_size, B.balance_workspace_size,
             B.grad_norm_workspace_size)
    for f in sizes:
        f.cache_clear()
    yield rec
    for f in sizes:
        f.cache_clear()


def meta(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype, device="meta")


def test_norm_inputs(lib):
    x, w = t(6, 16), t(16)
    for bad in (t(16), t(2, 3, 16), t(16, 6).t(), t(6, 32)[:, ::2],
                torch.zeros(6, 16)):
        with pytest.raises(ValueError, match="x must"):
            lce.layer_norm_forward(bad, w)
        with pytest.raises(ValueError, match="x must"):
            lce.rms_norm(bad, w)
    with pytest.raises(TypeError):
        lce.rms_norm_forward(t(6, 16, dtype=torch.float16), w)
    for bad in (t(15), t(1, 16), t(32)[::2], meta(16), torch.zeros(16)):
        with pytest.raises(ValueError, match="weight"):
            lce.layer_norm_forward(x, bad)
        with pytest.raises(ValueError, match="bias"):
            lce.layer_norm_forward(x, w, bad)
    with pytest.raises(ValueError, match="bias"):  # one type for both
        lce.layer_norm_forward(x, w, t(16, dtype=BF))
    for bad in (t(5, 16), t(6, 16, dtype=BF), t(16, 6).t(), meta(6, 16)):
        with pytest.raises(ValueError, match="y_out"):
            lce.layer_norm_forward(x, w, y_out=bad)
    assert not lib.calls
    y = t(6, 16)
    assert lce.layer_norm_forward(x, w, t(16), y_out=y)[0] is y
    assert lib.calls[-1][1][5] == B.LCE_F32
    lce.rms_norm_forward(t(6, 16, dtype=BF), t(16))
    assert lib.calls[-1][1][2] == B.LCE_BF16 and lib.calls[-1][1][5] == B.LCE_F32


def test_norm_backward_inputs(lib):
    x, w, m, r, dy = t(6, 16), t(16), t(6), t(6), t(6, 16)
    ok = dict(x=x, weight=w, mean=m, rstd=r, dy=dy)
    for name, bads in dict(dy=[t(6, 15), t(6, 16, dtype=BF), t(16, 6).t(),
                               meta(6, 16)],
                           rstd=[t(5), t(6, dtype=BF), t(12)[::2]],
                           mean=[t(7), t(6, 1), meta(6)]).items():
        for bad in bads:
            with pytest.raises(ValueError, match=name):
                lce.layer_norm_backward(**{**ok, name: bad})
    with pytest.raises(ValueError, match="dx_out"):
        lce.layer_norm_backward(**ok, dx_out=t(6, 17))
    with pytest.raises(TypeError, match="grad_dtype"):
        lce.layer_norm_backward(**ok, grad_dtype=torch.float16)
    for ws in (t(1, dtype=torch.uint8).expand(4096),
               meta(4096, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="workspace"):
            lce.rms_norm_backward(x, w, r, dy, workspace=ws)
    assert not lib.calls
    ws = t(2048, dtype=F32)
    lce.rms_norm_backward(x, w, r, dy, workspace=ws)
    assert lib.calls[-1][1][15] == 8192  # bytes, whatever the tensor's type
    dx, dw = lce.rms_norm_backward(x, w, r, dy, compute_dweight=False)
    assert dw is None and lib.calls[-1][1][14] is None  # no workspace


def test_balance_inputs(lib):
    z, e, m = t(6, 16), t(6, 2, dtype=I32), t(6, dtype=torch.bool)
    for bad in (t(16), t(16, 6).t(), torch.zeros(6, 16)):
        with pytest.raises(ValueError, match="logits"):
            lce.balance_forward(bad, e)
    for bad in (t(5, 2, dtype=I32), t(6, 2), t(6, dtype=I32),
                t(2, 6, dtype=I32).t()):
        with pytest.raises(ValueError, match="experts"):
            lce.balance_forward(z, bad)
        with pytest.raises(ValueError, match="experts"):
            lce.expert_counts(bad if bad.dim() == 1 else bad.float(), 16)
    for bad in (t(5, dtype=torch.bool), t(6), t(6, 1, dtype=torch.bool),
                t(12, dtype=torch.bool)[::2], meta(6, dtype=torch.bool)):
        with pytest.raises(ValueError, match="mask"):
            lce.balance_forward(z, e, mask=bad)
        with pytest.raises(ValueError, match="mask"):
            lce.balance_backward(z, t(16), t(), mask=bad)
        with pytest.raises(ValueError, match="mask"):
            lce.expert_counts(e, 16, mask=bad)
    with pytest.raises(ValueError, match="scoring"):
        lce.balance_forward(z, e, scoring="tanh")
    with pytest.raises(ValueError, match="slopes"):
        lce.balance_backward(z, t(15), t())
    with pytest.raises(ValueError, match="dloss"):
        lce.balance_backward(z, t(16), t(2))
    with pytest.raises(ValueError, match="dlogits_out"):
        lce.balance_backward(z, t(16), t(), dlogits_out=t(6, 15))
    with pytest.raises(ValueError, match="counts_out"):
        lce.expert_counts(e, 16, counts_out=t(16))
    assert not lib.calls
    lce.balance_forward(z, e, mask=m)
    lce.expert_counts(e, 16, m)
    assert len(lib.calls) == 2


def test_gradient_lists(lib, monkeypatch):
    g = [t(3, 4), t(5, dtype=BF)]
    with pytest.raises(ValueError, match="one device"):
        lce.grad_norm([meta(3), t(3)])
    with monkeypatch.context() as m:
        m.setattr(torch.Tensor, "get_device", lambda g: g.dim())
        with pytest.raises(ValueError, match="one device"):
            lce.grad_norm([t(3), t(3, 1)])
    with pytest.raises(ValueError, match="CUDA"):
        lce.grad_norm([torch.zeros(3)])
    with pytest.raises(TypeError, match="dtype"):
        lce.grad_norm([t(3, dtype=torch.float16)])
    for bad in (t(6)[::2], t(1, 4).expand(3, 4), t(4, 6)[:, :3]):
        with pytest.raises(ValueError, match="gaps"):
            lce.clip_grad_norm([bad], 1.0)
    for bad in (-1.0, math.nan):
        with pytest.raises(ValueError, match="max_norm"):
            lce.clip_grad_norm(g, bad)
        with pytest.raises(ValueError, match="max_norm"):
            lce.clip_grads(g, t(), bad)
    n = t()
    for outs in ([t(4, 4), t(5, dtype=BF)], [t(3, 4), t(5)],
                 [t(4, 3).t(), t(5, dtype=BF)],
                 [t(3, 4), t(5, dtype=torch.float16)]):
        with pytest.raises(ValueError, match="output"):
            lce.clip_grads(g, n, 1.0, grads_out=outs)
    with pytest.raises(ValueError, match="outputs for"):
        lce.clip_grads(g, n, 1.0, grads_out=g[:1])
    for bad in (t(2), t(dtype=torch.float64), meta(())):
        with pytest.raises(ValueError, match="norm"):
            lce.clip_grads(g, bad, 1.0)
    assert not lib.calls
    lce.clip_grads(g, n, 1.0, grads_out=[t(12), t(5, dtype=BF)])
    lce.clip_grad_norm([g[0].t(), g[1]], 1.0, grads_out=[t(3, 4).t(), g[1]])
    lce.clip_grad_norm([g[0].t(), g[1]], 1.0)
    name, args = lib.calls[-1]
    assert name == "lce_clip_grad_norm" and list(args[3]) == [12, 5]
    assert list(args[2]) == [B.LCE_F32, B.LCE_BF16]
    assert list(args[0]) == list(args[1]) == [x.data_ptr() for x in g]


def test_a_call_runs_with_its_tensors_device_current(monkeypatch):
    """Tensors on another device than the current one: the call is made with
    theirs current, on its stream."""
    seen = []

    class Guard:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            seen.append(("in", self.device.index))

        def __exit__(self, *exc):
            seen.append("out")

    class Lib:
        @staticmethod
        def f(*args):
            seen.append(args)
            return 0

    monkeypatch.setattr(B, "_lib", Lib)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream",
                        lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0,
                        raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    B._call("f", torch.device("cuda", 0), 1, 2)
    assert seen == [(1, 2, 100)]
    del seen[:]
    B._call("f", torch.device("cuda", 3), 1, 2)
    assert seen == [("in", 3), (1, 2, 103), "out"]


@pytest.fixture(scope="module")
def c():
    return lce.load(build_if_missing=True)


P = ctypes.c_void_p(0x1000)  # aligned, never dereferenced
ODD = ctypes.c_void_p(0x1001)
NULL = ctypes.c_void_p(0)


def test_c_norm(c):
    assert c.lce_norm_workspace_size(-1, 8) == 0
    assert c.lce_norm_workspace_size(8, 0) == 0
    assert c.lce_norm_workspace_size(8, (1 << 20) + 1) == 0
    assert c.lce_norm_workspace_size(0, 8) > 0

    def f(kind=0, x=P, dt=0, w=P, b=NULL, pdt=0, L=4, H=8, eps=1e-5, y=P,
          mean=NULL, rstd=NULL):
        return c.lce_norm_forward(kind, x, dt, w, b, pdt, L, H, eps, y, mean,
                                  rstd, NULL)

    for kw in (dict(kind=2), dict(x=NULL), dict(x=ODD), dict(w=ODD),
               dict(b=ODD), dict(L=-1), dict(L=(1 << 31) + 1), dict(H=0),
               dict(H=(1 << 20) + 1), dict(eps=-1.0), dict(eps=math.nan),
               dict(eps=math.inf), dict(y=NULL), dict(y=ODD),
               dict(mean=ctypes.c_void_p(0x1002)), dict(rstd=ODD),
               dict(kind=1, b=P), dict(kind=1, mean=P)):
        assert f(**kw) == B.LCE_ERR_INVALID_ARG, kw
    for kw in (dict(dt=2), dict(pdt=-1)):
        assert f(**kw) == B.LCE_ERR_UNSUPPORTED
    assert f(L=0, x=NULL, y=NULL) == B.LCE_OK

    def g(kind=0, x=P, dt=0, w=P, pdt=0, mean=P, rstd=P, dy=P, L=4, H=8, gdt=1,
          dx=P, dw=P, db=P, ws=P, n=1 << 20):
        return c.lce_norm_backward(kind, x, dt, w, pdt, mean, rstd, dy, L, H,
                                   gdt, dx, dw, db, ws, n, NULL)

    for kw in (dict(x=NULL), dict(dy=NULL), dict(rstd=NULL), dict(mean=NULL),
               dict(dx=NULL, dw=NULL, db=NULL), dict(dw=ODD), dict(db=ODD),
               dict(dx=ODD), dict(dy=ODD), dict(ws=NULL),
               dict(ws=ctypes.c_void_p(0x1008)), dict(kind=1),
               dict(kind=1, mean=NULL), dict(kind=1, db=NULL)):
        assert g(**kw) == B.LCE_ERR_INVALID_ARG, kw
    assert g(gdt=3) == B.LCE_ERR_UNSUPPORTED
    assert g(n=16) == B.LCE_ERR_WORKSPACE


def test_c_balance(c):
    for L, E in ((-1, 8), (8, 0), (8, 1025), ((1 << 30) + 1, 8)):
        assert c.lce_balance_workspace_size(L, E) == 0

    def f(z=P, dt=0, e=P, m=NULL, L=4, E=8, K=2, s=0, coef=1.0, loss=P,
          counts=P, slopes=P, ws=P, n=1 << 20):
        return c.lce_balance_forward(z, dt, e, m, L, E, K, s, coef, loss,
                                     counts, slopes, ws, n, NULL)

    for kw in (dict(z=NULL), dict(z=ODD), dict(e=NULL), dict(e=ODD), dict(L=-1),
               dict(E=0), dict(E=1025), dict(K=0), dict(K=33),
               dict(L=1 << 30, K=2), dict(s=2), dict(coef=math.nan),
               dict(coef=math.inf), dict(loss=NULL), dict(counts=ODD),
               dict(slopes=NULL), dict(ws=NULL), dict(ws=ODD)):
        assert f(**kw) == B.LCE_ERR_INVALID_ARG, kw
    assert f(dt=7) == B.LCE_ERR_UNSUPPORTED
    assert f(n=8) == B.LCE_ERR_WORKSPACE

    def g(z=P, dt=0, m=NULL, L=4, E=8, s=0, slopes=P, d=P, out=P):
        return c.lce_balance_backward(z, dt, m, L, E, s, slopes, d, out, NULL)

    for kw in (dict(z=NULL), dict(slopes=NULL), dict(d=NULL), dict(out=NULL),
               dict(out=ODD), dict(E=2000), dict(L=-2), dict(s=-1)):
        assert g(**kw) == B.LCE_ERR_INVALID_ARG, kw
    assert g(L=0, z=NULL, out=NULL) == B.LCE_OK
    for args in ((NULL, NULL, 4, 8, 2, P), (P, NULL, 4, 8, 2, NULL),
                 (ODD, NULL, 4, 8, 2, P), (P, NULL, 4, 1025, 2, P),
                 (P, NULL, 4, 8, 0, P), (P, NULL, 4, 8, 2, ODD)):
        assert c.lce_expert_counts(*args, NULL) == B.LCE_ERR_INVALID_ARG


def test_c_grads(c):
    assert c.lce_grad_norm_workspace_size(-1) == 0
    assert c.lce_grad_norm_workspace_size(0) > 0

    def table(rows):
        n = len(rows)
        return ((ctypes.c_void_p * n)(*[r[0] for r in rows]),
                (ctypes.c_void_p * n)(*[r[1] for r in rows]),
                (ctypes.c_int * n)(*[r[2] for r in rows]),
                (ctypes.c_int64 * n)(*[r[3] for r in rows]), n)

    def norm(rows, out=P, ws=P, size=1 << 20):
        g, _, d, s, n = table(rows)
        return c.lce_grad_norm(g, d, s, n, out, ws, size, NULL)

    def clip(rows, nrm=P, limit=1.0):
        g, o, d, s, n = table(rows)
        first = c.lce_clip_grads(g, o, d, s, n, nrm, limit, NULL)
        assert c.lce_clip_grad_norm(g, o, d, s, n, limit, nrm, P, 1 << 20,
                                    NULL) == first
        return first

    A, BB = 0x10000, 0x20000
    ok = [(A, A, 1, 100)]
    for rows in ([(0, A, 1, 4)], [(A + 2, A, 1, 4)], [(A, A, 1, -1)],
                 [(A, A, 1, (1 << 40) + 1)],
                 [(A, A, 1, 1 << 40), (BB, BB, 1, 1)]):
        assert norm(rows) == B.LCE_ERR_INVALID_ARG
        assert clip(rows) == B.LCE_ERR_INVALID_ARG
    assert norm([(A, A, 5, 4)]) == B.LCE_ERR_UNSUPPORTED
    assert norm(ok, out=NULL) == B.LCE_ERR_INVALID_ARG
    assert norm(ok, ws=NULL) == B.LCE_ERR_INVALID_ARG
    assert norm(ok, size=8) == B.LCE_ERR_WORKSPACE
    assert clip(ok, nrm=NULL) == B.LCE_ERR_INVALID_ARG
    g, o, d, s, n = table(ok)
    assert c.lce_clip_grad_norm(g, o, d, s, n, 1.0, P, NULL, 1 << 20,
                                NULL) == B.LCE_ERR_INVALID_ARG
    assert c.lce_clip_grad_norm(g, o, d, s, n, 1.0, P, P, 8,
                                NULL) == B.LCE_ERR_WORKSPACE
    for limit in (-1.0, math.nan):
        assert clip(ok, limit=limit) == B.LCE_ERR_INVALID_ARG
    for rows in ([(A, 0, 1, 4)], [(A, BB + 1, 0, 4)],
                 [(A, A, 1, 100), (A, A, 1, 100)],           # twice
                 [(A, A, 1, 100), (A + 396, A + 396, 1, 9)],  # one in another
                 [(A, A + 4, 1, 100)],                        # onto itself
                 [(A, BB, 1, 100), (BB + 8, BB + 4000, 1, 1)],
                 [(A, BB, 1, 9), (BB, A, 1, 9)],              # crosswise
                 [(A, A, 1, 100), (BB, A + 398, 0, 8)]):
        assert clip(rows) == B.LCE_ERR_INVALID_ARG, rows
    assert clip(ok, nrm=ctypes.c_void_p(A + 40)) == B.LCE_ERR_INVALID_ARG
