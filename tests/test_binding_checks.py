"""What the Python calls of the sparse MLP check before they reach the C ABI,
without a GPU: host tensors that say they are on one, and a library that only
records what it is given."""
import pytest
import torch

import chunked_lm_head_gemm_gb300 as lce
from chunked_lm_head_gemm_gb300 import _binding as B


class OnGpu(torch.Tensor):
    @property
    def is_cuda(self):
        return True


def t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)


class Recorder:
    def __init__(self):
        self.calls = []

    def lce_experts_workspace_size(self, *args):
        return 4096

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(B, "load", lambda *a: rec)
    monkeypatch.setattr(B, "_stream_ptr", lambda device: 0)
    B.experts_workspace_size.cache_clear()
    yield rec
    B.experts_workspace_size.cache_clear()


BF, I32 = torch.bfloat16, torch.int32


def bad(*shape, dtype):
    """Tensors that are not a contiguous `dtype` tensor of `shape`."""
    n, m = shape
    other = torch.float64 if dtype is not torch.float64 else torch.float32
    return [t(n - 1, m, dtype=dtype), t(n, m + 1, dtype=dtype),
            t(n * m, dtype=dtype), t(n, m, dtype=other),
            t(m, n, dtype=dtype).t(), t(n, 1, dtype=dtype).expand(n, m),
            torch.zeros(n, m, dtype=dtype, device="meta")]


def test_output_tensors_of_the_routing(lib):
    z, e, dw = t(6, 16), t(6, 4, dtype=I32), t(6, 4)
    for out in bad(6, 4, dtype=torch.float32):
        with pytest.raises(ValueError, match="weights_out"):
            lce.route_forward(z, 4, weights_out=out)
    for out in bad(6, 4, dtype=I32):
        with pytest.raises(ValueError, match="experts_out"):
            lce.route_forward(z, 4, experts_out=out)
    for out in bad(6, 16, dtype=torch.float32):
        with pytest.raises(ValueError, match="dlogits_out"):
            lce.route_backward(z, e, dw, dlogits_out=out)
    assert not lib.calls
    w, i, dz = t(6, 4), t(6, 4, dtype=I32), t(6, 16)
    assert lce.route_forward(z, 4, weights_out=w, experts_out=i) == (w, i)
    assert lce.route_backward(z, e, dw, dlogits_out=dz) is dz
    assert len(lib.calls) == 2


def test_output_and_workspace_of_the_experts(lib):
    x, W, Wd = t(6, 16, dtype=BF), t(3, 8, 16, dtype=BF), t(3, 16, 8, dtype=BF)
    args = (x, W, W, Wd, t(6, 2), t(6, 2, dtype=I32))
    for out in bad(6, 16, dtype=BF):
        with pytest.raises(ValueError, match="y_out"):
            lce.experts_forward(*args, y_out=out)
    for ws in (t(1, dtype=torch.uint8).expand(4096),
               t(8192, dtype=torch.uint8)[::2],
               torch.zeros(4096, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            lce.experts_forward(*args, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            lce.experts_backward(*args, x, workspace=ws)
    assert not lib.calls
    y, ws = t(6, 16, dtype=BF), t(4096, dtype=torch.uint8)
    assert lce.experts_forward(*args, workspace=ws, y_out=y) is y
    lce.experts_backward(*args, x, workspace=ws)
    assert len(lib.calls) == 2


def test_host_tensors_are_refused_before_the_library(monkeypatch):
    """Calls that take their stream from a tensor's device refuse a host
    tensor, as does a stream of a device that is none."""
    rec = Recorder()
    monkeypatch.setattr(B, "load", lambda *a: rec)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0,
                        raising=False)
    one = torch.ones(1)
    with pytest.raises(ValueError, match="CUDA"):
        B.shard_sums(one, torch.ones(1, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        B.scale_gradients(torch.ones(2, 8), None, one)
    with pytest.raises(ValueError, match="CUDA"):
        B.tc_gemm(one, one, 1, 1, 1, False, False)
    with pytest.raises(ValueError, match="CUDA"):
        B.get_error("cpu")
    assert not rec.calls


def test_options_are_the_values_at_the_call(lib):
    """A scale that lives in a tensor is read at each call, and options that
    the C struct cannot hold are refused, not cut to 32 bits."""
    z, e, dw = t(6, 16), t(6, 4, dtype=I32), t(6, 4)
    scale = torch.tensor(2.5)
    for value in (2.5, 4.0):
        scale.fill_(value)
        lce.route_forward(z, 4, scale=scale)
        lce.route_backward(z, e, dw, scale=scale)
        assert lib.calls[-2][1][5].contents.scale == value
        assert lib.calls[-1][1][6].contents.scale == value
    n = len(lib.calls)
    for kw in (dict(n_group=2 ** 32 + 1), dict(topk_group=2 ** 32 + 1),
               dict(group_top=1 - 2 ** 32)):
        with pytest.raises(ValueError, match="32 bits"):
            lce.route_forward(z, 4, **kw)
    with pytest.raises(ValueError, match="scoring"):
        lce.route_forward(z, 4, scoring="tanh")
    assert len(lib.calls) == n
