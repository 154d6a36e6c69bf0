"""More of what the operators around a step refuse and take, without a GPU: the
C ABI before it touches a device, the Python calls on host tensors that say they
are on one."""
import ctypes

import pytest
import torch

import chunked_lm_head_gemm_gb300 as lce
from chunked_lm_head_gemm_gb300 import _binding as B
from tests.test_step_binding import BF, NULL, P, c, lib, t  # noqa: F401

A, BB, CC = 0x10000, 0x20000, 0x30000


def clip_grad_norm(c, rows, norm):  # noqa: F811
    """lce_clip_grad_norm of (gradient, output, type, elements), with no
    workspace, which is looked at behind the pointers that overlap."""
    n = len(rows)
    return c.lce_clip_grad_norm(
        (ctypes.c_void_p * n)(*[r[0] for r in rows]),
        (ctypes.c_void_p * n)(*[r[1] for r in rows]),
        (ctypes.c_int * n)(*[r[2] for r in rows]),
        (ctypes.c_int64 * n)(*[r[3] for r in rows]), n, 1.0,
        ctypes.c_void_p(norm), P, 8, NULL)


@pytest.mark.parametrize("norm", [A, A + 40, A + 396, BB, BB + 196])
def test_the_norm_may_not_be_written_into_a_gradient(c, norm):  # noqa: F811
    """Gradients with outputs of their own: blocks still read them while the
    norm is written."""
    rows = [(A, CC, 1, 100), (BB, CC + 400, 0, 100)]
    assert clip_grad_norm(c, rows, norm) == B.LCE_ERR_INVALID_ARG


@pytest.mark.parametrize("norm", [A - 4, A + 400, BB - 4, BB + 200])
def test_the_norm_may_stand_beside_a_gradient(c, norm):  # noqa: F811
    rows = [(A, CC, 1, 100), (BB, CC + 400, 0, 100)]
    assert clip_grad_norm(c, rows, norm) == B.LCE_ERR_WORKSPACE


def test_an_empty_gradient_holds_no_norm(c):  # noqa: F811
    rows = [(A, CC, 1, 100), (BB, BB, 1, 0)]
    assert clip_grad_norm(c, rows, BB) == B.LCE_ERR_WORKSPACE


@pytest.mark.parametrize("shape", [(3, 0), (0, 3), (2, 0, 4), (0,)])
def test_empty_gradients_beside_transposed_ones(lib, shape):  # noqa: F811
    """An empty tensor fills its memory whatever its strides."""
    for empty in (t(*shape), t(*shape).permute(*range(len(shape))[::-1])):
        lce.clip_grad_norm([t(4, 6).t(), empty], 1.0)
        assert list(lib.calls[-1][1][3]) == [24, 0]
        lce.grad_norm([empty, t(4, 6).t()])
    with pytest.raises(ValueError, match="gaps"):
        lce.grad_norm([t(6)[::2], t(*shape)])


def test_parameters_without_a_gradient(lib):  # noqa: F811
    """[p.grad for p in parameters] has None for a parameter that took no part:
    it is passed by, and has no output."""
    g = [t(3, 4), t(5, dtype=BF)]
    outs = [t(3, 4), t(5, dtype=BF)]
    mixed, mixed_outs = [None, g[0], None, g[1]], [None, outs[0], None, outs[1]]
    lce.grad_norm(mixed)
    lce.clip_grads(mixed, t(), 1.0)
    lce.clip_grad_norm(mixed, 1.0)
    lce.clip_grad_norm(mixed, 1.0, grads_out=mixed_outs)
    for name, args in lib.calls:
        n = args[args.index(2)]
        assert n == 2 and list(args[0]) == [x.data_ptr() for x in g], name
    assert list(lib.calls[-1][1][1]) == [x.data_ptr() for x in outs]
    del lib.calls[:]
    for bad in ([outs[0], outs[0], None, outs[1]], [None, outs[0], None, None],
                outs):
        with pytest.raises(ValueError, match="output"):
            lce.clip_grad_norm(mixed, 1.0, grads_out=bad)
    assert not lib.calls


@pytest.mark.parametrize("L,H,slabs", [(16384, 65536, 132),
                                       (131072, 32768, 210),
                                       (131072, 4096, 750), (5, 65536, 5),
                                       (1 << 31, 8192, 1024)])
def test_the_norms_workspace_is_near_its_use(c, L, H, slabs):  # noqa: F811
    """Two sums of H columns for each of the blocks or clusters that a launch
    may have: rows of many columns have few. On 152 SMs 1024 threads of 16
    columns each are 38 rows of 65536 at a time, 76 of 32768, 608 of 4096;
    runs of 16384 / 128 + 48 = 176 rows are 93 of 16384 and runs of 1024 are
    128 of 131072, and one or a 64th of the rows at a time is rounding: 132,
    206, 746."""
    size = c.lce_norm_workspace_size(L, H)
    assert 0 < size <= slabs * 2 * H * 4
