"""What autograd sees of the norms, the balance loss and the clipping, without a
GPU: host tensors that say they are on one, and a library that only records."""
import pytest
import torch
from torch.autograd import forward_ad

import chunked_lm_head_gemm_gb300 as lce
from tests.test_step_binding import I32, lib, t  # noqa: F401


@pytest.mark.parametrize("no_grad", [False, True])
@pytest.mark.parametrize("kind,which", [("layer", 0), ("layer", 1),
                                        ("layer", 2), ("rms", 0), ("rms", 1)])
def test_a_tangent_is_refused_by_the_norms(lib, kind,  # noqa: F811
                                           which, no_grad):
    """Forward mode has no formula here; a result without a tangent would stand
    for a derivative of zero."""
    with forward_ad.dual_level(), torch.set_grad_enabled(not no_grad):
        args = [t(6, 16), t(16), t(16)][:3 if kind == "layer" else 2]
        args[which] = forward_ad.make_dual(args[which],
                                           torch.ones_like(args[which]))
        assert not args[which].requires_grad
        with pytest.raises(NotImplementedError, match="jvp"):
            (lce.layer_norm if kind == "layer" else lce.rms_norm)(*args)


def test_a_tangent_is_refused_by_the_balance_loss(lib):  # noqa: F811
    with forward_ad.dual_level():
        z = forward_ad.make_dual(t(6, 16), t(6, 16))
        with pytest.raises(NotImplementedError, match="jvp"):
            lce.balance_loss(z, t(6, 2, dtype=I32))


def test_inside_a_dual_level_without_tangents(lib):  # noqa: F811
    with forward_ad.dual_level():
        assert lce.rms_norm(t(6, 16), t(16)).shape == (6, 16)
    assert lib.calls[-1][0] == "lce_norm_forward"
    assert lib.calls[-1][1][-2] is None  # serving: no statistics


BF, BOOL = torch.bfloat16, torch.bool


def written(call, *tensors):
    """Whether autograd counts `call` as a write of each tensor."""
    before = [x._version for x in tensors]
    call()
    return all(x._version > b for x, b in zip(tensors, before))


def test_outputs_of_the_norms_count_as_written(lib):  # noqa: F811
    x, w, r, y = t(6, 16), t(16), t(6), t(6, 16)
    assert written(lambda: lce.layer_norm_forward(x, w, y_out=y), y)
    assert written(lambda: lce.rms_norm_forward(x, w, y_out=x), x)
    assert written(lambda: lce.layer_norm_backward(x, w, r, r, y, dx_out=y), y)
    assert written(lambda: lce.rms_norm_backward(x, w, r, y, dx_out=x), x)
    assert not written(lambda: lce.rms_norm_forward(x, w), x)


def test_outputs_of_the_routing_count_as_written(lib):  # noqa: F811
    z, e, c = t(6, 16), t(6, 2, dtype=I32), t(16, dtype=I32)
    k = t(6, 2)
    assert written(lambda: lce.balance_backward(z, t(16), t(), dlogits_out=z),
                   z)
    assert written(lambda: lce.expert_counts(e, 16, counts_out=c), c)
    assert written(lambda: lce.route_forward(z, 2, weights_out=k,
                                             experts_out=e), k, e)
    assert written(lambda: lce.route_backward(z, e, k, dlogits_out=z), z)


def test_clipped_gradients_count_as_written(lib):  # noqa: F811
    g = [t(3, 4), t(5, dtype=BF)]
    outs = [t(3, 4), t(5, dtype=BF)]
    assert written(lambda: lce.clip_grad_norm(g, 1.0), *g)
    assert written(lambda: lce.clip_grads(g, t(), 1.0), *g)
    assert written(lambda: lce.clip_grad_norm(g, 1.0, grads_out=outs), *outs)
    assert written(lambda: lce.clip_grads([None] + g, t(), 1.0,
                                          grads_out=[None] + outs), *outs)
    assert not written(lambda: lce.grad_norm(g), *g)
    assert not written(lambda: lce.clip_grad_norm(g, 1.0, grads_out=outs), g[0])


def test_other_outputs_count_as_written(lib):  # noqa: F811
    h, W, n = t(6, 16), t(8, 16), t(dtype=torch.int64)
    y = t(6, dtype=torch.int64)
    loss, lse, dH, dW = t(), t(6), t(6, 16), t(8, 16)
    ws = t(64, dtype=torch.uint8)
    kw = dict(workspace=ws)
    assert written(lambda: lce.forward(h, W, y, loss_out=loss, lse_out=lse,
                                       **kw), loss, lse)
    assert written(lambda: lce.backward(h, W, y, lse, t(), dH_out=dH,
                                        dW_out=dW, **kw), dH, dW)
    assert written(lambda: lce.forward_backward(
        h, W, y, loss_out=loss, lse_out=lse, dH_out=dH, dW_out=dW, **kw),
        loss, lse, dH, dW)
    assert written(lambda: lce.scale_gradients(dH, dW, t()), dH, dW)
    assert written(lambda: lce.scale_gradients(None, dW, t()), dW)
    assert written(lambda: lce.count_valid(y, 8, out=n), n)
    x, G, D = t(6, 16, dtype=BF), t(8, 16, dtype=BF), t(16, 8, dtype=BF)
    o, f, d = t(6, 16, dtype=BF), t(8, 16), t(16, 8)
    assert written(lambda: lce.mlp_forward(x, G, G, D, y_out=o, **kw), o)
    assert written(lambda: lce.mlp_backward(x, G, G, D, o, dx_out=o, dWg_out=f,
                                            dWu_out=W, dWd_out=d, **kw),
                   o, f, W, d)


def test_a_saved_tensor_that_is_clipped_is_an_error(lib):  # noqa: F811
    leaf = t(5).requires_grad_(True)
    g = leaf * 2
    loss = g.square().sum()  # keeps g
    lce.clip_grad_norm([g.detach()], 1.0)
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
