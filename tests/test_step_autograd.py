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
def test_a_tangent_is_refused_by_the_norms(lib, kind, which, no_grad):  # noqa: F811
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
