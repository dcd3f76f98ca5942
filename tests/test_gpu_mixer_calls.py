"""What the mixer calls refuse on CUDA tensors, beyond their shapes and types."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    from linear_attention_recurrent_gdn_gb300 import build
    build.build()
    from linear_attention_recurrent_gdn_gb300 import mixer
    return mixer


def test_forward_mode_tensors_are_refused(mx):
    fwd = torch.autograd.forward_ad
    x, w = torch.ones(2, 64, device="cuda"), torch.ones(64, device="cuda")
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        for call in (lambda: mx.add_norm(dual, None, w), lambda: mx.add_norm(x, dual, w),
                     lambda: mx.gated_norm(dual.view(2, 1, 64), w)):
            with pytest.raises(ValueError, match="differentiated"):
                call()
        y, _ = mx.add_norm(x, None, w)
    assert torch.equal(y, mx.add_norm(x, None, w)[0])


def test_unknown_activations_and_norms_are_refused(mx):
    x, w = torch.ones(2, 4, 64, device="cuda"), torch.ones(64, device="cuda")
    for call in (lambda: mx.conv(x, torch.ones(64, 4, device="cuda"), activation="relu"),
                 lambda: mx.gated_norm(x, w, x, activation="gelu"), lambda: mx.gated_norm(x, w, kind="batch"),
                 lambda: mx.add_norm(x[0], None, w, kind=0)):
        with pytest.raises(ValueError, match="expected one of"):
            call()
