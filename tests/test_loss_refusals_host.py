"""What the vocabulary-head losses refuse before any device work: forward-mode derivatives, which
would be dropped, and temperatures that float32 does not hold."""
import pytest
import torch
from torch.autograd import forward_ad

from tensor_train_compressed_ttembeddingbag_amd import loss as L


@pytest.mark.parametrize("which", ["hidden", "weight"])
@pytest.mark.parametrize("grad", [False, True])
def test_dual_tensors_are_refused(which, grad):
    h, w = torch.zeros(4, 8, requires_grad=grad), torch.zeros(20, 8, requires_grad=grad)
    t = torch.zeros(4, dtype=torch.int64)
    with forward_ad.dual_level():
        if which == "hidden":
            h = forward_ad.make_dual(h, torch.ones(4, 8))
        else:
            w = forward_ad.make_dual(w, torch.ones(20, 8))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            L.linear_cross_entropy(h, w, t)
        with pytest.raises(NotImplementedError, match="forward-mode"):
            L.linear_distillation(h, w, torch.zeros(4, 3), torch.zeros(4, 3, dtype=torch.int64))
        with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
            L.linear_cross_entropy(h[None], w, t[None])


@pytest.mark.parametrize("temperature", [1e-50, 1e39, float("inf"), -1.0])
def test_temperatures_outside_float32_are_refused(temperature):
    """The library takes a float32: what rounds to 0 or infinity there is the caller's mistake."""
    with pytest.raises(ValueError, match="temperature"):
        L.linear_distillation(torch.zeros(4, 8), torch.zeros(20, 8), torch.zeros(4, 3),
                              torch.zeros(4, 3, dtype=torch.int64), temperature=temperature)
