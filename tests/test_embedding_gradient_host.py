"""``embedding_gradient`` has no derivatives of its own: what asks for them is refused, not dropped."""
import pytest
import torch
from torch.autograd import forward_ad

from tensor_train_compressed_ttembeddingbag_amd.embedding import embedding_gradient

I4 = torch.zeros(4, dtype=torch.int64)


def test_a_gradient_that_requires_one_is_refused():
    up = torch.zeros(4, 8, requires_grad=True)
    with pytest.raises(RuntimeError, match="no gradient"):
        embedding_gradient(up, I4, 20)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):  # as any other
        embedding_gradient(up, I4, 20)
    with pytest.raises(ValueError, match="GPU"):
        embedding_gradient(up.detach(), I4, 20)


def test_dual_tensors_are_refused():
    with forward_ad.dual_level():
        up = forward_ad.make_dual(torch.zeros(4, 8), torch.ones(4, 8))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            embedding_gradient(up, I4, 20)
