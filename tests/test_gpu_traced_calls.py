"""What of a traced call is refused and what works, on the GPU."""
import pytest
import torch
from torch.fx.experimental.proxy_tensor import make_fx

from tensor_train_compressed_ttembeddingbag_amd import loss as L
from tensor_train_compressed_ttembeddingbag_amd.embedding import embedding
from tensor_train_compressed_ttembeddingbag_amd.quant import int8_linear, quantize_rows

pytestmark = pytest.mark.gpu


def test_calls_without_gradients_are_refused():
    h, w = torch.randn(4, 8, device="cuda"), torch.randn(20, 8, device="cuda")
    t, rows = torch.arange(4, device="cuda"), quantize_rows(w)
    for f in (lambda h: int8_linear(h, rows), lambda h: L.linear_policy(h, w, t, h[:, 0]),
              lambda h: embedding(t, rows) + h):
        with pytest.raises(RuntimeError, match="cannot be traced"):
            torch.jit.trace(f, (h,))
        with pytest.raises(RuntimeError, match="cannot be traced"):
            make_fx(f)(h)
        f(h)


def test_backwards_are_refused_under_make_fx():
    h = torch.randn(4, 8, device="cuda", requires_grad=True)
    w, t = torch.randn(20, 8, device="cuda", requires_grad=True), torch.arange(4, device="cuda")
    for out in (embedding(t, w), L.linear_cross_entropy(h, w, t, reduction="none"),
                L.linear_policy(h, w, t, h[:, 0], reduction="none")):
        with pytest.raises(RuntimeError, match="cannot be traced"):
            make_fx(lambda g: torch.autograd.grad(out, w, g, retain_graph=True))(torch.ones_like(out))
        torch.autograd.grad(out, w, torch.ones_like(out))


@pytest.mark.parametrize("grad", [False, True])
def test_rows_are_recorded(grad):
    """As their autograd function, which takes other numbers of tokens; not under make_fx."""
    w = torch.randn(20, 8, device="cuda", requires_grad=grad)
    with pytest.raises(RuntimeError, match="cannot be traced"):
        make_fx(lambda t: embedding(t, w))(torch.arange(4, device="cuda"))
    f = torch.jit.trace(lambda t, w: embedding(t, w, scale=2.0), (torch.arange(4, device="cuda"), w))
    t = torch.tensor([3, 3, 19], device="cuda")
    out = f(t, w)
    assert torch.equal(out, 2 * w[t])
    if not grad:
        return
    out.sum().backward()
    assert bool((w.grad[3] == 4).all()) and bool((w.grad[19] == 2).all()) and not bool(w.grad[0].any())
