"""Numbers that come as tensors: what is kept per kind of call is found by their values, so a tensor that is
changed in place between two calls counts with what it holds at each.

Both sides are the same kernels on the same inputs, with the number as a float: the same bits."""
import pytest
import torch

from tensor_train_compressed_ttembeddingbag_amd import loss as L
from tensor_train_compressed_ttembeddingbag_amd.embedding import embedding, embedding_gradient

pytestmark = pytest.mark.gpu


def data():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    h = torch.randn(12, 32, device="cuda", generator=g)
    w = torch.randn(50, 32, device="cuda", generator=g)
    t = torch.randint(0, 50, (12,), device="cuda", generator=g)
    x = torch.randn(12, device="cuda", generator=g)
    return h, w, t, x


OFF = [0, 2, 5, 9, 12]
# a number's name, two values, and a call with it
CALLS = {
    "scale": (2.0, 6.0, lambda h, w, t, x, s: embedding(t, w, scale=s)),
    "scale of a gradient": (2.0, 6.0, lambda h, w, t, x, s: embedding_gradient(h, t, 50, scale=s)),
    "padding_idx": (3, 7, lambda h, w, t, x, s: embedding_gradient(h, t, 50, padding_idx=s)),
    "num_rows": (50, 60, lambda h, w, t, x, s: embedding_gradient(h, t, s)),
    "beta": (0.1, 0.5, lambda h, w, t, x, s: L.linear_preference(h, w, t, off(), beta=s)),
    "smoothing of pairs": (0.1, 0.5, lambda h, w, t, x, s: L.linear_preference(h, w, t, off(), label_smoothing=s)),
    "margin": (0.25, 0.5, lambda h, w, t, x, s: L.linear_preference(h, w, t, off(), margin=s)),
    "ignored targets": (3, 7, lambda h, w, t, x, s: L.linear_preference(h, w, t, off(), ignore_index=s)),
    "clip_low": (0.1, 0.4, lambda h, w, t, x, s: L.linear_policy(h, w, t, x, logp(h, w, t, x), clip_low=s)),
    "clip_high": (0.1, 0.4, lambda h, w, t, x, s: L.linear_policy(h, w, t, x, logp(h, w, t, x), clip_high=s)),
    "kl_coef": (0.1, 0.4, lambda h, w, t, x, s: L.linear_policy(h, w, t, x, None, x, kl_coef=s)),
    "temperature": (0.5, 2.0, lambda h, w, t, x, s: L.linear_policy(h, w, t, x, x, temperature=s)),
    "ignored actions": (3, 7, lambda h, w, t, x, s: L.linear_policy(h, w, t, x, ignore_index=s)),
    "smoothing": (0.1, 0.5, lambda h, w, t, x, s: L.linear_cross_entropy(h, w, t, label_smoothing=s)),
    "ignore_index": (3, 7, lambda h, w, t, x, s: L.linear_cross_entropy(h, w, t, ignore_index=s)),
    "temperature of a teacher": (0.5, 2.0, lambda h, w, t, x, s: L.linear_distillation(
        h, w, x.view(12, 1).expand(12, 3).contiguous(), t.view(12, 1).repeat(1, 3), temperature=s)),
}


def off():
    return torch.tensor(OFF, device="cuda")


def logp(h, w, t, x):
    """The policy's own, moved so that positions are clipped on both sides: their ratio is exp x, and x is
    their advantage too."""
    return -L.linear_cross_entropy(h, w, t, reduction="none") - x


@pytest.mark.parametrize("device", ["cpu", "cuda"])
@pytest.mark.parametrize("name", list(CALLS))
def test_changed_in_place(name, device):
    a, b, call = CALLS[name]
    h, w, t, x = data()
    t[0], t[1] = 3, 7  # (for the two that name a row)
    number = torch.tensor(a, dtype=torch.float64 if isinstance(a, float) else torch.int64, device=device)
    want_a, want_b = call(h, w, t, x, a), call(h, w, t, x, b)
    assert not torch.equal(want_a, want_b)
    assert torch.equal(call(h, w, t, x, number), want_a)
    number.fill_(b)
    assert torch.equal(call(h, w, t, x, number), want_b)


def test_a_scale_that_requires_a_gradient_is_refused():
    h, w, t, _ = data()
    s = torch.tensor(2.0, requires_grad=True)
    for f in (lambda: embedding(t, w, scale=s), lambda: embedding_gradient(h, t, 50, scale=s)):
        with pytest.raises(RuntimeError, match="scale gets no gradient"):
            f()
        with torch.no_grad():
            f()
