"""Distillation entries: their logits are the ones in the position's sum, so what the products'
rounding does to a logit is the same on both sides of a divergence, and lists of any length and
order, with repeated rows."""
import math

import pytest
import torch

from tensor_train_compressed_ttembeddingbag_amd import loss as L
from test_gpu_loss_range import DT, check, inputs, lowest_values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n", [3, 70])
@pytest.mark.parametrize("k", [1, 5])
def test_confident_students(k, n, dt):
    """A teacher with all weight on one row (given once or five times) that the student agrees
    with: divergences of 1e-4 to 1e-2, with logits of 20.  As for cross entropy a loss is off by
    the sum's own rounding, 2^-20, and by the logits' errors times the others' share."""
    print("case confident", k, n, dt, flush=True)
    v, d = 4000, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    w = (torch.randn(v, d, device="cuda", generator=g) * d ** -0.5).to(DT[dt])
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    h = (w[t].float() * (15.0 + 3 * torch.rand(n, 1, device="cuda", generator=g))).to(DT[dt])
    ref = torch.nn.functional.cross_entropy(h.double() @ w.double().t(), t, reduction="none")
    assert float(ref.min()) < 2e-2
    dz = 2 * (d * 2.0 ** -24 + (2.0 ** -21 if dt == "fp32" else 0)) * \
        (h.double().abs() @ w.double().abs().t()).amax(1)
    # five entries share the weight: their own softmax's log is off by 2^-22
    bound = 2.0 ** -20 + ref * dz + (2.0 ** -21 if k > 1 else 0)
    idx, tl = t[:, None].expand(n, k), torch.zeros(n, k, device="cuda")
    ent = -math.log(k)  # of the entries as they are given
    got = L.linear_distillation(h, w, tl, idx, reduction="none").double() - ent
    assert float(((got - ref).abs() / bound).max()) <= 1
    x = h.detach().requires_grad_(True)
    assert torch.equal(L.linear_distillation(x, w, tl, idx, reduction="none").detach().double(),
                       got + ent)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("scale", [1.0, 8.0])
def test_matched_students(scale, dt):
    """A teacher of all rows whose logits are the student's own: the divergence is 0.  What the
    products' rounding leaves of it is of second order, dz^2, besides 2^-20 of the terms (lse and
    the logs) -- however large the logits are."""
    print("case matched", scale, dt, flush=True)
    n, v, d = 40, 128, 200
    h, w, _, _ = inputs(n, v, d, 5, dt)
    h = (h.float() * scale).to(DT[dt])
    z = h.double() @ w.double().t()
    idx = torch.arange(v, device="cuda").expand(n, v)
    got = L.linear_distillation(h, w, z.float(), idx, reduction="none").double()
    lp = torch.log_softmax(z, 1)
    ent = -(lp.exp() * lp).sum(1)
    dz = (d * 2.0 ** -24 + (2.0 ** -21 if dt == "fp32" else 0)) * \
        (h.double().abs() @ w.double().abs().t()).amax(1) + 2.0 ** -24 * z.abs().amax(1)
    assert float((got.abs() / (2.0 ** -20 * (1 + ent) + dz * dz)).max()) <= 1


@pytest.mark.parametrize("scale", [1.0, 12.0])
def test_gradient_of_the_logits_sums_to_zero(scale):
    """With a column of ones in the weight that no hidden state uses, dh there is the sum of the
    logits' gradient: 0, up to 2^-20 of its terms (exponentials, two parts of G) whatever the
    logits' size, as the entries' probabilities and the sum's come from the same logits."""
    print("case zero sum", scale, flush=True)
    n, v, d, k = 100, 3000, 129, 8
    h, w, t, g = inputs(n, v, d, 6)
    h = h * scale
    h[:, 128], w[:, 128] = 0, 1
    idx = (t[:, None] + torch.arange(k, device="cuda")) % v
    tl = torch.randn(n, k, device="cuda", generator=g)
    x = h.requires_grad_(True)
    dh, = torch.autograd.grad(L.linear_distillation(x, w, tl, idx, reduction="sum"), x)
    terms = 2.0  # sum of |p - q| is 2 at most
    assert float(dh[:, 128].abs().max()) <= 2.0 ** -20 * terms


@pytest.mark.parametrize("k", [63, 64, 65, 500, 2048])
@pytest.mark.parametrize("n", [5, 90])
def test_long_and_repeating_lists(n, k):
    """More entries than rows, in any order."""
    print("case long lists", n, k, flush=True)
    v, d = 300, 40
    for dt in ("bf16", "fp32"):
        h, w, _, g = inputs(n, v, d, k, dt)
        idx = torch.randint(0, v, (n, k), device="cuda", generator=g)
        idx[0] = 7
        tl = torch.randn(n, k, device="cuda", generator=g) * 2
        check(h, w, dt, tl=tl, idx=idx, T=1.3)
        # empty entries anywhere leave the others' result
        gap = torch.full((n, 2 * k), -1, device="cuda")
        gap[:, ::2] = idx
        if 2 * k <= 2048:
            a = L.linear_distillation(h, w, tl, idx, reduction="none")
            b = L.linear_distillation(h, w, tl.repeat_interleave(2, 1), gap, reduction="none")
            assert float((a - b).abs().max()) <= 2.0 ** -20 * (1 + float(a.abs().max()) + math.log(k))


def test_weightless_entries_of_masked_rows():
    """An entry of weight 0 whose row the student masks with -inf adds nothing."""
    print("case weightless", flush=True)
    for dt in ("bf16", "fp16", "fp32"):
        h, w, t, _ = inputs(9, 200, 24, 8, dt)
        h[:, 3], w[:, 3] = 1, 0
        w[50, 3] = -math.inf
        t = t % 50
        idx = torch.stack([t, torch.full_like(t, 50)], 1)
        tl = torch.tensor([0.0, torch.finfo(torch.float32).min], device="cuda").expand(9, 2)
        a = L.linear_distillation(h, w, tl, idx, reduction="none")
        b = L.linear_distillation(h, w, tl[:, :1], t[:, None], reduction="none")
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_positions_with_nothing_but_lowest_values(dt):
    lowest_values(dt, "distill")
