"""Norms of the gradients' errors.  Element by element a bound has to allow for every rounding at
its worst and in one direction, which over thousands of positions is 10 % of an element; over a
whole tensor independent roundings add up like their squares:
  g     eg^2 = (u g)^2 + p^2 (dz^2 + 2^-42),  dz^2 = (D 2^-48 [+ 2^-42]) sum_d (h w)^2
  dh    |error|^2 <= sum of eg^2 w^2 + (V 2^-48 [+ 2^-42]) (g^2 w^2) + (u_out dh)^2, dW alike
with u, u_out the largest rounding of each; their mean square is a third of that or less, which
is what the bound has to spare.  A bias in any of them, or a lost part, goes past it."""
import pytest
import torch

from tensor_train_compressed_ttembeddingbag_amd import loss as L
from test_gpu_loss_range import DT, U, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,v,d", [(70, 5000, 136), (2100, 4500, 515), (8200, 20000, 64)])
def test_norms(n, v, d, dt, op):
    print("case norms", n, v, d, dt, op, flush=True)
    h, w, t, g = inputs(n, v, d, n, dt)
    x, y = h.clone().requires_grad_(True), w.clone().requires_grad_(True)
    T = 1.0 if op == "xent" else 0.7
    if op == "xent":
        out = L.linear_cross_entropy(x, y, t, label_smoothing=0.1)
    else:
        idx = torch.randint(0, v, (n, 12), device="cuda", generator=g)
        tl = torch.randn(n, 12, device="cuda", generator=g)
        tl[:, 0] += 4
        idx[:, 0] = t
        out = L.linear_distillation(x, y, tl, idx, temperature=T)
    got = torch.autograd.grad(out, (x, y))
    u, uo = U[dt], (2.0 ** -24 if dt == "fp32" else U[dt])
    f32 = 2.0 ** -42 if dt == "fp32" else 0.0
    H, W = h.double(), w.double()
    q = torch.zeros(n, v, dtype=torch.float64, device="cuda")
    if op == "xent":
        q += 0.1 / v
        q[torch.arange(n, device="cuda"), t] += 0.9
    else:
        q.scatter_add_(1, idx, torch.softmax(tl.double() / T, 1))
    p = torch.softmax(H @ W.t() / T, 1)
    gr = (p - q) * (T / n)
    eg2 = (u * gr) ** 2 + (p * (T / n)) ** 2 * \
        ((d * 2.0 ** -48 + f32) * (H ** 2 @ (W ** 2).t()) / T ** 2 + 2.0 ** -42)
    if dt != "bf16":
        eg2 += (2.0 ** -39 * T / n) ** 2
    for a, ref, e2, name in (
            (got[0], gr @ W, eg2 @ W ** 2 + (v * 2.0 ** -48 + f32) * (gr ** 2 @ W ** 2), "dh"),
            (got[1], gr.t() @ H, eg2.t() @ H ** 2 + (n * 2.0 ** -48 + f32) * ((gr ** 2).t() @ H ** 2), "dW")):
        # fp16's last step, half of 2^-24, of every element
        e2 = e2 + (uo * ref) ** 2 + (2.0 ** -50 if dt == "fp16" else 0.0)
        err = float(((a.double() - ref) ** 2).sum() / e2.sum()) ** 0.5
        print("  ", name, "%.2f" % err, flush=True)
        assert err <= 1, (name, err)
