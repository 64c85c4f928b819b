"""Preference and policy losses of more than 16384 positions, where the largest of the positions' gradients is found by
a launch of its own, from the slopes: against the definitions in float64, within the tolerances that
``test_gpu_logp_losses`` derives.  The largest slopes are 10^4 times the others and stand where a search that
misses its end or its beginning would not see them."""
import pytest
import torch

from test_gpu_logp_losses import IGN, Head, compare, make, ragged, upstream, want_policy, want_prefer
from tensor_train_compressed_ttembeddingbag_amd import loss as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", ["first", "last", "nowhere"])
@pytest.mark.parametrize("reduction", ["none", "mean"])
@pytest.mark.parametrize("dt", ["fp16", "fp32", "bf16"])
def test_policy(dt, reduction, at):
    n, v, d = 17003, 300, 40
    print("case policy slopes", dt, reduction, at, flush=True)
    h, w, t, g = make(n, v, d, dt, seed=7)
    t[1:n - 1:3] = IGN
    lp = Head(h, w, t, dt, 1.0, t != IGN).l
    noise = torch.randn(3, n, device="cuda", generator=g)
    adv, old, ref = noise[0], (lp + 0.3 * noise[1]).float(), (lp + 0.5 * noise[2]).float()
    if at != "nowhere":
        k = 0 if at == "first" else n - 1
        adv[k], old[k] = -1e4, float(lp[k])  # a ratio of 1 within the bounds
    up = upstream(n, reduction, g)
    want = want_policy(h, w, t, dt, reduction, up, adv, old, ref, 0.2, 0.2, 0.1, 1.0)
    compare(lambda a, b: L.linear_policy(a, b, t, adv, old, ref, kl_coef=0.1, reduction=reduction,
                                         return_logps=True), want, h, w, up, reduction)


@pytest.mark.parametrize("kind", ["sigmoid", "square"])
@pytest.mark.parametrize("reduction", ["none", "mean"])
@pytest.mark.parametrize("dt", ["fp16", "fp32"])
def test_preference(dt, reduction, kind):
    n, v, d, pairs = 17003, 300, 40, 900
    print("case preference slopes", dt, reduction, kind, flush=True)
    h, w, t, g = make(n, v, d, dt, seed=8)
    t[::4] = IGN
    ref = (Head(h, w, t, dt, 1.0, t != IGN).l + 0.4 * torch.randn(n, device="cuda", generator=g)).float()
    off = ragged(n, pairs, g, 123)
    up = upstream(pairs, reduction, g)
    want = want_prefer(h, w, t, dt, reduction, up, off, ref, kind, 0.2, 0.0, 0.0, True)
    compare(lambda a, b: L.linear_preference(a, b, t, off, ref, kind=kind, beta=0.2, average=True,
                                             reduction=reduction, return_ratios=True), want, h, w, up, reduction)
