"""Preference and policy losses through a vocabulary head (loss.linear_preference, loss.linear_policy)
against their definitions in float64: losses, second outputs and both gradients.

Tolerances, derived per element (u = half a step of the type that the gradient of the logits and the
outputs are rounded to: bf16 2^-8, fp16 2^-11; fp32 enters as two fp16 parts, 2^-21 for a product of
two rounded operands, and its outputs round by 2^-24):
  logit    dz = (D 2^-24 [+ 2^-21]) max_v sum_d |h w| / T
  logp     el = 2 dz + 2^-21 (1 + |lse| + |z_t|)              (lse, its logs, the rounding to fp32)
  loss     sum |dL/dl| el, the second order of it, and 2^-23 of the value
  dL/dl    c = dL/dl is off by |d2L/dl2| el and 2^-22 of itself; where a bound (clip, hinge) lies within
           el, by all of what it switches
  g        u |g| + p (2 dz + 2^-20) + 2^-22 [v = t]           (p - [v = t], rounding and exp)
  dh, dW   sum |c| (g's error) |w| + dc |g| |w| + (count 2^-24 [+ 2^-21]) sum |c g w| + u |result| + tiny
where tiny covers fp16's subnormal steps: 2^-25 of an output; of a g 2^-38 of the largest c (c is divided by
the power of two above the largest, at most twice it; the g that this leaves, times 2^14, ends in fp16 steps of
2^-24, so rounding is off by 2^-25 2^-14 2).  All of it is computed in float64 from the inputs."""
import math

import pytest
import torch

from tensor_train_compressed_ttembeddingbag_amd import abi, loss as L

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -21}
IGN = -100


def make(n, v, d, dt, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randn(v, d, device="cuda", generator=g) * d ** -0.5
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    h = torch.randn(n, d, device="cuda", generator=g)
    if n:
        h = h + w[t] * 6.0
    return h.to(DT[dt]), w.to(DT[dt]), t, g


class Head:
    """The log-probabilities of the targets and what they may be off by."""

    def __init__(self, h, w, t, dt, T, ok):
        self.dt, self.T, self.ok, self.t = dt, T, ok, t
        self.H = torch.where(ok[:, None], h.double(), 0.0)
        self.W = w.double()
        n, d = self.H.shape
        z = self.H @ self.W.t().contiguous() / T
        self.dz = (d * 2.0 ** -24 + (2.0 ** -21 if dt == "fp32" else 0)) * \
            (self.H.abs() @ self.W.abs().t().contiguous()).amax(1) / T if n else z.new_zeros(0)
        lse = torch.logsumexp(z, 1)
        zt = z.gather(1, torch.where(ok, t, 0)[:, None])[:, 0]
        self.p = torch.exp(z - lse[:, None])
        self.l = torch.where(ok, zt - lse, 0.0)
        self.el = (2 * self.dz + 2.0 ** -21 * (1 + lse.abs() + zt.abs())) * ok

    def grads(self, c, ec):
        """((dh, bound), (dw, bound)) from dL/dl and its error."""
        dt, ok = self.dt, self.ok
        c, ec = c * ok / self.T, ec * ok / self.T
        q = torch.zeros_like(self.p)
        q[ok.nonzero()[:, 0], self.t[ok]] = 1.0
        g = self.p - q
        eg = U[dt] * g.abs() + self.p * (2 * self.dz[:, None] + 2.0 ** -20) + 2.0 ** -22 * q
        eg = eg * c.abs()[:, None] + g.abs() * (ec + 2.0 ** -22 * c.abs())[:, None]
        g = -g * c[:, None]
        if dt != "bf16" and len(c):
            eg = eg + 2.0 ** -38 * c.abs().max() * ok[:, None]
        uo = 2.0 ** -24 if dt == "fp32" else U[dt]
        sub = 2.0 ** -25 if dt == "fp16" else 2.0 ** -133
        extra = 2.0 ** -21 if dt == "fp32" else 0.0
        n, v = g.shape
        gt = g.t().contiguous()
        dh, dw = g @ self.W, gt @ self.H
        bh = eg @ self.W.abs() + (v * 2.0 ** -24 + extra) * (g.abs() @ self.W.abs()) + uo * dh.abs() + sub
        bw = eg.t().contiguous() @ self.H.abs() + (n * 2.0 ** -24 + extra) * (gt.abs() @ self.H.abs()) + \
            uo * dw.abs() + sub
        return (dh, bh), (dw, bw)


def reduced(rows, err, reduction, count):
    if reduction == "none":
        return rows, err + 2.0 ** -23 * rows.abs()
    div = max(1, count) if reduction == "mean" else 1
    return rows.sum() / div, err.sum() / div + 2.0 ** -23 * (rows.sum() / div).abs()


def scaled(c, ec, up, reduction, count):
    f = up.double() if reduction == "none" else up.double() / (max(1, count) if reduction == "mean" else 1)
    return c * f, ec * f.abs() + 2.0 ** -22 * (c * f).abs()


def want_policy(h, w, t, dt, reduction, up, adv, old, ref, low, high, kl, T):
    ok = (t != IGN) & (t >= 0) & (t < w.shape[0])
    head = Head(h, w, t, dt, T, ok)
    A = torch.where(ok, adv.double(), 0.0)
    l, el = head.l, head.el
    if old is None:
        r, er = torch.ones_like(l), torch.zeros_like(l)
        slope_err = torch.zeros_like(l)
    else:
        r = torch.exp(l - torch.where(ok, old.double(), 0.0))
        er = r * torch.expm1(el)
        slope_err = er
    held = r.clamp(1 - low, 1 + high) * A
    rows, c = -torch.minimum(r * A, held), torch.where(r * A <= held, -r * A, 0.0)
    err, ec = er * A.abs(), slope_err * A.abs()
    near = ((r - (1 - low)).abs() <= er) | ((r - (1 + high)).abs() <= er)
    ec = ec + torch.where(near & (er > 0), (r * A).abs() + ec, 0.0)
    if kl:
        d = torch.where(ok, ref.double(), 0.0) - l
        rows = rows + kl * (torch.expm1(d) - d)
        c = c - kl * torch.expm1(d)
        err = err + kl * (torch.expm1(d).abs() * el + torch.exp(d) * torch.expm1(el) * el)
        ec = ec + kl * torch.exp(d) * torch.expm1(el)
    rows, c, err, ec = (torch.where(ok, x, 0.0) for x in (rows, c, err, ec))
    count = int(ok.sum())
    out = reduced(rows, err, reduction, count)
    if up is None:
        return out, (l, el)
    return out, (l, el), *head.grads(*scaled(c, ec, up, reduction, count))


def want_prefer(h, w, t, dt, reduction, up, off, ref, kind, beta, e, margin, average):
    n, off = len(t), off.tolist()
    P = len(off) // 2
    ok = (t != IGN) & (t >= 0) & (t < w.shape[0])
    ok[off[-1]:] = False
    head = Head(h, w, t, dt, 1.0, ok)
    seq = torch.zeros(n, dtype=torch.int64, device="cuda")
    for j, (a, b) in enumerate(zip(off, off[1:])):
        seq[a:b] = j
    per = head.l - (0.0 if ref is None else torch.where(ok, ref.double(), 0.0))
    zero = torch.zeros(2 * P, dtype=torch.float64, device="cuda")
    count = zero.index_add(0, seq[ok], torch.ones_like(per[ok]))
    share = 1.0 / count.clamp(min=1) if average else torch.ones_like(zero)
    ratio = zero.index_add(0, seq[ok], per[ok]) * share
    er = zero.index_add(0, seq[ok], head.el[ok]) * share
    x, ex = ratio[:P] - ratio[P:], er[:P] + er[P:]
    if kind == "square":
        gap = x - 0.5 / beta
        rows, s, err, es = gap * gap, 2 * gap, 2 * gap.abs() * ex + ex * ex, 2 * ex
    else:
        y, ey = beta * x - margin, beta * ex
        if kind == "hinge":
            near = (y - 1).abs() <= ey
            rows, s = torch.relu(1 - y), -beta * (y < 1).double()
            err, es = ey, beta * near.double()
        else:
            sp = torch.nn.functional.softplus
            rows = (1 - e) * sp(-y) + e * sp(y)
            s = beta * (torch.sigmoid(y) - (1 - e))
            # the second derivative is S(y) S(-y), which changes by a factor exp(ey) at most
            curve = torch.sigmoid(y) * torch.sigmoid(-y) * torch.exp(ey)
            err, es = (s / beta).abs() * ey + curve * ey * ey, beta * curve * ey
    out = reduced(rows, err, reduction, P)
    more = (ratio.view(2, P), (er + 2.0 ** -23 * ratio.abs()).view(2, P))
    if up is None:
        return out, more
    s, es = scaled(s, es, up, reduction, P)
    c, ec = torch.cat([s, -s]) * share, torch.cat([es, es]) * share
    if P == 0:
        c = ec = torch.zeros(1, dtype=torch.float64, device="cuda")
        seq = torch.zeros_like(seq)
    return out, more, *head.grads(c[seq], ec[seq])


def check(got, want, name):
    ref, bound = want
    got = got.double()
    assert got.shape == ref.shape, name
    assert torch.isfinite(got).all(), name
    bad = ((got - ref).abs() / (bound + 1e-30)) if got.numel() else torch.zeros(1)
    assert float(bad.max()) <= 1.0, (name, float(bad.max()))


def compare(call, want, h, w, up, reduction):
    h, w = h.detach().requires_grad_(True), w.detach().requires_grad_(True)
    out, more = call(h, w)
    dh, dw = torch.autograd.grad(out, (h, w), up if reduction == "none" else up.reshape(()))
    for a, b, name in zip((out.detach(), more, dh, dw), want, ("loss", "more", "dh", "dW")):
        check(a, b, name)
    with torch.no_grad():
        out, more = call(h, w)
    check(out, want[0], "loss alone")
    check(more, want[1], "more alone")


def upstream(n, reduction, g):
    if reduction == "none":
        return torch.randn(n, device="cuda", generator=g)
    return torch.tensor(1.7, device="cuda")


def ragged(n, pairs, g, tail):
    """offsets of 2 P sequences, some of them empty"""
    cut = torch.randint(0, n - tail + 1, (2 * pairs - 1,), device="cuda", generator=g).sort().values
    ends = torch.tensor([n - tail], device="cuda")
    return torch.cat([torch.zeros_like(ends), cut, ends])


SIZES = [(2, 1, 1), (1, 1000, 64), (3, 37, 5), (17, 301, 72), (48, 2048, 128), (65, 513, 130),
         (100, 1031, 67), (200, 4099, 256), (300, 700, 515), (513, 5000, 64)]


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,v,d", SIZES)
def test_policy(n, v, d, dt):
    print("case policy", n, v, d, dt, flush=True)
    h, w, t, g = make(n, v, d, dt, seed=n + v)
    ones = torch.ones(n, dtype=torch.bool, device="cuda")
    for k, (reduction, ign, kl, T, low, high) in enumerate(
            (("mean", 0.3, 0.0, 1.0, 0.2, 0.2), ("none", 0.2, 0.05, 0.7, 0.1, 0.3),
             ("sum", 0.0, 0.5, 2.0, 0.0, math.inf), ("none", 0.0, 0.0, 1.0, 1.5, 0.0))):
        tt = torch.where(torch.rand(n, device="cuda", generator=g) < ign, IGN, t)
        lp = Head(h, w, t, dt, T, ones).l
        noise = torch.randn(3, n, device="cuda", generator=g)
        adv, old, ref = noise[0], (lp + 0.3 * noise[1]).float(), (lp + 0.5 * noise[2]).float()
        if k == 3:
            old = None
        drop = tt == IGN  # not looked at where a position does not count
        adv[drop] = float("nan")
        ref[drop] = float("inf")
        if old is not None:
            old[drop] = float("nan")
        hh = h.clone()
        hh[drop] = float("nan")
        up = upstream(n, reduction, g)
        want = want_policy(h, w, tt, dt, reduction, up, adv, old, ref, low, high, kl, T)
        compare(lambda a, b: L.linear_policy(a, b, tt, adv, old, ref if kl else None, clip_low=low,
                                             clip_high=high, kl_coef=kl, temperature=T,
                                             reduction=reduction, return_logps=True),
                want, hh, w, up, reduction)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,v,d", SIZES)
def test_preference(n, v, d, dt):
    print("case prefer", n, v, d, dt, flush=True)
    h, w, t, g = make(n, v, d, dt, seed=n + v + 1)
    ones = torch.ones(n, dtype=torch.bool, device="cuda")
    lp = Head(h, w, t, dt, 1.0, ones).l
    for reduction, ign, kind, beta, e, margin, average, pairs in (
            ("mean", 0.3, "sigmoid", 0.1, 0.0, 0.0, False, 1 + n // 9),
            ("none", 0.0, "sigmoid", 0.5, 0.2, 0.3, True, 1 + n // 40),
            ("sum", 0.1, "hinge", 0.3, 0.0, -0.5, False, 1 + n // 20),
            ("none", 0.5, "square", 0.4, 0.0, 0.0, True, 1 + n // 5),
            ("mean", 0.0, "sigmoid", 2.0, 1.0, 0.0, True, 3)):
        tail = n // 10
        off = ragged(n, pairs, g, tail)
        tt = torch.where(torch.rand(n, device="cuda", generator=g) < ign, IGN, t)
        ref = (lp + 0.4 * torch.randn(n, device="cuda", generator=g)).float()
        if e == 1.0:
            ref = None
        drop = tt == IGN
        drop[n - tail:] = True
        hh = h.clone()
        hh[drop] = float("nan")
        if ref is not None:
            ref[drop] = float("nan")
        if tail:
            tt[-1] = v + 5  # behind the last sequence: no index
        up = upstream(pairs, reduction, g)
        want = want_prefer(h, w, tt, dt, reduction, up, off, ref, kind, beta, e, margin, average)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        compare(lambda a, b: L.linear_preference(
            a, b, tt, off, ref, beta=beta, kind=kind, label_smoothing=e, margin=margin,
            average=average, reduction=reduction, return_ratios=True, dev_status=status),
            want, hh, w, up, reduction)
        assert int(status) == 0


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_many_positions(dt):
    """Past what one workgroup sums, past what is counted by blocks, several pieces of the vocabulary."""
    n, v, d = (9000, 33000, 64) if dt == "bf16" else (8500, 3000, 40)
    print("case many", n, v, d, dt, flush=True)
    h, w, t, g = make(n, v, d, dt, seed=5)
    t[::3] = IGN
    lp = Head(h, w, t, dt, 1.0, t != IGN).l
    noise = torch.randn(3, n, device="cuda", generator=g)
    adv, old, ref = noise[0], (lp + 0.3 * noise[1]).float(), (lp + 0.5 * noise[2]).float()
    for reduction in ("mean", "none"):
        up = upstream(n, reduction, g)
        want = want_policy(h, w, t, dt, reduction, up, adv, old, ref, 0.2, 0.2, 0.1, 1.0)
        compare(lambda a, b: L.linear_policy(a, b, t, adv, old, ref, kl_coef=0.1, reduction=reduction,
                                             return_logps=True), want, h, w, up, reduction)
        del want
    off = ragged(n, 700, g, 111)
    up = upstream(700, "mean", g)
    want = want_prefer(h, w, t, dt, "mean", up, off, ref, "sigmoid", 0.1, 0.0, 0.0, False)
    compare(lambda a, b: L.linear_preference(a, b, t, off, ref, return_ratios=True), want, h, w, up, "mean")


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_shapes_and_strides(dt):
    h, w, t, g = make(60, 90, 45, dt, seed=2)
    base = torch.zeros(3, 4, 5, 60, device="cuda", dtype=DT[dt])
    base[..., 7:52] = h.view(3, 4, 5, 45)
    wide = torch.zeros(90, 101, device="cuda", dtype=DT[dt])
    wide[:, 3:48] = w
    tt = t.view(3, 4, 5)
    adv = torch.randn(3, 1, 5, device="cuda", generator=g)
    old = (Head(h, w, t, dt, 1.0, t >= 0).l + 0.1).float().view(3, 4, 5)
    up = torch.randn(3, 4, 5, device="cuda", generator=g)
    (out, lp), (dh, bh), (dw, bw) = (None, None), (None, None), (None, None)
    want = want_policy(h, w, t, dt, "none", up.reshape(-1), adv.broadcast_to(3, 4, 5).reshape(-1),
                       old.reshape(-1), None, 0.2, 0.2, 0.0, 1.0)
    a, b = base[..., 7:52].requires_grad_(), wide[:, 3:48].requires_grad_()
    out, lp = L.linear_policy(a, b, tt.int(), adv, old.transpose(0, 1).contiguous().transpose(0, 1),
                              reduction="none", return_logps=True)
    assert out.shape == (3, 4, 5) and lp.shape == (3, 4, 5)
    dh, dw = torch.autograd.grad(out, (a, b), up)
    for x, y, name in zip((out.detach().reshape(-1), lp.reshape(-1), dh.reshape(60, 45), dw), want,
                          ("loss", "logps", "dh", "dW")):
        check(x, y, name)
    off = torch.tensor([0, 10, 31, 31, 55], dtype=torch.int32, device="cuda")
    want = want_prefer(h, w, t, dt, "sum", torch.ones((), device="cuda"), off, None, "sigmoid", 0.1, 0.0,
                       0.0, False)
    loss = L.linear_preference(a, b, tt, off, reduction="sum")
    dh, dw = torch.autograd.grad(loss, (a, b))
    for x, y, name in zip((loss.detach(), dh.reshape(60, 45), dw), (want[0], *want[2:]), ("loss", "dh", "dW")):
        check(x, y, name)
    # only one of the two wanted: the same bits
    one, = torch.autograd.grad(L.linear_preference(a.detach(), b, tt, off, reduction="sum"), b)
    assert torch.equal(one, dw)
    one, = torch.autograd.grad(L.linear_preference(a, b.detach(), tt, off, reduction="sum"), a)
    assert torch.equal(one.reshape(60, 45), dh.reshape(60, 45))


@pytest.mark.parametrize("n", [0, 5, 100])
def test_nothing_counts(n):
    h = torch.full((n, 16), float("nan"), device="cuda", requires_grad=True)
    w = torch.randn(20, 16, device="cuda", requires_grad=True)
    t = torch.full((n,), IGN, dtype=torch.int64, device="cuda")
    adv = torch.ones(n, device="cuda")
    for reduction in ("mean", "sum", "none"):
        out, lp = L.linear_policy(h, w, t, adv, adv, reduction=reduction, return_logps=True)
        assert out.shape == ((n,) if reduction == "none" else ())
        assert not bool(out.any()) and not bool(lp.any())
        dh, dw = torch.autograd.grad(out.sum(), (h, w))
        assert not bool(dh.any()) and not bool(dw.any())
        with torch.no_grad():
            assert not bool(L.linear_policy(h, w, t, adv, reduction=reduction).any())
    off = torch.zeros(5, dtype=torch.int64, device="cuda")
    off[2:] = n
    for reduction, value in (("mean", math.log(2)), ("sum", 2 * math.log(2)), ("none", math.log(2))):
        out, ratios = L.linear_preference(h, w, t, off, reduction=reduction, return_ratios=True)
        assert not bool(ratios.any()) and ratios.shape == (2, 2)
        assert bool(((out - value).abs() <= 2.0 ** -22 * value).all())
        dh, dw = torch.autograd.grad(out.sum(), (h, w))
        assert not bool(dh.any()) and not bool(dw.any())
    none = torch.zeros(1, dtype=torch.int64, device="cuda")
    t[:] = 3  # all positions lie behind the last sequence
    for reduction in ("mean", "sum", "none"):
        out = L.linear_preference(h, w, t, none, reduction=reduction)
        assert out.shape == ((0,) if reduction == "none" else ()) and not bool(out.any())
        dh, dw = torch.autograd.grad(out.sum(), (h, w))
        assert not bool(dh.any()) and not bool(dw.any())


def test_no_tokens_and_no_pairs_have_their_own_forms():
    w = torch.randn(20, 16, device="cuda", requires_grad=True)
    h = torch.zeros(0, 16, device="cuda", requires_grad=True)
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    out = L.linear_policy(h, w, t, torch.zeros(0, device="cuda"))
    dh, dw = torch.autograd.grad(out, (h, w))
    assert float(out) == 0 and dh.shape == (0, 16) and not bool(dw.any())


def test_bad_indices_and_offsets():
    h, w, t, g = make(40, 50, 24, "fp32", seed=3)
    h.requires_grad_()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = t.clone()
    bad[4], bad[9] = 50, -7
    adv = torch.ones(40, device="cuda")
    out = L.linear_policy(h, w, bad, adv, reduction="none", dev_status=status)
    assert int(status) == abi.TT_DEV_BAD_INDEX
    assert float(out[4].detach()) == 0 and float(out[9].detach()) == 0
    dh, = torch.autograd.grad(out.sum(), h)
    assert not bool(dh[[4, 9]].any())
    status.zero_()
    with torch.no_grad():
        L.linear_policy(h, w, bad, adv, dev_status=status)
    assert int(status) == abi.TT_DEV_BAD_INDEX
    for off in ([1, 5, 40], [0, 30, 20], [0, 10, 41], [0, -3, 40], [0, 1 << 40, 40], [-5, 0, 1 << 50]):
        status.zero_()
        loss = L.linear_preference(h, w, t, torch.tensor(off, device="cuda"), dev_status=status)
        assert int(status) == abi.TT_DEV_BAD_OFFSETS, off
        torch.autograd.grad(loss, h)  # unspecified, but it ends
        torch.cuda.synchronize()


def test_infinities_of_the_constants():
    """An action that the old policy could not take, a reference that rules one out."""
    h, w, t, g = make(6, 30, 16, "fp32", seed=4)
    inf = float("inf")
    old = torch.tensor([-inf, -inf, inf, -inf, 0.0, 0.0], device="cuda")
    adv = torch.tensor([2.0, -1.0, 1.0, 0.0, 1.0, 1.0], device="cuda")
    h.requires_grad_()
    out = L.linear_policy(h, w, t, adv, old, reduction="none")
    assert float(out[0]) == pytest.approx(-2.4) and float(out[1]) == inf and float(out[2]) == 0.0
    assert math.isnan(float(out[3]))  # infinity times an advantage of 0
    dh, = torch.autograd.grad(out[[0, 2, 4]].sum(), h)
    assert not bool(dh[[0, 2, 5]].any())  # held at the clip, of no weight, or not asked for
    assert bool(torch.isnan(dh[[1, 3]]).all())  # 0 times an infinite slope, as in any chain rule
    ref = torch.tensor([-inf, 0.0, 0.0, 0.0, 0.0, 0.0], device="cuda")
    out = L.linear_policy(h, w, t, torch.zeros(6, device="cuda"), None, ref, kl_coef=0.5, reduction="none")
    assert float(out[0]) == inf and bool(torch.isfinite(out[1:]).all())


@pytest.mark.parametrize("op", ["policy", "preference"])
def test_against_differences(op):
    """Central differences of the definition in float64."""
    h, w, t, g = make(8, 13, 5, "fp32", seed=6)
    w = w * 2
    adv = torch.randn(8, device="cuda", generator=g)
    old = Head(h, w, t, "fp32", 0.8, t >= 0).l.float() + 0.1 * torch.randn(8, device="cuda", generator=g)
    ref = old + 0.2
    off = torch.tensor([0, 2, 3, 6, 7], device="cuda")
    up = torch.ones((), device="cuda")

    def value(h, w):
        if op == "policy":
            return want_policy(h, w, t, "fp32", "mean", None, adv, old, ref, 0.2, 0.2, 0.3, 0.8)[0][0]
        return want_prefer(h, w, t, "fp32", "mean", None, off, ref, "sigmoid", 0.7, 0.1, 0.2, True)[0][0]

    a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
    if op == "policy":
        loss = L.linear_policy(a, b, t, adv, old, ref, kl_coef=0.3, temperature=0.8)
    else:
        loss = L.linear_preference(a, b, t, off, ref, beta=0.7, label_smoothing=0.1, margin=0.2, average=True)
    dh, dw = torch.autograd.grad(loss, (a, b), up)
    step = 1e-5  # error of a difference: step^2 times a third derivative of some 10, and 1e-16 / step
    for grad, which in ((dh, 0), (dw, 1)):
        x = (h.double(), w.double())[which]
        for r in range(x.shape[0]):
            for k in range(x.shape[1]):
                e = torch.zeros_like(x)
                e[r, k] = step
                pair = [(x + s * e, w.double()) if which == 0 else (h.double(), x + s * e) for s in (1, -1)]
                diff = (value(*pair[0]) - value(*pair[1])) / (2 * step)
                assert abs(float(grad[r, k]) - float(diff)) <= 1e-8 + 2e-6 * float(grad.abs().max())


@pytest.mark.parametrize("op", ["policy", "preference"])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_captured(op, dt):
    """Forward and backward captured and replayed with new data between eager calls."""
    n = 150
    h, w, t, g = make(n, 700, 72, dt, seed=8)
    adv, old = torch.randn(n, device="cuda", generator=g), torch.full((n,), -5.0, device="cuda")
    off = torch.tensor([0, 20, 70, 100, 140], device="cuda")

    def step(h, w):
        a, b = h.detach().requires_grad_(), w.detach().requires_grad_()
        loss = L.linear_policy(a, b, t, adv, old) if op == "policy" else \
            L.linear_preference(a, b, t, off, old)
        return (loss.detach(), *torch.autograd.grad(loss, (a, b)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(h, w)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(h, w)
    for k in range(4):
        h.copy_(torch.randn(n, 72, device="cuda", generator=g))
        adv.copy_(torch.randn(n, device="cuda", generator=g))
        t.copy_(torch.randint(0, 700, (n,), device="cuda", generator=g))
        off[1:4] = torch.tensor([10 * k, 60, 60 + 5 * k])
        graph.replay()
        want = step(h, w)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_same_bits_again_and_two_streams():
    h, w, t, g = make(300, 5000, 128, "bf16", seed=10)
    adv, old = torch.randn(300, device="cuda", generator=g), torch.full((300,), -6.0, device="cuda")

    def step():
        a, b = h.detach().requires_grad_(), w.detach().requires_grad_()
        loss = L.linear_policy(a, b, t, adv, old)
        return (loss.detach(), *torch.autograd.grad(loss, (a, b)))

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    again = step()
    torch.cuda.synchronize()
    for a, b, c in zip(first, other, again):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_second_derivatives_are_refused():
    h, w, t, g = make(6, 30, 16, "fp32", seed=4)
    h.requires_grad_()
    loss = L.linear_policy(h, w, t, torch.ones(6, device="cuda"))
    dh, = torch.autograd.grad(loss, h, create_graph=True)
    with pytest.raises(RuntimeError):
        dh.sum().backward()


def test_constants_get_no_gradient():
    h, w, t, g = make(6, 30, 16, "fp32", seed=4)
    h.requires_grad_()
    adv = torch.ones(6, device="cuda", requires_grad=True)
    loss, lp = L.linear_policy(h, w, t, adv, return_logps=True)
    assert not lp.requires_grad
    loss.backward()
    assert adv.grad is None and h.grad is not None


def test_arguments_are_refused():
    h, w, t, g = make(6, 30, 16, "fp32", seed=4)
    adv, off = torch.ones(6, device="cuda"), torch.tensor([0, 2, 6], device="cuda")
    for match, error, f in (
            ("shape", ValueError, lambda: L.linear_policy(h, w, t[:5], adv)),
            ("broadcast", ValueError, lambda: L.linear_policy(h, w, t, adv[:5])),
            ("shape", ValueError, lambda: L.linear_policy(h, w, t, adv, adv[:5])),
            ("int64", TypeError, lambda: L.linear_policy(h, w, t.float(), adv)),
            ("advantages", TypeError, lambda: L.linear_policy(h, w, t, adv.double())),
            ("on cpu", ValueError, lambda: L.linear_policy(h, w, t, adv.cpu())),
            ("reduction", ValueError, lambda: L.linear_policy(h, w, t, adv, reduction="max")),
            ("entries", ValueError, lambda: L.linear_preference(h, w, t, off[:2])),
            ("entries", ValueError, lambda: L.linear_preference(h, w, t, off[None])),
            ("shape", ValueError, lambda: L.linear_preference(h, w, t, off, adv[:3])),
            ("on cpu", ValueError, lambda: L.linear_preference(h, w, t, off.cpu())),
            ("hidden is", TypeError, lambda: L.linear_preference(h, w.half(), t, off)),
            ("dev_status", TypeError, lambda: L.linear_preference(h, w, t, off, dev_status=t))):
        with pytest.raises(error, match=match):
            f()


@pytest.mark.parametrize("dt,n,v,d", [("bf16", 2100, 33000, 1024), ("fp32", 8300, 8300, 1024),
                                      ("fp16", 8300, 8300, 1024)])
def test_positions_without_a_gradient_are_left_out(dt, n, v, d):
    """Large enough for the backward to work on the positions with a slope alone."""
    print("case kept", n, v, d, dt, flush=True)
    h, w, t, g = make(n, v, d, dt, seed=12)
    t[5::7] = IGN
    lp = Head(h, w, t, dt, 1.0, t != IGN).l
    noise = torch.randn(2, n, device="cuda", generator=g)
    adv, old = noise[0], (lp + 0.4 * noise[1]).float()
    adv[n // 3:n // 2] = 0.0
    up = upstream(n, "mean", g)
    want = want_policy(h, w, t, dt, "mean", up, adv, old, None, 0.1, 0.1, 0.0, 1.0)
    compare(lambda a, b: L.linear_policy(a, b, t, adv, old, clip_low=0.1, clip_high=0.1, return_logps=True),
            want, h, w, up, "mean")
    del want
    up = upstream(n, "none", g)
    up[::3] = 0.0
    want = want_policy(h, w, t, dt, "none", up, adv, old, None, 0.1, 0.1, 0.0, 1.0)
    compare(lambda a, b: L.linear_policy(a, b, t, adv, old, clip_low=0.1, clip_high=0.1, reduction="none",
                                         return_logps=True), want, h, w, up, "none")
    del want
    off = ragged(n, 50, g, 20)
    ref = (lp + 0.3 * noise[0] - 0.02).float()
    up = upstream(50, "sum", g)
    want = want_prefer(h, w, t, dt, "sum", up, off, ref, "hinge", 0.2, 0.0, 0.0, False)
    compare(lambda a, b: L.linear_preference(a, b, t, off, ref, beta=0.2, kind="hinge", reduction="sum",
                                             return_ratios=True), want, h, w, up, "sum")
    del want
    a, b = h.clone().requires_grad_(), w.clone().requires_grad_()  # nothing has one
    dh, dw = torch.autograd.grad(L.linear_policy(a, b, t, torch.zeros_like(adv), old), (a, b))
    assert not bool(dh.any()) and not bool(dw.any())


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_repeated_backward(dt):
    """What is saved is left as it was."""
    h, w, t, g = make(40, 300, 64, dt, seed=14)
    h.requires_grad_(), w.requires_grad_()
    off = torch.tensor([0, 11, 20, 29, 38], device="cuda")
    for loss in (L.linear_policy(h, w, t, torch.randn(40, device="cuda", generator=g)),
                 L.linear_preference(h, w, t, off)):
        first = torch.autograd.grad(loss, (h, w), retain_graph=True)
        for a, b in zip(first, torch.autograd.grad(loss, (h, w))):
            assert torch.equal(a, b)


def test_changed_inputs_are_noticed():
    h, w, t, g = make(8, 30, 16, "fp32", seed=4)
    h.requires_grad_(), w.requires_grad_()
    loss = L.linear_policy(h, w, t, torch.ones(8, device="cuda"))
    with torch.no_grad():
        w.add_(1.0)
    with pytest.raises(RuntimeError, match="modified"):
        loss.backward()


@pytest.mark.parametrize("d", [1, 4, 31, 127, 128, 129, 132, 256, 385, 1024, 4097])
@pytest.mark.parametrize("n,v", [(3, 300), (64, 16500)])
def test_few_positions_of_fp32(n, v, d):
    """Without a gradient: 128 products are summed by themselves and the sums added, so a sum of d is
    rounded at most 128 + d / 128 + 1 times at the size of what it holds, not d times."""
    h, w, t, _ = make(n, v, d, "fp32", seed=d)
    head = Head(h, w, t, "fp32", 1.0, torch.ones(n, dtype=torch.bool, device="cuda"))
    A = (head.H.abs() @ head.W.abs().t().contiguous()).amax(1)
    dz = (min(d, 128) + d // 128 + 1) * 2.0 ** -24 * A
    z = head.H @ head.W.t().contiguous()
    lse, zt = torch.logsumexp(z, 1), z.gather(1, t[:, None])[:, 0]
    with torch.no_grad():
        _, logps = L.linear_policy(h, w, t, torch.ones(1, device="cuda").expand(n), return_logps=True)
    err = (logps.double() - head.l).abs()
    assert bool((err <= 2 * dz + 2.0 ** -21 * (1 + lse.abs() + zt.abs())).all())
