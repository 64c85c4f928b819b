"""Vocabulary-head losses (loss.linear_cross_entropy, loss.linear_distillation) against their
definitions in float64: losses and both gradients, over types, odd sizes, strides, ignored
positions, ragged and repeated teacher entries, and vocabularies of several pieces.

Tolerances, derived per element (u = half a step of the type that the gradient of the logits
and the outputs are rounded to: bf16 2^-8, fp16 2^-11; fp32 enters as two fp16 parts, so 2^-21
covers a product of two rounded operands, and its outputs round by 2^-24):
  logit    dz = (D 2^-24 [+ 2^-21]) max_v sum_d |h w| / T        (D rounded additions)
  loss     scale * (2 dz + 2^-21 (1 + |terms|))                   (lse, its logs and the sum)
  g        u |g| + p (2 dz + 2^-20)                               (rounding; exp of a shifted logit)
  dh, dW   sum (g's error) |w| + (count 2^-24 [+ 2^-21]) sum |g w| + u |result| + tiny
where tiny covers fp16's subnormal steps (2^-25 of an output; 2^-40 of the largest factor of a
g).  All of it is computed in float64 from the inputs."""
import math

import pytest
import torch

from tensor_train_compressed_ttembeddingbag_amd import abi, loss as L

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -21}
IGN = -100


def make(n, v, d, dt, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randn(v, d, device="cuda", generator=g) * d ** -0.5
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    h = torch.randn(n, d, device="cuda", generator=g)
    if n:
        h = h + w[t] * 6.0
    h = h * scale
    return h.to(DT[dt]), w.to(DT[dt]), t, g


def teacher(n, v, k, g, dt=torch.float32):
    idx = torch.randint(0, v, (n, k), device="cuda", generator=g)  # rows may repeat
    tl = torch.randn(n, k, device="cuda", generator=g) * 2
    drop = torch.rand(n, k, device="cuda", generator=g) < 0.3
    idx = torch.where(drop, -1 - idx, idx)
    return tl.to(dt), idx


def definition(h, w, dt, reduction, up, targets=None, e=0.0, tl=None, idx=None, T=1.0):
    """(loss, dh, dW) in float64 and the error bound of each."""
    H, W = h.double(), w.double()
    n, d = H.shape
    v = W.shape[0]
    if targets is not None:
        ok = (targets != IGN) & (targets >= 0) & (targets < v)
    else:
        ok = ((idx >= 0) & (idx < v) & (tl != -math.inf)).any(1)
    H = torch.where(ok[:, None], H, torch.zeros_like(H))
    z = H @ W.t() / T
    dz = (d * 2.0 ** -24 + (2.0 ** -21 if dt == "fp32" else 0)) * \
        (H.abs() @ W.abs().t()).amax(1) / T
    lse = torch.logsumexp(z, 1)
    q = torch.zeros_like(z)
    if targets is not None:
        q[ok.nonzero()[:, 0], targets[ok]] = 1 - e
        rows = lse - (q * z).sum(1) - e * z.mean(1)
        size = 1 + lse.abs() + (q * z).abs().sum(1) + e * z.abs().mean(1)
        scale, c = 1.0, 1.0
    else:
        ent = (idx >= 0) & (idx < v) & (tl != -math.inf)
        x = torch.where(ent, tl.double() / T, torch.full_like(tl, -math.inf, dtype=torch.float64))
        x = torch.where(ok[:, None], x, torch.zeros_like(x))
        lq = torch.log_softmax(x, 1)
        p = torch.where(ent, lq.exp(), torch.zeros_like(lq))
        q.scatter_add_(1, torch.where(ent, idx, torch.zeros_like(idx)), p)
        H1 = torch.where(p > 0, p * lq, torch.zeros_like(p)).sum(1)
        rows = T * T * (H1 - (q * z).sum(1) + lse)
        size = 1 + H1.abs() + lse.abs() + (q * z).abs().sum(1)
        scale, c = T * T, T
    rows = torch.where(ok, rows, torch.zeros_like(rows))
    lerr = scale * (2 * dz + 2.0 ** -21 * size) * ok
    cnt = max(1, int(ok.sum()))
    if reduction == "none":
        loss, lbound = rows, lerr
        f = up.double() * c * ok
    else:
        div = cnt if reduction == "mean" else 1
        loss, lbound = rows.sum() / div, lerr.sum() / div + 2.0 ** -23 * abs(rows.sum() / div)
        f = torch.full_like(rows, c * float(up) / div) * ok
    p = torch.exp(z - lse[:, None])
    g = p - q - (e / v if targets is not None else 0.0)
    eg = U[dt] * g.abs() + p * (2 * dz[:, None] + 2.0 ** -20) + 2.0 ** -22 * (q + e / v)
    g, eg = g * f[:, None], eg * f.abs()[:, None]
    if dt != "bf16":
        eg = eg + 2.0 ** -40 * f.abs().max() * ok[:, None]
    uo = 2.0 ** -24 if dt == "fp32" else U[dt]
    sub = 2.0 ** -25 if dt == "fp16" else 2.0 ** -133
    extra = 2.0 ** -21 if dt == "fp32" else 0.0
    dh, dw = g @ W, g.t() @ H
    bh = eg @ W.abs() + (v * 2.0 ** -24 + extra) * (g.abs() @ W.abs()) + uo * dh.abs() + sub
    bw = eg.t() @ H.abs() + (n * 2.0 ** -24 + extra) * (g.abs().t() @ H.abs()) + uo * dw.abs() + sub
    return (loss, lbound + 1e-30), (dh, bh), (dw, bw)


def check(got, want, name):
    ref, bound = want
    got = got.double()
    assert got.shape == ref.shape
    assert torch.isfinite(got).all(), name
    bad = (got - ref).abs() / bound
    assert float(bad.max() if bad.numel() else 0) <= 1.0, (name, float(bad.max()))


def run(h, w, reduction, up, **kw):
    h, w = h.detach().requires_grad_(True), w.detach().requires_grad_(True)
    f = L.linear_cross_entropy if "targets" in kw else L.linear_distillation
    out = f(h, w, reduction=reduction, **kw)
    dh, dw = torch.autograd.grad(out, (h, w), up if reduction == "none" else up.reshape(()))
    return out.detach(), dh, dw


def compare(h, w, dt, reduction, up, op, **kw):
    if op == "xent":
        got = run(h, w, reduction, up, targets=kw["targets"], label_smoothing=kw.get("e", 0.0))
    else:
        got = run(h, w, reduction, up, teacher_logits=kw["tl"], teacher_indices=kw["idx"],
                  temperature=kw.get("T", 1.0))
    want = definition(h, w, dt, reduction, up, **kw)
    for a, b, name in zip(got, want, ("loss", "dh", "dW")):
        check(a, b, name)
    return got


def upstream(n, reduction, g):
    if reduction == "none":
        return torch.randn(n, device="cuda", generator=g)
    return torch.tensor(1.7, device="cuda")


SIZES = [(1, 1, 1), (1, 1000, 64), (3, 37, 5), (17, 301, 72), (48, 2048, 128), (65, 513, 130),
         (100, 1031, 67), (200, 4099, 256), (300, 700, 515), (513, 5000, 64)]


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,v,d", SIZES)
def test_cross_entropy(n, v, d, dt):
    print("case xent", n, v, d, dt, flush=True)
    h, w, t, g = make(n, v, d, dt, seed=n + v)
    for reduction, e, ign in (("mean", 0.0, 0.3), ("none", 0.1, 0.0), ("sum", 0.0, 0.0)):
        tt = torch.where(torch.rand(n, device="cuda", generator=g) < ign, IGN, t)
        compare(h, w, dt, reduction, upstream(n, reduction, g), "xent", targets=tt, e=e)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,v,d", SIZES)
def test_distillation(n, v, d, dt):
    print("case distill", n, v, d, dt, flush=True)
    h, w, _, g = make(n, v, d, dt, seed=n + v + 1)
    for reduction, k, T in (("mean", 8, 2.0), ("none", 1, 0.7), ("sum", 33, 1.0)):
        tl, idx = teacher(n, v, k, g, DT[dt])
        compare(h, w, dt, reduction, upstream(n, reduction, g), "distill", tl=tl, idx=idx, T=T)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_several_pieces_of_the_vocabulary(dt):
    n, v, d = (8200, 33000, 64) if dt == "bf16" else (4100, 33000, 40)
    print("case pieces", n, v, d, dt, flush=True)
    h, w, t, g = make(n, v, d, dt, seed=5)
    t[::3] = IGN
    compare(h, w, dt, "mean", upstream(n, "mean", g), "xent", targets=t, e=0.1)
    tl, idx = teacher(n, v, 5, g)
    compare(h, w, dt, "none", upstream(n, "none", g), "distill", tl=tl, idx=idx, T=1.5)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_large_tiles(dt):
    """Sizes whose three products all take the largest tiles, none a multiple of them."""
    n, v, d = 2100, 4500, 2056
    print("case large tiles", dt, flush=True)
    h, w, t, g = make(n, v, d, dt, seed=6)
    t[100:400] = IGN
    compare(h, w, dt, "mean", upstream(n, "mean", g), "xent", targets=t)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_strides_and_alignment(dt):
    n, v, d = 130, 777, 96
    print("case strides", dt, flush=True)
    h0, w0, t, g = make(n, v, d + 40, dt, seed=7)
    up = upstream(n, "mean", g)
    for a, b in ((0, 0), (8, 16), (3, 5), (1, 0)):
        h, w = h0[:, a:a + d], w0[:, b:b + d]
        assert not h.is_contiguous()
        compare(h, w, dt, "mean", up, "xent", targets=t)
    # rows in reverse memory order and columns first: not a layout the kernels read, copied
    ht = h0[:, :d].t().contiguous().t()
    compare(ht, w0[:, :d], dt, "mean", up, "xent", targets=t)
    # leading dimensions
    h3 = h0[:, :d].reshape(2, 65, d)
    got = L.linear_cross_entropy(h3, w0[:, :d], t.reshape(2, 65), reduction="none")
    assert got.shape == (2, 65)
    ref = L.linear_cross_entropy(h0[:, :d], w0[:, :d], t, reduction="none")
    assert torch.equal(got.reshape(-1), ref)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_positions_that_do_not_count_leave_nothing_behind(dt):
    n, v, d = 70, 300, 64
    print("case ignored", dt, flush=True)
    h, w, t, g = make(n, v, d, dt, seed=8)
    t[::2] = IGN
    clean = run(h, w, "mean", torch.tensor(1.0, device="cuda"), targets=t)
    bad = h.clone()
    for i, x in enumerate((float("nan"), float("inf"), -float("inf"), torch.finfo(DT[dt]).max,
                           torch.finfo(DT[dt]).min)):
        bad[2 * i] = x
    got = run(bad, w, "mean", torch.tensor(1.0, device="cuda"), targets=t)
    for a, b in zip(got, clean):
        assert torch.equal(a, b)
    assert (got[1][::2] == 0).all()
    # none counts: a mean of nothing is 0, and so is every gradient
    for red in ("mean", "sum", "none"):
        up = torch.ones(n if red == "none" else (), device="cuda")
        o, dh, dw = run(bad, w, red, up, targets=torch.full_like(t, IGN))
        assert (o == 0).all() and (dh == 0).all() and (dw == 0).all()
        o, dh, dw = run(bad, w, red, up, teacher_logits=torch.zeros(n, 4, device="cuda"),
                        teacher_indices=torch.full((n, 4), -1, device="cuda"))
        assert (o == 0).all() and (dh == 0).all() and (dw == 0).all()


def test_no_positions():
    print("case empty", flush=True)
    w = torch.randn(50, 16, device="cuda").bfloat16()
    h = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16)
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    for red in ("mean", "sum", "none"):
        up = torch.ones(0 if red == "none" else (), device="cuda")
        o, dh, dw = run(h, w, red, up, targets=t)
        assert o.shape == ((0,) if red == "none" else ()) and (o == 0).all()
        assert dh.shape == (0, 16) and (dw == 0).all()


def test_bad_indices_are_flagged_and_skipped():
    print("case bad indices", flush=True)
    n, v, d = 40, 200, 32
    h, w, t, g = make(n, v, d, "fp32", seed=9)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    L.linear_cross_entropy(h, w, t, dev_status=st)
    assert int(st) == 0
    t2 = t.clone()
    t2[3], t2[7] = v, -5
    ref = t.clone()
    ref[3] = ref[7] = IGN
    a = L.linear_cross_entropy(h, w, t2, reduction="none", dev_status=st)
    assert int(st) == abi.TT_DEV_BAD_INDEX
    assert torch.equal(a, L.linear_cross_entropy(h, w, ref, reduction="none"))
    st.zero_()
    tl, idx = teacher(n, v, 6, g)
    b = L.linear_distillation(h, w, tl, idx, reduction="none", dev_status=st)
    assert int(st) == 0
    idx2 = torch.where(idx < 0, v + 3, idx)
    c = L.linear_distillation(h, w, tl, idx2, reduction="none", dev_status=st)
    assert int(st) == abi.TT_DEV_BAD_INDEX and torch.equal(b, c)


def test_ignore_index_inside_the_vocabulary():
    print("case ignore index", flush=True)
    h, w, t, _ = make(33, 90, 24, "fp32", seed=10)
    t[5:9] = 7
    a = L.linear_cross_entropy(h, w, t, ignore_index=7, reduction="none")
    b = L.linear_cross_entropy(h, w, torch.where(t == 7, IGN, t), reduction="none")
    assert torch.equal(a, b)


def test_teacher_masks():
    """Logits of -inf are no entries; the type's lowest value is one of weight 0."""
    print("case teacher masks", flush=True)
    n, v, d, k = 20, 150, 48, 6
    h, w, _, g = make(n, v, d, "fp32", seed=11)
    tl, idx = teacher(n, v, k, g)
    idx = idx.abs() % v
    tl[:, 2] = -math.inf
    tl[4] = -math.inf          # a row whose mask leaves nothing
    tl[:, 3] = torch.finfo(torch.float32).min
    tl[4, 3] = -math.inf
    up = upstream(n, "none", g)
    out, dh, _ = compare(h, w, "fp32", "none", up, "distill", tl=tl, idx=idx, T=1.0)
    assert float(out[4]) == 0 and (dh[4] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
def test_large_and_far_logits(dt):
    """Logits in the thousands (exp of a raw logit overflows, most probabilities underflow) and
    factors of the loss over a wide range."""
    print("case far logits", dt, flush=True)
    n, v, d = 90, 1500, 64
    h, w, t, g = make(n, v, d, dt, seed=12, scale=200.0)
    compare(h, w, dt, "sum", upstream(n, "sum", g), "xent", targets=t)
    up = torch.randn(n, device="cuda", generator=g) * 10.0 ** torch.linspace(-3, 1, n, device="cuda")
    compare(h / 200, w, dt, "none", up, "xent", targets=t, e=0.1)


def test_nan_reaches_only_its_position():
    print("case nan", flush=True)
    h, w, t, _ = make(30, 100, 32, "bf16", seed=13)
    clean = L.linear_cross_entropy(h, w, t, reduction="none")
    h[4, 3] = float("nan")
    out = L.linear_cross_entropy(h, w, t, reduction="none")
    assert torch.isnan(out[4])
    keep = torch.arange(30, device="cuda") != 4
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_gradients_against_differences(op):
    """Central differences of the fp32 loss, taken in float64 from the definition: the returned
    gradient gives the change along random directions."""
    print("case differences", op, flush=True)
    n, v, d = 24, 130, 20
    h, w, t, g = make(n, v, d, "fp32", seed=14)
    up = torch.tensor(1.0, device="cuda")
    if op == "xent":
        kw = dict(targets=t, e=0.1)
        got = run(h, w, "mean", up, targets=t, label_smoothing=0.1)
    else:
        tl, idx = teacher(n, v, 7, g)
        kw = dict(tl=tl, idx=idx, T=2.0)
        got = run(h, w, "mean", up, teacher_logits=tl, teacher_indices=idx, temperature=2.0)
    for which in (0, 1):
        x = (h, w)[which].double()
        r = torch.randn(x.shape, device="cuda", generator=g, dtype=torch.float64)
        s = 1e-4
        f = [definition(*((x + a * r, w.double()) if which == 0 else (h.double(), x + a * r)),
                        "fp32", "mean", up, **kw)[0][0] for a in (s, -s)]
        num = float(f[0] - f[1]) / (2 * s)
        ana = float((got[1 + which].double() * r).sum())
        # second-order term of a central difference (s^2) and the gradient's own 2^-20
        scale = float((got[1 + which].double() * r).abs().sum())
        assert abs(num - ana) <= 1e-6 * scale + 1e-9


def test_repeated_calls_give_the_same_bits():
    print("case repeat", flush=True)
    h, w, t, _ = make(700, 3001, 200, "bf16", seed=15)
    up = torch.tensor(1.0, device="cuda")
    a = run(h, w, "mean", up, targets=t)
    for _ in range(3):
        b = run(h, w, "mean", up, targets=t)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_only_the_gradient_that_is_asked_for():
    print("case one gradient", flush=True)
    h, w, t, _ = make(80, 400, 64, "bf16", seed=16)
    up = torch.tensor(1.0, device="cuda")
    _, dh, dw = run(h, w, "mean", up, targets=t)
    x = h.detach().requires_grad_(True)
    assert torch.equal(torch.autograd.grad(L.linear_cross_entropy(x, w, t), x)[0], dh)
    y = w.detach().requires_grad_(True)
    assert torch.equal(torch.autograd.grad(L.linear_cross_entropy(h, y, t), y)[0], dw)
    with torch.no_grad():
        assert not L.linear_cross_entropy(x, y, t).requires_grad


def test_another_stream():
    print("case stream", flush=True)
    h, w, t, _ = make(300, 2000, 128, "fp16", seed=17)
    up = torch.tensor(1.0, device="cuda")
    ref = run(h, w, "mean", up, targets=t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(h, w, "mean", up, targets=t)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(ref, got))


@pytest.mark.parametrize("n", [20, 600])
def test_captured_calls(n):
    """Forward and backward through the C ABI captured into one graph (caller's buffers),
    replayed on new inputs between eager calls."""
    print("case graph", n, flush=True)
    v, d = 3000, 128
    h, w, t, g = make(n, v, d, "bf16", seed=18)
    desc = abi.make_loss_desc(h, w)
    sizes = abi.tt_loss_sizes(desc, w)
    buf = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes]
    loss = torch.empty(1, device="cuda")
    dh, dw, one = torch.empty_like(h), torch.empty_like(w), torch.ones(1, device="cuda")

    def step():
        abi.tt_loss_forward(desc, h, w, t, loss=loss, saved=buf[0], ws=buf[1])
        abi.tt_loss_backward(desc, h, w, buf[0], one, dh, dw, ws=buf[2])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        h2, w2, t2, _ = make(n, v, d, "bf16", seed=19 + k)
        t2[k::5] = IGN
        h.copy_(h2), w.copy_(w2), t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        ref = run(h, w, "mean", one, targets=t)
        assert torch.equal(loss[0], ref[0]) and torch.equal(dh, ref[1]) and torch.equal(dw, ref[2])


@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("n,d", [(1, 64), (5, 200), (64, 72), (63, 67), (64, 8), (65, 64)])
def test_loss_alone(n, d, op):
    """Without gradients the loss takes a shorter path for few positions; its values stay
    within the same bound, ignored rows (NaN in them) and flagged ones included."""
    print("case loss alone", n, d, op, flush=True)
    v = 500
    h, w, t, g = make(n, v, d, "bf16", seed=n + d)
    if n > 2:
        t[1] = IGN
        h[1] = float("nan")
    tl, idx = teacher(n, v, 6, g, torch.bfloat16)
    if n > 2:
        idx[1] = -1
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for red in ("none", "mean", "sum"):
        up = torch.ones(n if red == "none" else (), device="cuda")
        if op == "xent":
            got = L.linear_cross_entropy(h, w, t, label_smoothing=0.1, reduction=red,
                                         dev_status=st)
            want = definition(torch.nan_to_num(h), w, "bf16", red, up, targets=t, e=0.1)[0]
        else:
            got = L.linear_distillation(h, w, tl, idx, temperature=2.0, reduction=red,
                                        dev_status=st)
            want = definition(torch.nan_to_num(h), w, "bf16", red, up, tl=tl, idx=idx, T=2.0)[0]
        check(got, want, red)
    assert int(st) == 0
    if op == "xent" and n > 2:
        t[0] = v
        got = L.linear_cross_entropy(h, w, t, reduction="none", dev_status=st)
        assert int(st) == abi.TT_DEV_BAD_INDEX and float(got[0]) == 0 and float(got[1]) == 0


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 2, 31, 32])
def test_few_positions_keep_what_rounding_left(n, dt):
    """Up to 32 positions the gradient of the logits enters the products as two 16-bit parts:
    dh and dW are then off by their own rounding (u) and the second part's (2 u^2 of a part's
    terms, with the fp32 terms of `definition`), ignored positions among them or not."""
    print("case few positions", n, dt, flush=True)
    h, w, t, g = make(n, 700, 136, dt, seed=n)
    if n > 3:
        t[1] = t[n - 1] = IGN
    up = upstream(n, "none", g)
    got = run(h, w, "none", up, targets=t, label_smoothing=0.1)
    keep = U[dt]
    U[dt] = 2 * keep * keep
    try:
        _, (dh, bh), (dw, bw) = definition(h, w, dt, "none", up, targets=t, e=0.1)
    finally:
        U[dt] = keep
    check(got[1], (dh, bh + keep * dh.abs()), "dh")
    check(got[2], (dw, bw + keep * dw.abs()), "dW")


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n", [1, 70])
def test_confident_positions(n, dt):
    """Losses of 1e-4 to 1e-2, where lse and the target's logit agree in most digits.  The
    target's logit is the one in the sum, so a loss is off by the sum's own rounding (some 8
    terms of 2^-24 of a sum near 1) and by its logits' errors times the share of the others:
    2^-20 + loss * dz."""
    print("case confident", n, dt, flush=True)
    v, d = 4000, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    w = (torch.randn(v, d, device="cuda", generator=g) * d ** -0.5).to(DT[dt])
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    h = (w[t].float() * (15.0 + 3 * torch.rand(n, 1, device="cuda", generator=g))).to(DT[dt])
    got = L.linear_cross_entropy(h, w, t, reduction="none").double()
    hg = h.detach().requires_grad_(True)
    assert torch.equal(L.linear_cross_entropy(hg, w, t, reduction="none").detach().double(), got)
    ref = torch.nn.functional.cross_entropy(h.double() @ w.double().t(), t, reduction="none")
    dz = 2 * (d * 2.0 ** -24 + (2.0 ** -21 if dt == "fp32" else 0)) * \
        (h.double().abs() @ w.double().abs().t()).amax(1)
    assert float(ref.min()) < 2e-2
    assert float(((got - ref).abs() / (2.0 ** -20 + ref * dz)).max()) <= 1
