"""Vocabulary-head losses of views: rows far apart, odd offsets and strides, with and without
gradients, equal bit for bit to those of contiguous copies."""
import pytest
import torch

from tensor_train_compressed_ttembeddingbag_amd import loss as L
from test_gpu_loss_range import check, inputs

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def same(h, w, t):
    """Loss alone and with gradients of the views and of contiguous copies."""
    hc, wc = h.contiguous(), w.contiguous()
    for smoothing in (0.0, 0.1):
        kw = dict(reduction="none", label_smoothing=smoothing)
        a = L.linear_cross_entropy(h, w, t, **kw)
        assert torch.equal(a, L.linear_cross_entropy(hc, wc, t, **kw))
        assert torch.isfinite(a).all()
    tl, idx = torch.zeros(*t.shape, 3, device="cuda"), (t[..., None] + torch.arange(3, device="cuda")) % len(w)
    assert torch.equal(L.linear_distillation(h, w, tl, idx), L.linear_distillation(hc, wc, tl, idx))
    grads = []
    for x, y in ((h, w), (hc, wc)):
        x, y = x.detach().requires_grad_(True), y.detach().requires_grad_(True)
        grads.append(torch.autograd.grad(L.linear_cross_entropy(x, y, t), (x, y)))
    assert all(torch.equal(p, q) for p, q in zip(*grads))


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("last", [-1, slice(-1, None)])
def test_last_token_of_each_sequence(last, dt):
    """hidden[B, T, D][:, -1]: rows T D = 2.2 million elements apart."""
    print("case last token", last, dt, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    h = torch.randn(3, 1100, 2048, device="cuda", generator=g).to(DT[dt])[:, last]
    w = (torch.randn(500, 2048, device="cuda", generator=g) / 45).to(DT[dt])
    same(h, w, torch.randint(0, 500, h.shape[:-1], device="cuda", generator=g))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_weight_rows_far_apart(dt):
    print("case far weight", dt, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    w = torch.zeros(20, (1 << 21) + 8, device="cuda", dtype=DT[dt])[:, :64]
    w.copy_(torch.randn(20, 64, device="cuda", generator=g))
    h = torch.randn(70, 64, device="cuda", generator=g).to(DT[dt])
    same(h, w, torch.randint(0, 20, (70,), device="cuda", generator=g))


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 33, 64, 65])
def test_few_positions_of_any_stride_and_offset(n, dt):
    print("case offsets", n, dt, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    big_h = torch.randn(n, 117, device="cuda", generator=g).to(DT[dt])
    big_w = torch.randn(700, 131, device="cuda", generator=g).to(DT[dt])
    t = torch.randint(0, 700, (n,), device="cuda", generator=g)
    for d in (8, 64, 96):
        for a, b in ((0, 0), (3, 0), (0, 5), (1, 7)):
            same(big_h[:, a:a + d], big_w[:, b:b + d], t)


@pytest.mark.parametrize("share", [0.0, 0.4, 1.0])
@pytest.mark.parametrize("n", [8192, 8193, 9217, 40000])
def test_many_positions_keep_their_order(n, share):
    """Past 8192 positions the ones that count are counted by chunks: every position keeps its own
    loss and gradient, whatever else counts."""
    print("case order", n, share, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    h = torch.randn(n, 16, device="cuda", generator=g).bfloat16()
    w = torch.randn(90, 16, device="cuda", generator=g).bfloat16()
    t = torch.randint(0, 90, (n,), device="cuda", generator=g)
    skip = torch.rand(n, device="cuda", generator=g) < share
    t[skip] = -100
    x = h.clone().requires_grad_(True)
    out = L.linear_cross_entropy(x, w, t, reduction="none")
    dh, = torch.autograd.grad(out.sum(), x)
    z = h.double() @ w.double().t()
    ref = torch.nn.functional.cross_entropy(z, t, reduction="none", ignore_index=-100)
    # D + V rounded sums of terms within 60: 2^-24 (16 + 90) 60 and the logs
    assert float((out.detach().double() - ref).abs().max()) <= 2.0 ** -24 * 106 * 60
    assert (dh[skip] == 0).all() and (skip.all() or (dh[~skip].abs().amax(1) > 0).float().mean() > 0.9)
    mean = L.linear_cross_entropy(h, w, t)
    count = max(1, int((~skip).sum()))
    assert abs(float(mean) - float(ref.sum()) / count) <= 2.0 ** -20 * float(ref.sum()) / count


def test_time_of_many_positions():
    """The positions are counted in linear time: 2^20 of them take less than a tenth of the
    76 ms that a count per block took."""
    print("case linear", flush=True)
    n = 1 << 20
    h = torch.zeros(n, 64, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(200, 64, device="cuda", dtype=torch.bfloat16)
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    L.linear_cross_entropy(h, w, t)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    L.linear_cross_entropy(h, w, t)
    b.record()
    torch.cuda.synchronize()
    assert a.elapsed_time(b) < 7.6


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("at", [0, 19999])
def test_gradients_of_many_positions(at, dt):
    """Past 16384 positions the largest gradient is found ahead, wherever it lies."""
    print("case many factors", at, dt, flush=True)
    n, v, d = 20000, 90, 16
    h, w, t, g = inputs(n, v, d, 4, dt)
    up = torch.rand(n, device="cuda", generator=g) + 0.1
    up[at] = 1e4
    check(h, w, dt, t=t, up=up, step=2.0 ** -34)


def test_time_of_gradients_of_many_positions():
    """Linear as well: 2^20 positions' dhidden took 4.1 ms where every block looked for the
    largest gradient."""
    print("case linear backward", flush=True)
    n = 1 << 20
    h = torch.zeros(n, 64, device="cuda", dtype=torch.float16).requires_grad_(True)
    w = torch.zeros(200, 64, device="cuda", dtype=torch.float16)
    t = torch.zeros(n, dtype=torch.int64, device="cuda")
    up = torch.ones(n, device="cuda")
    out = L.linear_cross_entropy(h, w, t, reduction="none")
    torch.autograd.grad(out, h, up, retain_graph=True)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record()
    torch.autograd.grad(out, h, up)
    b.record()
    torch.cuda.synchronize()
    assert a.elapsed_time(b) < 3.0


@pytest.mark.parametrize("smoothing", [0.0, 0.1])
@pytest.mark.parametrize("n,v,d,dt", [(8192, 1_100_000, 8, "bf16"), (5, 68_000_000, 8, "bf16"),
                                      (8192, 1_100_000, 12, "fp32")])
def test_vocabularies_whose_statistics_are_added_up_by_pieces(n, v, d, dt, smoothing):
    """1000 distinct rows over and over: lse is that of the distinct ones and the log of their
    number (uneven at the end: counted).  Bound: D + 2 log2 V rounded sums of logits within 30,
    and the smoothing's mean, V / 256 tiles of fp32 sums within 30 of each."""
    print("case many tiles", n, v, d, dt, smoothing, flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    some = torch.randn(1000, d, device="cuda", generator=g).to(DT[dt])
    w = some.repeat((v + 999) // 1000, 1)[:v]
    h = torch.randn(n, d, device="cuda", generator=g).to(DT[dt])
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    if n > 10:
        t[7::11] = -100
    z = h.double() @ some.double().t()
    many = torch.full((1000,), v // 1000, device="cuda", dtype=torch.float64)
    many[: v % 1000] += 1
    lse = torch.logsumexp(z + many.log(), 1)
    ref = lse - (1 - smoothing) * z.gather(1, (t.clamp(min=0) % 1000)[:, None])[:, 0] \
        - smoothing * (z * many).sum(1) / v
    ref = torch.where(t >= 0, ref, torch.zeros_like(ref))
    bound = 2.0 ** -24 * (d + 50) * 30 + (2.0 ** -21 * 30 if dt == "fp32" else 0) + \
        smoothing * 2.0 ** -24 * 300 * 30
    out = L.linear_cross_entropy(h, w, t, reduction="none", label_smoothing=smoothing)
    assert float((out.double() - ref).abs().max()) <= bound
    x = h.clone().requires_grad_(True)
    kept = L.linear_cross_entropy(x, w, t, reduction="none", label_smoothing=smoothing)
    assert float((kept.detach().double() - ref).abs().max()) <= bound


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_hidden_states_are_not_kept_beside_their_packed_copy(dt):
    """The backward reads the packed rows alone: hidden states that are overwritten after the
    forward change nothing, and given up they are freed."""
    print("case kept", dt, flush=True)
    h, w, t, _ = inputs(1000, 300, 512, 7, dt)
    w.requires_grad_(True)
    want = torch.autograd.grad(L.linear_cross_entropy(x := h.clone().requires_grad_(True), w, t), (x, w))
    y = x * 1
    out = L.linear_cross_entropy(y, w, t)
    size = y.numel() * y.element_size()
    y.detach().zero_()
    before = torch.cuda.memory_allocated()
    del y
    assert before - torch.cuda.memory_allocated() >= size
    got = torch.autograd.grad(out, (x, w))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = x * 1
    out = L.linear_cross_entropy(y, w, t)
    y.zero_()
    got = torch.autograd.grad(out, (x, w))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
