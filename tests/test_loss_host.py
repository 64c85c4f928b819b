"""Refusals of the vocabulary-head losses, on the host: the C entry points reject descriptors,
pointers and workspaces before any device work, and the public functions their arguments."""
import ctypes

import pytest
import torch

from tensor_train_compressed_ttembeddingbag_amd import abi, loss as L

FAKE = 0x10000  # 256-byte aligned, never dereferenced


def desc(**kw):
    d = dict(n=10, v=100, d=64, hidden_stride=64, weight_stride=64, ignore_index=-100,
             dtype=abi.TT_DTYPE_BF16, teacher_dtype=abi.TT_DTYPE_F32,
             reduction=abi.TT_REDUCE_MEAN, k=0, label_smoothing=0.0, temperature=1.0)
    d.update(kw)
    return abi.TTLossDesc(*[d[f[0]] for f in abi.TTLossDesc._fields_])


BAD = [(-1, dict(n=-1)), (-1, dict(v=0)), (-1, dict(d=0)), (-1, dict(k=-1)), (-1, dict(dtype=3)),
       (-1, dict(dtype=-1)), (-1, dict(teacher_dtype=9)), (-1, dict(reduction=3)),
       (-1, dict(label_smoothing=1.5)), (-1, dict(label_smoothing=float("nan"))),
       (-1, dict(temperature=2.0)), (-1, dict(k=4, temperature=0.0)),
       (-1, dict(k=4, temperature=float("inf"))), (-1, dict(k=4, temperature=float("nan"))),
       (-1, dict(k=4, label_smoothing=0.1)), (-1, dict(hidden_stride=63)),
       (-1, dict(weight_stride=63)), (-2, dict(k=4096)), (-2, dict(n=1 << 24)),
       (-2, dict(v=1 << 31)), (-2, dict(weight_stride=1 << 22)),
       (-2, dict(n=1 << 22, k=1024)), (-2, dict(d=1 << 21, hidden_stride=1 << 21,
                                               weight_stride=1 << 21))]


@pytest.mark.parametrize("code,kw", BAD, ids=[str(b[1]) for b in BAD])
def test_bad_descriptors(code, kw):
    lib, d = abi.lib(), desc(**kw)
    r = ctypes.byref(d)
    assert lib.tt_loss_saved_size(r) == 0
    assert lib.tt_loss_workspace_size(r, FAKE, 0) == 0
    big = 1 << 40
    assert lib.tt_loss_forward(r, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, big, FAKE, big, None,
                               None) == code
    assert lib.tt_loss_backward(r, FAKE, FAKE, FAKE, big, FAKE, FAKE, FAKE, FAKE, big,
                                None) == code


def test_bad_pointers_and_workspaces():
    lib = abi.lib()
    d, dk = desc(), desc(k=4, temperature=2.0)
    r, rk = ctypes.byref(d), ctypes.byref(dk)
    big = 1 << 40
    args = [FAKE] * 6 + [big, FAKE, big, None, None]

    def fwd(ref, **kw):
        a = list(args)
        for k, x in kw.items():
            a[int(k[1:])] = x
        return lib.tt_loss_forward(ref, *a)

    for i in (0, 1, 2, 4, 7):
        assert fwd(r, **{"a%d" % i: None}) == -1, i
    assert fwd(rk, a3=None) == -1
    assert fwd(r, a0=FAKE + 1) == -1 and fwd(r, a1=FAKE + 1) == -1
    assert fwd(r, a5=FAKE + 16) == -3 and fwd(r, a7=FAKE + 16) == -3
    assert fwd(r, a6=lib.tt_loss_saved_size(r) - 1) == -3
    assert fwd(r, a8=lib.tt_loss_workspace_size(r, FAKE, 0) - 1) == -3
    # without saved the workspace is another one
    assert fwd(r, a5=None, a6=0, a8=lib.tt_loss_workspace_size(r, FAKE, 2) - 1) == -3
    assert lib.tt_loss_workspace_size(r, FAKE, 3) == 0
    assert lib.tt_loss_forward(None, *args) == -1

    bargs = [FAKE, FAKE, FAKE, big, FAKE, FAKE, FAKE, FAKE, big, None]

    def bwd(**kw):
        a = list(bargs)
        for k, x in kw.items():
            a[int(k[1:])] = x
        return lib.tt_loss_backward(r, *a)

    for i in (0, 1, 2, 4, 7):
        assert bwd(**{"a%d" % i: None}) == -1, i
    assert bwd(a5=FAKE + 1) == -1 and bwd(a6=FAKE + 1) == -1
    assert bwd(a2=FAKE + 16) == -3 and bwd(a7=FAKE + 16) == -3
    assert bwd(a3=lib.tt_loss_saved_size(r) - 1) == -3
    assert bwd(a8=lib.tt_loss_workspace_size(r, FAKE, 1) - 1) == -3


def test_workspace_is_bounded_in_the_vocabulary():
    """The workspace is that of one piece of the vocabulary, not of the logits."""
    lib = abi.lib()
    for kw in (dict(), dict(dtype=abi.TT_DTYPE_F32), dict(d=63, hidden_stride=63)):
        sizes = [lib.tt_loss_workspace_size(ctypes.byref(desc(n=8192, v=v, **kw)), FAKE, 1)
                 for v in (1 << 17, 1 << 20, 1 << 24)]
        assert 0 < max(sizes) < 800 << 20
        assert max(sizes) - min(sizes) < 64 << 20


def test_public_functions_refuse_bad_arguments():
    h, w = torch.zeros(4, 8), torch.zeros(20, 8)
    t = torch.zeros(4, dtype=torch.int64)
    tl, ti = torch.zeros(4, 3), torch.zeros(4, 3, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        L.linear_cross_entropy(h, w, t)
    with pytest.raises(ValueError, match="reduction"):
        L.linear_cross_entropy(h, w, t, reduction="avg")
    with pytest.raises(ValueError, match="targets"):
        L.linear_cross_entropy(h, w, t[:3])
    with pytest.raises(ValueError, match="label_smoothing"):
        L.linear_cross_entropy(h, w, t, label_smoothing=-0.1)
    with pytest.raises(ValueError, match="GPU"):
        L.linear_distillation(h, w, tl, ti)
    with pytest.raises(ValueError, match="same shape"):
        L.linear_distillation(h, w, tl[:, :2], ti)
    with pytest.raises(ValueError, match="teacher_indices"):
        L.linear_distillation(h, w, tl[:3], ti[:3])
    with pytest.raises(ValueError, match="temperature"):
        L.linear_distillation(h, w, tl, ti, temperature=0.0)
    with pytest.raises(ValueError, match="temperature"):
        L.linear_distillation(h, w, tl, ti, temperature=float("nan"))
    with pytest.raises(ValueError, match="entry"):
        L.linear_distillation(h, w, tl[:, :0], ti[:, :0])
    with pytest.raises(TypeError, match="teacher_logits"):
        L.linear_distillation(h, w, tl.double(), ti)


def test_sizes_without_positions():
    lib = abi.lib()
    for kw in (dict(n=0), dict(n=0, dtype=abi.TT_DTYPE_F32), dict(n=0, k=5)):
        r = ctypes.byref(desc(**kw))
        assert lib.tt_loss_saved_size(r) > 0
        assert lib.tt_loss_workspace_size(r, FAKE, 0) > 0
        assert lib.tt_loss_workspace_size(r, FAKE, 1) > 0
