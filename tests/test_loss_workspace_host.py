"""The workspaces of the vocabulary-head losses are those of a piece of the vocabulary, in every
mode, as include/tt_bag.h states them."""
import ctypes

import pytest

from tensor_train_compressed_ttembeddingbag_amd import abi
from test_loss_host import desc

MIB = 1 << 20


def up(x, m):
    return (x + m - 1) // m * m


@pytest.mark.parametrize("kw", [dict(), dict(label_smoothing=0.1), dict(dtype=abi.TT_DTYPE_F32),
                                dict(dtype=abi.TT_DTYPE_F32, label_smoothing=0.1),
                                dict(d=63, hidden_stride=63, weight_stride=63),
                                dict(k=64, temperature=2.0), dict(k=1), dict(reduction=abi.TT_REDUCE_NONE)],
                         ids=str)
@pytest.mark.parametrize("n", [1, 64, 100, 8192, 1 << 20, 1 << 23])
def test_bounds(n, kw):
    lib = abi.lib()
    for v in (1000, 1 << 17, 1 << 20, 1 << 24, 1 << 30):
        d = desc(n=n, v=v, **kw)
        fwd, bwd, only = (lib.tt_loss_workspace_size(ctypes.byref(d), None, m) for m in range(3))
        saved = lib.tt_loss_saved_size(ctypes.byref(d))
        size = 4 if d.dtype == abi.TT_DTYPE_F32 else 2
        rows, wide = up(n, 256), up(d.d, 64)
        packed = 256 * MIB + 256 * wide * size  # (pieces are whole groups of 256 rows)
        other = 64 * rows + MIB
        assert 0 < fwd <= 256 * MIB + packed + other
        assert fwd <= only <= fwd + saved + other
        grad = max(256 * MIB, 256 * rows * size) + 256 * rows * size
        sums = max(4 * rows * up(d.d, 64), 1024 * 4 * 65536)
        assert 0 < bwd <= grad + packed + sums + other
        if v <= 1 << 17 and n <= 8192:  # ordinary sizes keep all statistics, one pass over them
            assert fwd < 256 * MIB


def test_null_weight():
    d = desc()
    assert abi.lib().tt_loss_workspace_size(ctypes.byref(d), None, 1) == \
        abi.lib().tt_loss_workspace_size(ctypes.byref(d), 0x10001, 1) > 0
