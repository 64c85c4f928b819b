"""The widest products in 8 bits on the host: sums of values that are given may reach 128^2 a column, so their
width ends one column earlier, where 128^2 (2^17 - 1) < 2^31."""
import ctypes

import pytest

from tensor_train_compressed_ttembeddingbag_amd import abi


@pytest.mark.parametrize("dtype,d,fits", [(abi.TT_DTYPE_I8, 1 << 17, False), (abi.TT_DTYPE_I8, (1 << 17) - 1, True),
                                          (abi.TT_DTYPE_F32, 1 << 17, True)])
def test_width(dtype, d, fits):
    desc = abi.TTInt8Desc(10, 100, d, 1 << 17, 1 << 17, dtype, abi.TT_DTYPE_F32)
    assert (abi.lib().tt_int8_workspace_size(ctypes.byref(desc)) > 0) == fits
