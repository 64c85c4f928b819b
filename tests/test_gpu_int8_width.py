"""Sums of 8-bit products at the ends of 32 bits: values given as -128 in both operands, and quantised tokens
against a table of -128.  The sums are whole numbers, rounded to float32 once; scales of 1 leave them as they are."""
import pytest
import torch

from tensor_train_compressed_ttembeddingbag_amd import abi
from tensor_train_compressed_ttembeddingbag_amd.quant import Int8Rows, int8_linear

pytestmark = pytest.mark.gpu


def rows(values):
    return Int8Rows(values, torch.ones(len(values), device="cuda"))


@pytest.mark.parametrize("n", [2, 150])
def test_given_values(n):
    d = (1 << 17) - 1
    x = torch.full((n, d), -128, dtype=torch.int8, device="cuda")
    x[1] = 127
    w = torch.full((130, d), -128, dtype=torch.int8, device="cuda")
    out = int8_linear(rows(x), rows(w))
    want = torch.full((n, 130), float(128 * 128 * d))
    want[1] = float(-127 * 128 * d)
    assert torch.equal(out.cpu(), want)


def test_one_column_more_is_refused():
    x = torch.full((2, 1 << 17), -128, dtype=torch.int8, device="cuda")
    with pytest.raises(abi.TTError):
        int8_linear(rows(x), rows(x))


def test_quantised_tokens():
    d = 1 << 17
    x = torch.full((2, d), 127.0, device="cuda")  # a scale of 1
    x[1] = -127.0
    w = torch.full((130, d), -128, dtype=torch.int8, device="cuda")
    out = int8_linear(x, rows(w))
    assert bool((out[0] == -127.0 * 128 * d).all()) and bool((out[1] == 127.0 * 128 * d).all())
