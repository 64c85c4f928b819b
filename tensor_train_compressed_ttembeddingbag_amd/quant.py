"""Tables in 8-bit integers: a scale for every row.

``Int8Rows`` holds a table as int8 values [R, D] and one float32 scale a row; the row it stands
for is ``values[r] * scales[r]``.  ``embedding`` looks its rows up.
"""
from __future__ import annotations

import torch


class Int8Rows:
    """int8 values [R, D] and float32 scales [R] on the GPU.

    The rows of values have unit stride inside and lie a multiple of 16 bytes apart, from a
    multiple of 16 on; the last one's memory reaches to that distance too.  Values laid out
    otherwise are copied."""

    __slots__ = ("values", "scales")

    def __init__(self, values: torch.Tensor, scales: torch.Tensor):
        for t, dt, dim, name in ((values, torch.int8, 2, "values"),
                                 (scales, torch.float32, 1, "scales")):
            if not isinstance(t, torch.Tensor):
                raise TypeError("%s must be a torch.Tensor" % name)
            if t.dtype != dt:
                raise TypeError("%s must be %s, got %s" % (name, dt, t.dtype))
            if t.dim() != dim:
                raise ValueError("%s must have %d dimension(s)" % (name, dim))
        if not values.is_cuda or values.device != scales.device:
            raise ValueError("values and scales must be on one GPU")
        rows, d = values.shape
        if rows < 1 or d < 1:
            raise ValueError("values is empty")
        if scales.shape[0] != rows:
            raise ValueError("%d rows of values, %d scales" % (rows, scales.shape[0]))
        stride = values.stride(0)
        if (stride % 16 or stride < d or values.data_ptr() % 16
                or d > 1 and values.stride(1) != 1
                or values.storage_offset() + rows * stride > values.untyped_storage().nbytes()):
            copy = torch.zeros(rows, (d + 15) // 16 * 16, dtype=torch.int8, device=values.device)
            copy[:, :d] = values
            values = copy[:, :d]
        self.values, self.scales = values, scales.contiguous()

    @property
    def shape(self):
        return self.values.shape

    @property
    def device(self):
        return self.values.device

    @property
    def pitch(self) -> int:
        """Bytes between two rows of values."""
        return self.values.stride(0)
