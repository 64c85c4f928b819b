"""Tables in 8-bit integers: a scale for every row.

``Int8Rows`` holds a table as int8 values [R, D] and one float32 scale a row; the row it stands
for is ``values[r] * scales[r]``.  ``quantize_rows`` makes one of a float table, ``embedding`` looks
its rows up, and ``int8_linear`` multiplies hidden states, which get a scale for each token, with it:
the logits of a table used as an output head, at the matrix cores' rate for 8-bit integers and a
half or a fourth of the table's bytes.

Argument marshalling only; the computation runs in libttbag (``tt_int8_quantize`` and
``tt_int8_linear`` of ``include/tt_bag.h``).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import abi


class Int8Rows:
    """int8 values [R, D] and float32 scales [R] on the GPU.

    The rows of values have unit stride inside and lie a multiple of 16 bytes apart, from a
    multiple of 16 on; the memory of each reaches to the next multiple of 16 behind D (what is there
    does not matter).  Values laid out otherwise are copied."""

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
        whole = (d + 15) // 16 * 16
        end = values.storage_offset() + (rows - 1) * stride + whole
        if (stride % 16 or stride < whole or values.data_ptr() % 16
                or d > 1 and values.stride(1) != 1 or end > values.untyped_storage().nbytes()):
            copy = torch.zeros(rows, whole, dtype=torch.int8, device=values.device)
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


def _float_rows(t: torch.Tensor, name: str) -> torch.Tensor:
    """[..., D] as [N, D] with rows that are contiguous and do not overlap."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in abi._DTYPE:
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, t.dtype))
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError("%s must have a last dimension" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    abi._no_dual(name, t)
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1])
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        t = t.contiguous()
    return t


def quantize_rows(x: torch.Tensor) -> Int8Rows:
    """x [R, D] (float32, bfloat16 or float16) in 8 bits, a scale for each row:
    ``scales = amax(|x|, 1) / 127``, ``values = round(x / scales)``.

    A row with a value that is not finite gets the scale NaN; one whose scale would be below the
    normal numbers becomes zeros.  x gets no gradient."""
    abi._no_trace("quantize_rows")
    if isinstance(x, torch.Tensor) and (x.dim() != 2 or x.shape[0] < 1):
        raise ValueError("x must have two dimensions and a row")
    x = _float_rows(x, "x")
    n, d = x.shape
    pitch = (d + 15) // 16 * 16
    values = torch.empty((n, pitch), dtype=torch.int8, device=x.device)
    scales = torch.empty(n, dtype=torch.float32, device=x.device)
    abi._launch("tt_int8_quantize", x, n, d, abi._DTYPE[x.dtype], x.data_ptr(),
                x.stride(0) if n > 1 else d, values.data_ptr(), pitch, scales.data_ptr())
    return Int8Rows(values[:, :d], scales)


_plans = {}


def int8_linear(hidden, weight: Int8Rows, *, dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """``hidden @ weight.T`` as [..., V], both in 8-bit integers: hidden [..., D] is quantised with a
    scale for each token as by ``quantize_rows`` (or is an ``Int8Rows``), the products are summed
    exactly and scaled; D is at most 2^17, and less than that where hidden is an ``Int8Rows``.  In dtype: hidden's own, float32 from an ``Int8Rows``.

    There is no gradient: a hidden that requires one is refused while gradients are enabled."""
    abi._no_trace("int8_linear")
    if not isinstance(weight, Int8Rows):
        raise TypeError("weight must be an Int8Rows")
    given = isinstance(hidden, Int8Rows)
    if given:
        rows, shape, source = hidden.values, hidden.shape[:1], torch.int8
    else:
        rows = _float_rows(hidden, "hidden")
        if hidden.requires_grad and torch.is_grad_enabled():
            raise RuntimeError("int8_linear has no gradient: detach hidden or call it under "
                               "torch.no_grad()")
        shape, source = hidden.shape[:-1], rows.dtype
    (n, d), v = rows.shape, weight.shape[0]
    if dtype is None:
        dtype = torch.float32 if given else source
    elif dtype not in abi._DTYPE:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % dtype)
    if d != weight.shape[1]:
        raise ValueError("hidden has rows of %d, weight of %d" % (d, weight.shape[1]))
    if rows.device != weight.device:
        raise ValueError("hidden is on %s, weight on %s" % (rows.device, weight.device))
    stride = rows.stride(0) if given or n > 1 else d
    key = (n, v, d, stride, weight.pitch, source, dtype)
    plan = _plans.get(key)
    if plan is None:
        desc = abi.TTInt8Desc(n, v, d, stride, weight.pitch,
                              abi.TT_DTYPE_I8 if given else abi._DTYPE[source], abi._DTYPE[dtype])
        ref = ctypes.byref(desc)
        size = abi.lib().tt_int8_workspace_size(ref)
        if not size:
            raise abi.TTError("tt_int8_workspace_size", -2)
        if len(_plans) > 4096:
            _plans.clear()
        plan = _plans[key] = (desc, ref, size)
    _, ref, size = plan
    out = rows.new_empty(shape + (v,), dtype=dtype)
    # (256 bytes stand for none)
    ws = rows.new_empty(size, dtype=torch.uint8) if size > 256 else None
    abi._launch("tt_int8_linear", rows, ref, rows.data_ptr(),
                hidden.scales.data_ptr() if given else None, weight.values.data_ptr(),
                weight.scales.data_ptr(), out.data_ptr(), abi._ptr(ws), size)
    return out
