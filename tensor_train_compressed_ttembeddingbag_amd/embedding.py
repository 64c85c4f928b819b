"""Rows of a dense table times a scale, and the table's gradient by sorted tokens.

``embedding`` looks rows of a weight [V, D] up -- an ordinary table in float32, bfloat16 or
float16, or an ``Int8Rows`` table -- and is differentiable in a float weight (once, in reverse
mode); ``embedding_gradient`` is that gradient by itself, for training steps without autograd.
With the table as the head of the losses in ``loss`` it is the other end of a tied model.

Argument marshalling only; the computation runs in libttbag (``tt_embed_forward`` and
``tt_embed_backward`` of ``include/tt_bag.h``).
"""
from __future__ import annotations

import ctypes
import math
import operator
from typing import Optional

import torch

from . import abi
from .quant import Int8Rows

_descs = {}
_MAX_STRIDE = 1 << 32  # elements between rows: the library's limit


def _desc(n, v, d, weight_stride, grad_stride, padding_idx, dtype, out_dtype, scale):
    """The descriptor of a kind of call, its reference and the backward's workspace size."""
    key = (n, v, d, weight_stride, grad_stride, padding_idx, dtype, out_dtype, scale)
    got = _descs.get(key)
    if got is None:
        if not math.isfinite(ctypes.c_float(scale).value):  # the library's type
            raise ValueError("scale must be finite in float32")
        desc = abi.TTEmbedDesc(n, v, d, weight_stride, grad_stride, padding_idx, dtype, out_dtype,
                               scale)
        ref = ctypes.byref(desc)
        size = 0 if dtype == abi.TT_DTYPE_I8 else abi.lib().tt_embed_workspace_size(ref)
        if len(_descs) > 4096:
            _descs.clear()
        got = _descs[key] = (desc, ref, size)
    return got


def _padding(padding_idx: Optional[int], v: int) -> int:
    if padding_idx is None:
        return -1
    padding_idx = operator.index(padding_idx)
    if not -v <= padding_idx < v:
        raise ValueError("padding_idx must be within the table's %d rows" % v)
    return padding_idx % v


def _indices(indices: torch.Tensor, device, dev_status) -> torch.Tensor:
    if not isinstance(indices, torch.Tensor):
        raise TypeError("indices must be a torch.Tensor")
    if indices.dtype == torch.int32:
        indices = indices.to(torch.int64)
    if indices.dtype != torch.int64:
        raise TypeError("indices must be int64 or int32, got %s" % indices.dtype)
    if indices.device != device:
        raise ValueError("indices is on %s, not on %s" % (indices.device, device))
    if dev_status is not None:
        abi._need(dev_status, torch.int32, "dev_status")
        abi._numel(dev_status, 1, "dev_status")
        if dev_status.device != device:
            raise ValueError("dev_status is on %s, not on %s" % (dev_status.device, device))
    return indices.contiguous()


def _forward(indices, weight, scale, padding_idx, dtype, dev_status):
    int8 = isinstance(weight, Int8Rows)
    values = weight.values if int8 else weight
    (v, d), n = values.shape, indices.numel()
    stride = values.stride(0) if v > 1 else (d + 15) // 16 * 16 if int8 else d
    desc, ref, _ = _desc(n, v, d, stride, d, padding_idx,
                         abi.TT_DTYPE_I8 if int8 else abi._DTYPE[values.dtype],
                         abi._DTYPE[dtype], scale)
    out = values.new_empty(indices.shape + (d,), dtype=dtype)
    abi._launch("tt_embed_forward", values, ref, indices.data_ptr(), values.data_ptr(),
                weight.scales.data_ptr() if int8 else None, out.data_ptr(), abi._ptr(dev_status))
    return out


def _gradient(grad_out, indices, v, d, scale, padding_idx, dtype, dev_status):
    n = indices.numel()
    g = grad_out if grad_out.dim() == 2 else grad_out.reshape(n, d)
    if d > 1 and g.stride(1) != 1 or n > 1 and not d <= g.stride(0) <= _MAX_STRIDE:
        g = g.contiguous()
    _, ref, size = _desc(n, v, d, d, g.stride(0) if n > 1 else d, padding_idx, abi._DTYPE[dtype],
                         abi._DTYPE[g.dtype], scale)
    if not size:
        raise abi.TTError("tt_embed_workspace_size", -2)
    dw = g.new_empty((v, d), dtype=dtype)
    # (256 bytes stand for none)
    ws = g.new_empty(size, dtype=torch.uint8) if size > 256 else None
    abi._launch("tt_embed_backward", g, ref, indices.data_ptr(), g.data_ptr(), dw.data_ptr(),
                abi._ptr(ws), size, abi._ptr(dev_status))
    return dw


def _backward(ctx, grad_out):
    indices, = ctx.saved_tensors
    v, d, scale, padding_idx, dtype, dev_status = ctx.call
    dw = _gradient(grad_out, indices, v, d, scale, padding_idx, dtype, dev_status)
    return None, dw, None, None, None, None


_backward_once = torch.autograd.function.once_differentiable(_backward)


class _EmbeddingFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, indices, weight, scale, padding_idx, dtype, dev_status):
        ctx.call = (*weight.shape, scale, padding_idx, weight.dtype, dev_status)
        ctx.save_for_backward(indices)
        return _forward(indices, weight, scale, padding_idx, dtype, dev_status)

    @staticmethod
    def backward(ctx, grad_out):
        # gradients of gradients are refused; only create_graph=True runs with them enabled
        return (_backward_once if torch.is_grad_enabled() else _backward)(ctx, grad_out)


def embedding(indices: torch.Tensor, weight, *, scale: float = 1.0,
              padding_idx: Optional[int] = None, dtype: Optional[torch.dtype] = None,
              dev_status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``scale * weight[indices]`` as [..., D], from indices [...] (int64 or int32).

    weight [V, D] is a float32, bfloat16 or float16 tensor or an ``Int8Rows``; the rows come in
    dtype (the weight's own; float32 from ``Int8Rows``).  The row padding_idx is looked up like the
    others but gets no gradient.  An index outside [0, V) gives a row of zeros, has no gradient and
    sets ``TT_DEV_BAD_INDEX`` in dev_status (an int32 GPU tensor of one element) if that is
    given.  The gradient is dense, of the weight's dtype, summed in float32 in a fixed order.
    scale is a constant (a tensor of one element is read at the call)."""
    int8 = isinstance(weight, Int8Rows)
    if not int8 and not isinstance(weight, torch.Tensor):
        raise TypeError("weight must be a torch.Tensor or an Int8Rows")
    traced = torch._C._is_tracing()
    if int8 or not traced:
        abi._no_trace("embedding")
    if not int8:
        abi._no_dual("embedding", weight)
        if weight.dtype not in abi._DTYPE:
            raise TypeError("weight must be float32, bfloat16, float16 or an Int8Rows, got %s"
                            % weight.dtype)
        if weight.dim() != 2 or weight.numel() == 0:
            raise ValueError("weight must have two dimensions and a row")
        if not weight.is_cuda:
            raise ValueError("weight must be on the GPU")
    if dtype is None:
        dtype = torch.float32 if int8 else weight.dtype
    elif dtype not in abi._DTYPE:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % dtype)
    scale = abi._number(scale, "scale")
    indices = _indices(indices, weight.device, dev_status)
    padding_idx = _padding(padding_idx, weight.shape[0])
    if not int8 and (weight.shape[1] > 1 and weight.stride(1) != 1
                     or weight.shape[0] > 1
                     and not weight.shape[1] <= weight.stride(0) <= _MAX_STRIDE):
        weight = weight.contiguous()
    # (torch.jit.trace records an autograd function as what it is)
    if traced or not int8 and weight.requires_grad and torch.is_grad_enabled():
        return _EmbeddingFunction.apply(indices, weight, scale, padding_idx, dtype, dev_status)
    return _forward(indices, weight, scale, padding_idx, dtype, dev_status)


def embedding_gradient(grad_out: torch.Tensor, indices: torch.Tensor, num_rows: int, *,
                       scale: float = 1.0, padding_idx: Optional[int] = None,
                       dtype: Optional[torch.dtype] = None,
                       dev_status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient [num_rows, D] of the weight of ``embedding(indices, weight, ...)`` from
    grad_out [..., D], in dtype (grad_out's own if not given).  It has no gradient of its own: a
    grad_out that requires one is refused while gradients are enabled."""
    if not isinstance(grad_out, torch.Tensor):
        raise TypeError("grad_out must be a torch.Tensor")
    abi._no_trace("embedding_gradient")
    abi._no_dual("embedding_gradient", grad_out)
    if grad_out.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("embedding_gradient has no gradient: detach grad_out or call it under "
                           "torch.no_grad()")
    if grad_out.dtype not in abi._DTYPE:
        raise TypeError("grad_out must be float32, bfloat16 or float16, got %s" % grad_out.dtype)
    if dtype is None:
        dtype = grad_out.dtype
    elif dtype not in abi._DTYPE:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % dtype)
    if not grad_out.is_cuda:
        raise ValueError("grad_out must be on the GPU")
    indices = _indices(indices, grad_out.device, dev_status)
    if grad_out.dim() < 1 or grad_out.shape[:-1] != indices.shape or grad_out.shape[-1] < 1:
        raise ValueError("grad_out must have the shape of indices and a last dimension")
    num_rows, scale = operator.index(num_rows), abi._number(scale, "scale")
    if num_rows < 1:
        raise ValueError("num_rows must be positive")
    return _gradient(grad_out, indices, num_rows, grad_out.shape[-1], scale,
                     _padding(padding_idx, num_rows), dtype, dev_status)
