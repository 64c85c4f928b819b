"""Losses over the rows of an embedding table used as an output head.

``linear_cross_entropy`` and ``linear_distillation`` take hidden states [..., D] and a weight
[V, D] -- an ordinary table, or the rows of a TT table from ``full_weight()`` -- and return the
loss of the logits ``hidden @ weight.T`` without ever holding the [N, V] logits: the forward
keeps a running maximum and sum per position, the backward works through the vocabulary in
pieces.  Both are differentiable in hidden and weight (once, in reverse mode), for float32,
bfloat16 and float16, and return the loss in float32.

Argument marshalling only; the computation runs in libttbag (``tt_loss_forward`` and
``tt_loss_backward`` of ``include/tt_bag.h``).
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch
from torch.autograd import forward_ad

from . import abi

_REDUCTION = {"none": abi.TT_REDUCE_NONE, "mean": abi.TT_REDUCE_MEAN, "sum": abi.TT_REDUCE_SUM}


class _Plan:
    """The checked descriptor of one kind of call and the buffer sizes that go with it."""

    def __init__(self, hidden, weight, k, reduction, kw):
        self.desc = abi.make_loss_desc(hidden, weight, k=k, reduction=_REDUCTION[reduction], **kw)
        self.saved, self.fwd, self.bwd, self.only = abi.tt_loss_sizes(self.desc, weight)
        self.ref = ctypes.byref(self.desc)
        self.dtype = hidden.dtype
        self.n, self.d = hidden.shape
        self.v = weight.shape[0]


_plans = {}


def _bytes(n: int, device) -> torch.Tensor:
    return torch.empty(n, dtype=torch.uint8, device=device)


# What abi.tt_loss_forward and tt_loss_backward check of every buffer is known here by
# construction, so the two calls go to the library directly: a small loss is bound by the
# host, and the checks were a third of its calls.
def _forward(plan, hidden, weight, targets, teacher_logits, shape, dev_status, save):
    dev = hidden.device
    loss = torch.empty(shape, dtype=torch.float32, device=dev)
    saved = _bytes(plan.saved, dev) if save else None
    size = plan.fwd if save else plan.only
    ws = _bytes(size, dev)
    rc = abi.lib().tt_loss_forward(
        plan.ref, hidden.data_ptr(), weight.data_ptr(), targets.data_ptr(),
        None if teacher_logits is None else teacher_logits.data_ptr(), loss.data_ptr(),
        saved.data_ptr() if save else None, plan.saved, ws.data_ptr(), size,
        None if dev_status is None else dev_status.data_ptr(), abi._stream(None, hidden))
    if rc:
        raise abi.TTError("tt_loss_forward", rc)
    return loss, saved


def _backward(ctx, grad_loss):
    weight, saved = ctx.saved_tensors
    plan, dev = ctx.plan, weight.device
    grad_loss = grad_loss.contiguous()
    need_h, need_w = ctx.needs_input_grad[:2]
    dh = torch.empty((plan.n, plan.d), dtype=plan.dtype, device=dev) if need_h else None
    dw = torch.empty((plan.v, plan.d), dtype=plan.dtype, device=dev) if need_w else None
    ws = _bytes(plan.bwd, dev)
    rc = abi.lib().tt_loss_backward(
        plan.ref, saved.data_ptr(), weight.data_ptr(), saved.data_ptr(), plan.saved,
        grad_loss.data_ptr(), dh.data_ptr() if need_h else None,
        dw.data_ptr() if need_w else None, ws.data_ptr(), plan.bwd, abi._stream(None, weight))
    if rc:
        raise abi.TTError("tt_loss_backward", rc)
    return dh, dw, None, None, None, None, None


_backward_once = torch.autograd.function.once_differentiable(_backward)


class _LossFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, plan, targets, teacher_logits, shape, dev_status):
        loss, saved = _forward(plan, hidden, weight, targets, teacher_logits, shape, dev_status,
                               True)
        ctx.plan = plan
        # `saved` has the hidden rows that count, packed: the backward does not read hidden itself
        ctx.save_for_backward(weight, saved)
        return loss

    @staticmethod
    def backward(ctx, grad_loss):
        # gradients of gradients are refused; only create_graph=True runs with them enabled
        return (_backward_once if torch.is_grad_enabled() else _backward)(ctx, grad_loss)


_MAX_WEIGHT_STRIDE = 1 << 21  # the library's limit; hidden states may lie any distance apart


def _rows(t: torch.Tensor, far: bool) -> torch.Tensor:
    """[..., D] as [N, D] with contiguous rows (a view where the strides allow it)."""
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1])
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and (
            t.stride(0) < t.shape[1] or not far and t.stride(0) > _MAX_WEIGHT_STRIDE):
        t = t.contiguous()
    return t


def _loss(hidden, weight, targets, teacher_logits, shape, k, reduction, dev_status, **kw):
    if forward_ad._current_level >= 0:  # (unpack_dual by itself is 3 % of a small loss)
        for t in (hidden, weight):
            if forward_ad.unpack_dual(t).tangent is not None:
                raise NotImplementedError(
                    "the vocabulary-head losses have no forward-mode derivative")
    hidden, weight = _rows(hidden, True), _rows(weight, False)
    key = (hidden.shape, hidden.stride(), weight.shape, weight.stride(), hidden.dtype,
           weight.dtype, hidden.device, weight.device, k, reduction, *kw.values())
    plan = _plans.get(key)
    if plan is None:
        if reduction not in _REDUCTION:
            raise ValueError("reduction must be one of %s" % sorted(_REDUCTION))
        if len(_plans) > 1024:
            _plans.clear()
        plan = _plans[key] = _Plan(hidden, weight, k, reduction, kw)
    if targets.dtype != torch.int64:
        raise TypeError("indices must be int64 or int32, got %s" % targets.dtype)
    for t in (targets, teacher_logits, dev_status):
        if t is not None and t.device != hidden.device:
            raise ValueError("a buffer is on %s, hidden on %s" % (t.device, hidden.device))
    if dev_status is not None:
        abi._need(dev_status, torch.int32, "dev_status")
        abi._numel(dev_status, 1, "dev_status")
    if reduction != "none":
        shape = ()
    if torch.is_grad_enabled() and (hidden.requires_grad or weight.requires_grad):
        return _LossFunction.apply(hidden, weight, plan, targets, teacher_logits, shape,
                                   dev_status)
    return _forward(plan, hidden, weight, targets, teacher_logits, shape, dev_status, False)[0]


def linear_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, *,
                         ignore_index: int = -100, label_smoothing: float = 0.0,
                         reduction: str = "mean",
                         dev_status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Softmax cross entropy of the logits ``hidden @ weight.T`` against target rows.

    hidden [..., D], weight [V, D], targets [...] (integers in [0, V), or ignore_index for a
    position that does not count).  With e = label_smoothing and z the logits,
    ``loss_i = lse_i - (1 - e) z_i,t - (e / V) sum_v z_iv``.  reduction "none" returns [...]
    (0 at ignored positions), "sum" their sum, "mean" the sum over the positions that count (0
    if there are none).  A target outside [0, V) is treated as ignored and sets
    ``TT_DEV_BAD_INDEX`` in dev_status (an int32 GPU tensor of one element) if that is given."""
    if hidden.dim() < 1 or targets.shape != hidden.shape[:-1]:
        raise ValueError("targets must have the shape of hidden without its last dimension")
    if targets.dtype == torch.int32:
        targets = targets.to(torch.int64)
    if not 0.0 <= label_smoothing <= 1.0:
        raise ValueError("label_smoothing must be in [0, 1]")
    return _loss(hidden, weight, targets.contiguous(), None, targets.shape, 0, reduction,
                 dev_status, ignore_index=ignore_index, label_smoothing=label_smoothing)


def linear_distillation(hidden: torch.Tensor, weight: torch.Tensor, teacher_logits: torch.Tensor,
                        teacher_indices: torch.Tensor, *, temperature: float = 1.0,
                        reduction: str = "mean",
                        dev_status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """T^2 times the KL divergence of the student ``softmax(hidden @ weight.T / T)`` from a
    teacher given by its k top logits per position.

    hidden [..., D], weight [V, D], teacher_logits and teacher_indices [..., k]; the teacher's
    distribution is ``softmax(teacher_logits / T)`` over the entries with an index >= 0 and a
    logit above -inf (an index may repeat); a position without entries does not count.  The
    teacher gets no gradient.  reduction and dev_status as in ``linear_cross_entropy``."""
    if hidden.dim() < 1 or teacher_indices.dim() < 1 or \
            teacher_indices.shape[:-1] != hidden.shape[:-1]:
        raise ValueError("teacher_indices must have the shape of hidden with k in the place of "
                         "its last dimension")
    if teacher_logits.shape != teacher_indices.shape:
        raise ValueError("teacher_logits and teacher_indices must have the same shape")
    if teacher_logits.dtype not in abi._DTYPE:
        raise TypeError("teacher_logits must be float32, bfloat16 or float16, got %s"
                        % teacher_logits.dtype)
    k = teacher_indices.shape[-1]
    if k < 1:
        raise ValueError("at least one teacher entry per position is needed")
    if not 0.0 < ctypes.c_float(temperature).value < float("inf"):  # the library's type
        raise ValueError("temperature must be positive and finite in float32")
    if teacher_indices.dtype == torch.int32:
        teacher_indices = teacher_indices.to(torch.int64)
    return _loss(hidden, weight, teacher_indices.contiguous(),
                 teacher_logits.detach().contiguous(), teacher_indices.shape[:-1], k, reduction,
                 dev_status, temperature=temperature, teacher_dtype=teacher_logits.dtype)
