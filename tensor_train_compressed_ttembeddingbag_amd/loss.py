"""Losses over the rows of an embedding table used as an output head.

``linear_cross_entropy`` and ``linear_distillation`` take hidden states [..., D] and a weight
[V, D] -- an ordinary table, or the rows of a TT table from ``full_weight()`` -- and return the
loss of the logits ``hidden @ weight.T`` without ever holding the [N, V] logits: the forward
keeps a running maximum and sum per position, the backward works through the vocabulary in
pieces.  Both are differentiable in hidden and weight (once), for float32, bfloat16 and
float16, and return the loss in float32.

Argument marshalling only; the computation runs in libttbag (``tt_loss_forward`` and
``tt_loss_backward`` of ``include/tt_bag.h``).
"""
from __future__ import annotations

from typing import Optional

import torch

from . import abi

_REDUCTION = {"none": abi.TT_REDUCE_NONE, "mean": abi.TT_REDUCE_MEAN, "sum": abi.TT_REDUCE_SUM}


class _LossFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, desc, targets, teacher_logits, dev_status):
        loss, saved = abi.tt_loss_forward(desc, hidden, weight, targets, teacher_logits,
                                          dev_status=dev_status)
        ctx.desc = desc
        ctx.save_for_backward(hidden, weight, saved)
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_loss):
        hidden, weight, saved = ctx.saved_tensors
        dh, dw = abi.tt_loss_backward(ctx.desc, hidden, weight, saved, grad_loss.contiguous(),
                                      need=ctx.needs_input_grad[:2])
        return dh, dw, None, None, None, None


def _rows(t: torch.Tensor) -> torch.Tensor:
    """[..., D] as [N, D] with contiguous rows (a view where the strides allow it)."""
    if t.dim() != 2:
        t = t.reshape(-1, t.shape[-1])
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        t = t.contiguous()
    return t


def _loss(hidden, weight, targets, teacher_logits, shape, k, reduction, dev_status, **kw):
    if reduction not in _REDUCTION:
        raise ValueError("reduction must be one of %s" % sorted(_REDUCTION))
    hidden, weight = _rows(hidden), _rows(weight)
    desc = abi.make_loss_desc(hidden, weight, k=k, reduction=_REDUCTION[reduction], **kw)
    if torch.is_grad_enabled() and (hidden.requires_grad or weight.requires_grad):
        loss = _LossFunction.apply(hidden, weight, desc, targets, teacher_logits, dev_status)
    else:
        loss = abi.tt_loss_forward(desc, hidden, weight, targets, teacher_logits,
                                   dev_status=dev_status)[0]
    return loss.view(shape if reduction == "none" else ())


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
    if not 0.0 < temperature < float("inf"):
        raise ValueError("temperature must be positive and finite")
    if teacher_indices.dtype == torch.int32:
        teacher_indices = teacher_indices.to(torch.int64)
    return _loss(hidden, weight, teacher_indices.contiguous(),
                 teacher_logits.detach().contiguous(), teacher_indices.shape[:-1], k, reduction,
                 dev_status, temperature=temperature, teacher_dtype=teacher_logits.dtype)
