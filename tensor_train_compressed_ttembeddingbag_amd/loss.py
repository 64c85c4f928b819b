"""Losses over the rows of an embedding table used as an output head.

``linear_cross_entropy``, ``linear_distillation``, ``linear_preference`` and ``linear_policy`` take
hidden states [..., D] and a weight [V, D] -- an ordinary table, or the rows of a TT table from
``full_weight()`` -- and return the loss of the logits ``hidden @ weight.T`` without ever holding
the [N, V] logits: the forward keeps a running maximum and sum per position, the backward works
through the vocabulary in pieces, with the gradient of a piece's logits in 16 bits (float32: two
fp16 parts).  All are differentiable in hidden and weight (once, in reverse mode), for float32,
bfloat16 and float16, and return the loss in float32.

Argument marshalling only; the computation runs in libttbag (``tt_loss_*``, ``tt_prefer_*`` and
``tt_policy_*`` of ``include/tt_bag.h``).
"""
from __future__ import annotations

import ctypes
import operator
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
    abi._no_proxies("tt_loss_backward")
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
    abi._no_trace("a vocabulary-head loss")  # (its autograd function too: it is given a plan for these sizes)
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
    ignore_index = int(ignore_index)
    label_smoothing = abi._number(label_smoothing, "label_smoothing")
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
    temperature = abi._number(temperature, "temperature")
    if not 0.0 < ctypes.c_float(temperature).value < float("inf"):  # the library's type
        raise ValueError("temperature must be positive and finite in float32")
    if teacher_indices.dtype == torch.int32:
        teacher_indices = teacher_indices.to(torch.int64)
    return _loss(hidden, weight, teacher_indices.contiguous(),
                 teacher_logits.detach().contiguous(), teacher_indices.shape[:-1], k, reduction,
                 dev_status, temperature=temperature, teacher_dtype=teacher_logits.dtype)


# ---------------------------------------------------------------- preference and policy losses
_KIND = {"sigmoid": abi.TT_PREFER_SIGMOID, "hinge": abi.TT_PREFER_HINGE,
         "square": abi.TT_PREFER_SQUARE}


class _LogpPlan:
    """The descriptor of one kind of preference or policy loss, its entry points and sizes."""

    def __init__(self, name, desc, hidden, weight):
        lib = abi.lib()
        self.desc, self.ref = desc, ctypes.byref(desc)
        self.forward, self.backward = "tt_%s_forward" % name, "tt_%s_backward" % name
        size = getattr(lib, "tt_%s_workspace_size" % name)
        self.saved = getattr(lib, "tt_%s_saved_size" % name)(self.ref)
        if not self.saved:
            raise abi.TTError("tt_%s_saved_size" % name, -2)
        self.fwd = size(self.ref, abi.TT_LOSS_FORWARD)
        self.bwd = size(self.ref, abi.TT_LOSS_BACKWARD)
        self.only = size(self.ref, abi.TT_LOSS_ONLY)
        (self.n, self.d), self.v = hidden.shape, weight.shape[0]


def _logp_forward(plan, hidden, weight, inputs, shape, more_shape, dev_status, save):
    """(loss, the second output or None, saved or None)"""
    new = hidden.new_empty
    loss = new(shape, dtype=torch.float32)
    more = None if more_shape is None else new(more_shape, dtype=torch.float32)
    saved = new(plan.saved, dtype=torch.uint8) if save else None
    size = plan.fwd if save else plan.only
    ws = new(size, dtype=torch.uint8)
    abi._launch(plan.forward, hidden, plan.ref, hidden.data_ptr(), weight.data_ptr(),
                *[abi._ptr(t) for t in inputs], loss.data_ptr(), abi._ptr(more), abi._ptr(saved),
                plan.saved, ws.data_ptr(), size, abi._ptr(dev_status))
    return loss, more, saved


def _logp_backward(ctx, grad_loss, _):
    weight, saved = ctx.saved_tensors
    plan, new = ctx.plan, weight.new_empty
    if grad_loss is None:
        return (None,) * 7
    grad_loss = grad_loss.contiguous()
    need_h, need_w = ctx.needs_input_grad[:2]
    dh = new((plan.n, plan.d)) if need_h else None
    dw = new((plan.v, plan.d)) if need_w else None
    ws = new(plan.bwd, dtype=torch.uint8)
    abi._launch(plan.backward, weight, plan.ref, weight.data_ptr(), saved.data_ptr(), plan.saved,
                grad_loss.data_ptr(), abi._ptr(dh), abi._ptr(dw), ws.data_ptr(), plan.bwd)
    return dh, dw, None, None, None, None, None


_logp_backward_once = torch.autograd.function.once_differentiable(_logp_backward)


class _LogpFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, plan, inputs, shape, more_shape, dev_status):
        loss, more, saved = _logp_forward(plan, hidden, weight, inputs, shape, more_shape,
                                          dev_status, True)
        ctx.plan = plan
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(weight, saved)
        if more is not None:
            ctx.mark_non_differentiable(more)
        return loss, more

    @staticmethod
    def backward(ctx, grad_loss, _):
        # gradients of gradients are refused; only create_graph=True runs with them enabled
        return (_logp_backward_once if torch.is_grad_enabled() else _logp_backward)(
            ctx, grad_loss, None)


def _logp_loss(name, hidden, weight, inputs, shape, more_shape, reduction, dev_status, make, key):
    """key: what make(desc of the product) depends on beside hidden and weight."""
    what = "linear_%s" % ("preference" if name == "prefer" else name)
    abi._no_trace(what)  # (as the losses above)
    abi._no_dual(what, hidden, weight)
    hidden, weight = _rows(hidden, True), _rows(weight, False)
    key = (name, hidden.shape, hidden.stride(), weight.shape, weight.stride(), hidden.dtype,
           weight.dtype, hidden.device, weight.device, reduction, *key)
    plan = _plans.get(key)
    if plan is None:
        if reduction not in _REDUCTION:
            raise ValueError("reduction must be one of %s" % sorted(_REDUCTION))
        if len(_plans) > 1024:
            _plans.clear()
        head = abi.make_loss_desc(hidden, weight)  # checks the two
        plan = _plans[key] = _LogpPlan(name, make(head, _REDUCTION[reduction]), hidden, weight)
    for t in (*inputs, dev_status):
        if t is not None and t.device != hidden.device:
            raise ValueError("a buffer is on %s, hidden on %s" % (t.device, hidden.device))
    if dev_status is not None:
        abi._need(dev_status, torch.int32, "dev_status")
        abi._numel(dev_status, 1, "dev_status")
    if reduction != "none":
        shape = ()
    if torch.is_grad_enabled() and (hidden.requires_grad or weight.requires_grad):
        return _LogpFunction.apply(hidden, weight, plan, inputs, shape, more_shape, dev_status)
    return _logp_forward(plan, hidden, weight, inputs, shape, more_shape, dev_status, False)[:2]


def _integers(t: torch.Tensor, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype == torch.int32:
        t = t.to(torch.int64)
    if t.dtype != torch.int64:
        raise TypeError("%s must be int64 or int32, got %s" % (name, t.dtype))
    return t.contiguous()


def _constant(t, shape, name: str, broadcast: bool = False):
    """A constant per position, float32 and contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in abi._DTYPE:
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, t.dtype))
    if t.shape != shape:
        if not broadcast:
            raise ValueError("%s must have the shape of hidden without its last dimension" % name)
        try:
            t = t.broadcast_to(shape)
        except RuntimeError:
            raise ValueError("%s does not broadcast to the shape of hidden without its last "
                             "dimension" % name) from None
    if t.dtype == torch.float32 and not t.requires_grad and t.is_contiguous():
        return t
    return t.detach().float().contiguous()


def linear_preference(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                      offsets: torch.Tensor, reference_logps: Optional[torch.Tensor] = None, *,
                      beta: float = 0.1, kind: str = "sigmoid", label_smoothing: float = 0.0,
                      margin: float = 0.0, average: bool = False, ignore_index: int = -100,
                      reduction: str = "mean", return_ratios: bool = False,
                      dev_status: Optional[torch.Tensor] = None):
    """A preference loss over P pairs of sequences, from their tokens' log-probabilities under the
    logits ``hidden @ weight.T``.

    hidden [..., D], weight [V, D], targets [...] (as in ``linear_cross_entropy``: ignore_index for
    positions that do not count, a prompt's for instance), offsets [2 P + 1]: sequence j has the
    positions offsets[j] .. offsets[j + 1] - 1 of the flattened ones; sequences 0 .. P - 1 are
    preferred to P .. 2 P - 1, and positions behind the last one do not count.  reference_logps
    [...]: the tokens' log-probabilities under the reference, for instance
    ``-linear_cross_entropy(..., reduction="none")`` of its hidden states; None: no reference.

    With h_j the sum (average: the mean) of logp - reference_logp over the sequence and
    ``x_p = h_p - h_(P + p)``, ``y = beta x - margin``, e = label_smoothing:

    * "sigmoid": ``-(1 - e) log sigmoid(y) - e log sigmoid(-y)``
    * "hinge": ``max(0, 1 - y)``
    * "square": ``(x - 1 / (2 beta))^2`` (no margin)

    reduction "none" returns [P], "sum" their sum, "mean" their mean (0 if there are none).
    return_ratios: also h as [2, P], without gradient.  Offsets that do not start at 0, fall or
    pass the positions set ``TT_DEV_BAD_OFFSETS`` in dev_status, and the result is unspecified."""
    if hidden.dim() < 1 or targets.shape != hidden.shape[:-1]:
        raise ValueError("targets must have the shape of hidden without its last dimension")
    targets, offsets = _integers(targets, "targets"), _integers(offsets, "offsets")
    if offsets.dim() != 1 or offsets.numel() % 2 != 1:
        raise ValueError("offsets must have 2 P + 1 entries")
    if kind not in _KIND:
        raise ValueError("kind must be one of %s" % sorted(_KIND))
    ignore_index, beta = operator.index(ignore_index), abi._number(beta, "beta")
    label_smoothing = abi._number(label_smoothing, "label_smoothing")
    margin = abi._number(margin, "margin")
    if not 0.0 < beta < float("inf"):
        raise ValueError("beta must be positive and finite")
    if not 0.0 <= label_smoothing <= 1.0 or label_smoothing and kind != "sigmoid":
        raise ValueError("label_smoothing must be in [0, 1], and is for kind \"sigmoid\"")
    if not -float("inf") < margin < float("inf") or margin and kind == "square":
        raise ValueError("margin must be finite, and is not for kind \"square\"")
    if reference_logps is not None:
        reference_logps = _constant(reference_logps, targets.shape, "reference_logps")
    pairs = offsets.numel() // 2

    def make(h, r):
        return abi.TTPreferDesc(h.n, h.v, h.d, h.hidden_stride, h.weight_stride, ignore_index,
                                pairs, beta, label_smoothing, margin, h.dtype, r, _KIND[kind],
                                bool(average))

    loss, ratios = _logp_loss("prefer", hidden, weight, (targets, offsets, reference_logps),
                              (pairs,), (2, pairs) if return_ratios else None, reduction,
                              dev_status, make, (pairs, beta, label_smoothing, margin, kind,
                                                 bool(average), ignore_index))
    return (loss, ratios) if return_ratios else loss


def linear_policy(hidden: torch.Tensor, weight: torch.Tensor, actions: torch.Tensor,
                  advantages: torch.Tensor, old_logps: Optional[torch.Tensor] = None,
                  reference_logps: Optional[torch.Tensor] = None, *, clip_low: float = 0.2,
                  clip_high: float = 0.2, kl_coef: float = 0.0, temperature: float = 1.0,
                  ignore_index: int = -100, reduction: str = "mean", return_logps: bool = False,
                  dev_status: Optional[torch.Tensor] = None):
    """The clipped policy loss with a KL term, of actions under the logits
    ``hidden @ weight.T / temperature``.

    hidden [..., D], weight [V, D], actions [...] (integers in [0, V), or ignore_index for a
    position that does not count), advantages (broadcast to [...]), old_logps [...]: the actions'
    log-probabilities under the policy that took them (None: this one), reference_logps [...]:
    those under the reference (needed with kl_coef).  With logp the actions' log-probabilities,
    ``r = exp(logp - old_logp)`` and ``d = reference_logp - logp``:

    ``loss_i = -min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A) + kl_coef (exp(d) - d - 1)``

    reduction "none" returns [...] (0 where a position does not count), "sum" their sum, "mean"
    the sum over the positions that count.  return_logps: also logp [...], without gradient (0
    where a position does not count): the old_logps of the next steps.  Advantages and the given
    log-probabilities are constants.  dev_status as in ``linear_cross_entropy``."""
    if hidden.dim() < 1 or actions.shape != hidden.shape[:-1]:
        raise ValueError("actions must have the shape of hidden without its last dimension")
    actions = _integers(actions, "actions")
    ignore_index = operator.index(ignore_index)
    clip_low, clip_high = abi._number(clip_low, "clip_low"), abi._number(clip_high, "clip_high")
    kl_coef = abi._number(kl_coef, "kl_coef")
    temperature = abi._number(temperature, "temperature")
    if not clip_low >= 0.0 or not clip_high >= 0.0:
        raise ValueError("clip_low and clip_high must not be negative")
    if not 0.0 <= kl_coef < float("inf"):
        raise ValueError("kl_coef must be finite and not negative")
    if not 0.0 < ctypes.c_float(temperature).value < float("inf"):  # the library's type
        raise ValueError("temperature must be positive and finite in float32")
    if kl_coef and reference_logps is None:
        raise ValueError("kl_coef needs reference_logps")
    advantages = _constant(advantages, actions.shape, "advantages", True)
    if old_logps is not None:
        old_logps = _constant(old_logps, actions.shape, "old_logps")
    if reference_logps is not None:
        reference_logps = _constant(reference_logps, actions.shape, "reference_logps")

    def make(h, r):
        return abi.TTPolicyDesc(h.n, h.v, h.d, h.hidden_stride, h.weight_stride, ignore_index,
                                clip_low, clip_high, kl_coef, h.dtype, r, temperature)

    loss, logps = _logp_loss("policy", hidden, weight,
                             (actions, advantages, old_logps, reference_logps), actions.shape,
                             actions.shape if return_logps else None, reduction, dev_status, make,
                             (clip_low, clip_high, kl_coef, temperature, ignore_index))
    return (loss, logps) if return_logps else loss
