"""The loss against a teacher's top logits and true labels, and its gradient:
marshalling of torch tensors to the C ABI of ``include/train_ops.h``.

Both run on the current torch stream of the tensors' device, allocate nothing
but their results through torch, and never wait for the GPU.
"""
from __future__ import annotations

import torch

from . import _lib
from .embedding import (_ID_TYPES, _TYPES, _code, _enqueue, _fits, _forward_mode, _no_tangent,
                        _row_stride, _wrote)
from .layernorm import _matrix, _new_like, _same_rows


def _arguments(logits, top_ids, top_logits, labels, temperature, soft_weight, hard_weight,
               ignore_id):
    """The first arguments of ``train_distill``, and the device."""
    code, rows, vocab, stride, index = _matrix("logits", logits)
    lead = logits.shape[:-1]
    i_ptr = t_ptr = l_ptr = None
    i_code = t_code = l_code = i_stride = t_stride = top_k = 0
    if top_ids is not None or top_logits is not None:
        i_code = _code("top_ids", top_ids, _ID_TYPES, index)
        t_code = _code("top_logits", top_logits, _TYPES, index)
        shape = top_ids.shape
        if shape[:-1] != lead or len(shape) != len(lead) + 1:
            raise ValueError("top_ids: expected logits.shape[:-1] + (top_k,)")
        if top_logits.shape != shape:
            raise ValueError("top_logits: expected the shape of top_ids")
        top_k = shape[-1]
        i_stride = top_k if top_ids.is_contiguous() else _row_stride("top_ids", top_ids)
        t_stride = top_k if top_logits.is_contiguous() else _row_stride("top_logits", top_logits)
        i_ptr, t_ptr = top_ids.data_ptr(), top_logits.data_ptr()
    if labels is not None:
        l_code = _code("labels", labels, _ID_TYPES, index)
        if labels.shape != lead or not labels.is_contiguous():
            raise ValueError("labels: expected logits.shape[:-1], contiguous")
        l_ptr = labels.data_ptr()
    _fits("ignore_id", ignore_id)
    return (logits.data_ptr(), code, stride, rows, vocab, i_ptr, i_code, i_stride, t_ptr, t_code,
            t_stride, top_k, l_ptr, l_code, ignore_id, temperature, soft_weight,
            hard_weight), index


class _Distill(torch.autograd.Function):
    """The loss of logits that require grad."""

    @staticmethod
    def forward(ctx, logits, top_ids, top_logits, labels, how):
        ctx.save_for_backward(logits, top_ids, top_logits, labels)
        ctx.how = how
        return distill_loss(logits, top_ids, top_logits, labels, **how)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        logits, top_ids, top_logits, labels = ctx.saved_tensors
        args, index = _arguments(logits, top_ids, top_logits, labels, **ctx.how)
        grad_out = grad_out.contiguous()
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        _enqueue(index, _lib.load().train_distill, *args, None, grad_out.data_ptr(), 1.0,
                 grad.data_ptr(), args[1], args[4])
        return grad, None, None, None, None


def distill_loss(logits: torch.Tensor, top_ids: torch.Tensor | None,
                 top_logits: torch.Tensor | None, labels: torch.Tensor | None = None, *,
                 temperature: float = 1.0, soft_weight: float = 1.0, hard_weight: float = 0.0,
                 ignore_id: int = -100) -> torch.Tensor:
    """Each row's loss against a teacher's top logits and a true label, float32 of
    ``logits.shape[:-1]``.

    ``logits`` are ``[..., vocab]`` in bfloat16, float16 or float32.  ``top_ids``
    (int32 or int64) and ``top_logits``, both ``[..., top_k]`` with ``top_k`` at most
    1024, are what the teacher holds most likely: with ``T`` the temperature, ``p``
    their softmax at ``T`` and ``q`` the softmax of ``logits`` at ``T``, the first
    term is ``soft_weight * T**2 * sum(p * (log p - log q[top_ids]))``.  An entry
    whose id lies outside the vocabulary or whose logit is -inf is left out; a token
    may be named twice.  Without a teacher (None) there is no such term.

    ``labels`` (int32 or int64, contiguous) add ``-hard_weight * log
    softmax(logits)[label]``.  A row whose label is ``ignore_id``, or lies outside
    the vocabulary, is left out: its loss and gradient are 0, whatever it holds.

    If ``logits`` require grad, so does the result; it can be differentiated once.
    The teacher gets no gradient, and arguments with a forward-mode tangent are refused.
    As with torch's own operators, a backward pass that is captured into a CUDA graph
    needs leaves that no eager result still alive depends on.
    """
    args, index = _arguments(logits, top_ids, top_logits, labels, temperature, soft_weight,
                             hard_weight, ignore_id)
    if _forward_mode():
        _no_tangent("distill_loss", logits, top_logits)
    if torch.is_grad_enabled():
        if top_logits is not None and top_logits.requires_grad:
            raise RuntimeError("distill_loss: the teacher's logits get no gradient; detach them")
        if logits.requires_grad:
            return _Distill.apply(logits, top_ids, top_logits, labels,
                                  dict(temperature=temperature, soft_weight=soft_weight,
                                       hard_weight=hard_weight, ignore_id=ignore_id))
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
    _enqueue(index, _lib.load().train_distill, *args, loss.data_ptr(), None, 1.0, None, 0, 0)
    return loss


def distill_loss_grad(logits: torch.Tensor, top_ids: torch.Tensor | None,
                      top_logits: torch.Tensor | None, labels: torch.Tensor | None = None, *,
                      temperature: float = 1.0, soft_weight: float = 1.0,
                      hard_weight: float = 0.0, ignore_id: int = -100,
                      row_grad: torch.Tensor | None = None, scale: float = 1.0,
                      out: torch.Tensor | None = None, dtype: torch.dtype | None = None):
    """``distill_loss`` and its gradient for the logits in one pass over them:
    ``(loss, grad)``.

    The gradient of row i's loss is multiplied by ``scale * row_grad[i]``: what the
    loss counts in the mean that is minimised, and the loss scale.  ``row_grad`` is
    float32 of ``logits.shape[:-1]``, contiguous (default: all 1); a row where it is
    0 gets a gradient of 0 whatever its logits hold.  ``grad`` has the shape of
    ``logits`` and is of type ``dtype`` (default: theirs), or is written to ``out``,
    which may be ``logits``.  The results have no history.
    """
    args, index = _arguments(logits, top_ids, top_logits, labels, temperature, soft_weight,
                             hard_weight, ignore_id)
    g_ptr = None
    if row_grad is not None:
        if (_code("row_grad", row_grad, _TYPES, index) != _lib.TRAIN_FP32
                or row_grad.shape != logits.shape[:-1] or not row_grad.is_contiguous()):
            raise ValueError("row_grad: expected float32 of logits.shape[:-1], contiguous")
        g_ptr = row_grad.data_ptr()
    given = out
    if out is None:
        o_code = args[1] if dtype is None else _TYPES.get(dtype)
        if o_code is None:
            raise TypeError(f"dtype: expected {', '.join(map(str, _TYPES))}")
        out = _new_like(logits, dtype)
        o_stride = args[4]
    else:
        o_code, o_stride = _same_rows("out", out, logits.shape, index)
        if dtype is not None and out.dtype != dtype:
            raise ValueError(f"out: expected {dtype}")
    loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
    _enqueue(index, _lib.load().train_distill, *args, loss.data_ptr(), g_ptr, scale,
             out.data_ptr(), o_code, o_stride)
    if given is not None:
        _wrote((given,))
    return loss, out


__all__ = ["distill_loss", "distill_loss_grad"]
