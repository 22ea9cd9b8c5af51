"""Layer norm and its backward pass: marshalling of torch tensors to the C ABI
of ``include/train_ops.h``.

Both run on the current torch stream of the tensors' device, allocate nothing
but their results and workspace through torch, and never wait for the GPU.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import check
from .embedding import (_TYPES, _code, _enqueue, _forward_mode, _no_tangent, _row_stride,
                        _wrote)


def _vector(name, t, dim, index):
    """Code and address of a vector of ``dim`` elements."""
    try:
        if (t.get_device() == index and t.numel() == dim and t.dim() == 1
                and t.is_contiguous()):
            return _TYPES[t.dtype], t.data_ptr()
    except (AttributeError, KeyError):
        pass
    _code(name, t, _TYPES, index)
    raise ValueError(f"{name}: expected {dim} consecutive elements")


def _matrix(name, t):
    """Code, rows, width, row stride and device of a tensor's rows."""
    try:
        code, dim, index = _TYPES[t.dtype], t.shape[-1], t.get_device()
        if dim > 0 and index >= 0:
            return (code, t.numel() // dim, dim,
                    dim if t.is_contiguous() else _row_stride(name, t), index)
    except (AttributeError, KeyError, IndexError):
        pass
    if not isinstance(t, torch.Tensor) or t.dim() == 0:
        raise TypeError(f"{name}: expected a tensor of one dimension or more")
    _code(name, t, _TYPES, t.get_device())
    raise ValueError(f"{name}: rows have no elements")


def _same_rows(name, t, shape, index):
    """Code and row stride of another tensor with these rows."""
    try:
        if t.get_device() == index and t.shape == shape:
            return _TYPES[t.dtype], shape[-1] if t.is_contiguous() else _row_stride(name, t)
    except (AttributeError, KeyError):
        pass
    _code(name, t, _TYPES, index)
    raise ValueError(f"{name}: expected shape {tuple(shape)}")


def _new_like(x, dtype):
    """An empty tensor of x's shape, rows one behind the other."""
    if dtype is None:
        dtype = x.dtype
    if x.is_contiguous():
        return torch.empty_like(x) if dtype is x.dtype else torch.empty_like(x, dtype=dtype)
    return torch.empty(x.shape, dtype=dtype, device=x.device)


class _LayerNorm(torch.autograd.Function):
    """Layer norm of a tensor, weight or bias that requires grad."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, out_dtype):
        y, stats = layer_norm(x, weight, bias, eps=eps, stats=True, out_dtype=out_dtype)
        ctx.save_for_backward(x, weight, stats)
        ctx.bias_type = None if bias is None else bias.dtype
        ctx.mark_non_differentiable(stats)
        ctx.set_materialize_grads(False)
        return y, stats

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out, _):
        if grad_out is None:
            return None, None, None, None, None
        x, weight, stats = ctx.saved_tensors
        try:
            _row_stride("grad_out", grad_out)
        except ValueError:  # one row for many, or rows that step unevenly
            grad_out = grad_out.contiguous()
        need = ctx.needs_input_grad
        grads = layer_norm_grad(grad_out, x, weight, stats, x_grad=need[0], weight_grad=need[1],
                                bias_grad=need[2], param_dtype=ctx.bias_type)
        return (*grads, None, None)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(n_rows, dim):
    need = ctypes.c_int64()
    check(_lib.load().train_layer_norm_grad_workspace(n_rows, dim, ctypes.byref(need)))
    return need.value


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, *, eps: float = 1e-5, stats: bool = False,
               out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None):
    """``(x - mean) / sqrt(var + eps) * weight + bias`` over the last dimension,
    rounded once.

    ``x`` is ``[..., dim]`` in bfloat16, float16 or float32; ``weight`` and
    ``bias``, ``[dim]`` and of one type if both are given, are 1 and 0 if not.
    The result has ``x``'s shape and is of ``out_dtype`` (default: ``x``'s), or
    is written to ``out``, which may be ``x``.  With ``stats`` the result is
    ``(y, stats)``: float32 ``[2, ...]`` with each row's mean and ``1 / sqrt(var +
    eps)``, which ``layer_norm_grad`` takes.

    If ``x``, ``weight`` or ``bias`` requires grad, so does the result.  It can be
    differentiated once, and ``out`` is refused then.  ``stats`` have no gradient, and
    arguments with a forward-mode tangent are refused.  As with torch's own operators, a
    backward pass that is captured into a CUDA graph needs leaves that no eager result
    still alive depends on.
    """
    code, rows, dim, stride, index = _matrix("x", x)
    w_ptr = b_ptr = None
    p_code = 0
    if weight is not None:
        p_code, w_ptr = _vector("weight", weight, dim, index)
    if bias is not None:
        b_code, b_ptr = _vector("bias", bias, dim, index)
        if weight is not None and b_code != p_code:
            raise TypeError(f"bias: expected {weight.dtype}, the weight's type, got {bias.dtype}")
        p_code = b_code
    if _forward_mode():
        _no_tangent("layer_norm", x, weight, bias)
    if torch.is_grad_enabled() and (x.requires_grad
                                    or (weight is not None and weight.requires_grad)
                                    or (bias is not None and bias.requires_grad)):
        if out is not None:
            raise RuntimeError("layer_norm: out= cannot be given where a gradient is required")
        y, kept = _LayerNorm.apply(x, weight, bias, eps, out_dtype)
        return (y, kept) if stats else y
    given = out
    if out is None:
        o_code = code if out_dtype is None else _TYPES.get(out_dtype)
        if o_code is None:
            raise TypeError(f"out_dtype: expected {', '.join(map(str, _TYPES))}")
        out = _new_like(x, out_dtype)
        o_stride = dim
    else:
        o_code, o_stride = _same_rows("out", out, x.shape, index)
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out: expected {out_dtype}")
    kept = None
    if stats:
        shape = x.shape
        kept = torch.empty((2, rows) if len(shape) == 2 else (2, *shape[:-1]),
                           dtype=torch.float32, device=x.device)
    _enqueue(index, _lib.load().train_layer_norm, x.data_ptr(), code, stride, rows, dim, w_ptr,
             b_ptr, p_code, eps, out.data_ptr(), o_code, o_stride,
             kept.data_ptr() if stats else None)
    if given is not None:
        _wrote((given,))
    return (out, kept) if stats else out


def _param_grad(name, want, dim, dtype, device, index, accumulate):
    """The tensor for a parameter's gradient that an argument asks for, or None."""
    if want is None or want is False:
        return None
    if want is True:
        if accumulate:
            raise ValueError(f"{name}: accumulate needs the tensor to add to")
        return torch.empty(dim, dtype=dtype, device=device)
    _vector(name, want, dim, index)
    return want


def layer_norm_grad(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor | None,
                    stats: torch.Tensor, *, x_grad: torch.Tensor | bool = True,
                    weight_grad: torch.Tensor | bool = True,
                    bias_grad: torch.Tensor | bool = True, accumulate: bool = False,
                    param_dtype: torch.dtype | None = None):
    """Gradients of ``layer_norm``: ``(x_grad, weight_grad, bias_grad)``.

    ``grad_out`` is the gradient of the result, of its shape; ``x``, ``weight`` and
    ``stats`` are the forward pass's.  Each gradient is asked for with True, left
    out with False (None is returned in its place) or given as the tensor to write
    to.  ``x_grad`` is of ``x``'s type and may be ``grad_out`` or ``x``.  The other
    two are ``[dim]``, both of ``param_dtype`` (default: the weight's type, or
    float32 without one), summed over all rows in fp32 in a fixed order and rounded
    once; with ``accumulate`` they are tensors, and the sums are added to what they
    hold.  The results have no history.
    """
    x_code, rows, dim, x_stride, index = _matrix("x", x)
    g_code, g_stride = _same_rows("grad_out", grad_out, x.shape, index)
    if (_code("stats", stats, _TYPES, index) != _lib.TRAIN_FP32 or not stats.is_contiguous()
            or stats.shape[:1] != (2,) or stats.shape[1:] != x.shape[:-1]):
        raise ValueError(f"stats: expected float32 of shape {(2, *x.shape[:-1])}")
    w_code, w_ptr = (0, None) if weight is None else _vector("weight", weight, dim, index)
    device = x.device
    given = ()
    if x_grad is True:
        dx = _new_like(x, None)
        dx_stride = dim
    elif x_grad is None or x_grad is False:
        dx, dx_stride = None, dim
    else:
        dx = x_grad
        given = (dx,)
        d_code, dx_stride = _same_rows("x_grad", dx, x.shape, index)
        if d_code != x_code:
            raise TypeError(f"x_grad: expected {x.dtype}, the type of x")
    dtype = param_dtype or next(
        (t.dtype for t in (weight_grad, bias_grad, weight) if isinstance(t, torch.Tensor)),
        torch.float32)
    p_code = _TYPES.get(dtype)
    if p_code is None:
        raise TypeError(f"param_dtype: expected {', '.join(map(str, _TYPES))}")
    dw = _param_grad("weight_grad", weight_grad, dim, dtype, device, index, accumulate)
    db = _param_grad("bias_grad", bias_grad, dim, dtype, device, index, accumulate)
    for name, t in (("weight_grad", dw), ("bias_grad", db)):
        if t is not None and t.dtype != dtype:
            raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if dw is not None and dw is weight_grad:
        given += (dw,)
    if db is not None and db is bias_grad:
        given += (db,)
    need = _workspace_bytes(rows, dim) if dw is not None or db is not None else 0
    workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _enqueue(index, _lib.load().train_layer_norm_grad, grad_out.data_ptr(), g_code, g_stride,
             x.data_ptr(), x_code, x_stride, rows, dim, w_ptr, w_code, stats.data_ptr(),
             None if dx is None else dx.data_ptr(), dx_stride,
             None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr(),
             p_code, 1 if accumulate else 0, workspace.data_ptr() if need else None, need)
    if given:
        _wrote(given)
    return dx, dw, db


__all__ = ["layer_norm", "layer_norm_grad"]
