"""The embedding lookup with scaling and its gradient by sorted tokens:
marshalling of torch tensors to the C ABI of ``include/train_ops.h``.

Both run on the current torch stream of the tensors' device, allocate nothing
but their result and workspace through torch, and never wait for the GPU.
"""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd import forward_ad

from . import _lib
from ._lib import check

_TYPES = {torch.bfloat16: _lib.TRAIN_BF16, torch.float16: _lib.TRAIN_FP16,
          torch.float32: _lib.TRAIN_FP32}
_ID_TYPES = {torch.int32: _lib.TRAIN_INT32, torch.int64: _lib.TRAIN_INT64}

# The current device and stream, from torch's quick private calls (0.1 us each, where
# the public ones take 0.2 and 2.9) as long as it has them.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _code(name, t, codes, index):
    """Code of a tensor's type, after the checks that every argument gets."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor")
    code = codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected {', '.join(map(str, codes))}, got {t.dtype}")
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name}: on {t.device}, expected "
                         + (f"cuda:{index}" if index >= 0 else "a CUDA device"))
    return code


def _row_stride(name, t):
    """Elements from one row to the next of a tensor whose last dimension is
    dense and whose leading ones step evenly from row to row."""
    dim = t.shape[-1]
    if t.is_contiguous():
        return dim
    if dim > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    stride = None
    span = 1  # rows below the dimension looked at
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 0:
            return dim
        if n == 1:
            continue
        if stride is None:
            stride = st
        elif st != stride * span:
            raise ValueError(f"{name}: rows must step evenly through its leading dimensions")
        span *= n
    if stride is None:
        return dim
    if stride < dim:
        raise ValueError(f"{name}: rows overlap")
    return stride


def _fits(name, number):
    """Refuses a token number that the C ABI would take modulo 2^64."""
    if not -2 ** 63 <= number < 2 ** 63:
        raise ValueError(f"{name}: expected a number of 64 bits, got {number}")


def _refuse(name, t, ids):
    """Says what is wrong with a call's matrix ``t`` or its ids."""
    index = t.get_device() if isinstance(t, torch.Tensor) else -1
    _code(name, t, _TYPES, index)
    _code("ids", ids, _ID_TYPES, index)
    if not ids.is_contiguous():
        raise ValueError("ids: must be contiguous")
    raise TypeError(f"{name}: expected a tensor of two dimensions" if name == "table"
                    else f"{name}: expected a tensor of one dimension or more")


def _enqueue(index, call, *args):
    """``call(*args, stream)`` with device ``index`` current, on its current stream."""
    if index == _current_device():
        rc = call(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = call(*args, _raw_stream(index))
    if rc:
        check(rc)


def _no_tangent(name, *tensors):
    """Refuses arguments of an operator that carry a forward-mode tangent, within a level
    of forward mode."""
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise RuntimeError(f"{name}: there is no forward-mode derivative")


# Whether there may be tangents: without a level none has one.  A look at torch's own count
# takes 0.06 us, each tensor's tangent 0.9.
def _forward_mode():
    return getattr(forward_ad, "_current_level", 0) >= 0


# Counts a change of tensors that the caller gave and a call wrote to: a graph that saved
# one then refuses its backward pass, as behind torch's own operators in place.  (0.15 us
# through torch's private call, as long as it has it, 0.3 through the public one.)
_wrote = getattr(torch._C, "_increment_version", torch.autograd.graph.increment_version)


class _Embed(torch.autograd.Function):
    """The lookup of a table that requires grad."""

    @staticmethod
    def forward(ctx, table, ids, scale, first_row, out_dtype):
        ctx.save_for_backward(ids)
        ctx.scale, ctx.first_row = scale, first_row
        ctx.n_rows, ctx.dtype = table.shape[0], table.dtype
        return embed(table, ids, scale=scale, first_row=first_row, out_dtype=out_dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        ids, = ctx.saved_tensors
        try:
            _row_stride("grad_out", grad_out)
        except ValueError:  # one row for many, or rows that step unevenly
            grad_out = grad_out.contiguous()
        grad = embed_grad(grad_out, ids, n_rows=ctx.n_rows, scale=ctx.scale,
                          first_row=ctx.first_row, dtype=ctx.dtype)
        return grad, None, None, None, None


@functools.lru_cache(maxsize=256)
def _workspace_bytes(n_ids, n_rows, dim):
    need = ctypes.c_int64()
    check(_lib.load().train_embed_grad_workspace(n_ids, n_rows, dim, ctypes.byref(need)))
    return need.value


def embed(table: torch.Tensor, ids: torch.Tensor, *, scale: float = 1.0, first_row: int = 0,
          out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Rows of ``table`` that ``ids`` name, times ``scale``, rounded once.

    ``table`` is ``[n_rows, dim]`` in bfloat16, float16 or float32; ``ids`` has
    any shape, int32 or int64, and the result is ``ids.shape + (dim,)`` in
    ``out_dtype`` (default: the table's), or is written to ``out``.  The table
    may hold the slice of a vocabulary that starts at token ``first_row``: a
    token outside the slice gives a row of zeros.

    If the table requires grad, so does the result: its gradient is
    ``embed_grad`` into a new table of the same type.  It can be
    differentiated once, and ``out`` is refused then.  A table with a
    forward-mode tangent is refused.
    """
    try:
        t_code, i_code = _TYPES[table.dtype], _ID_TYPES[ids.dtype]
        rows, dim = table.shape
        index = table.get_device()
        fine = index >= 0 and ids.get_device() == index and ids.is_contiguous()
    except (AttributeError, KeyError, ValueError):
        fine = False
    if not fine:
        _refuse("table", table, ids)
    _fits("first_row", first_row)
    if _forward_mode():
        _no_tangent("embed", table)
    if table.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise RuntimeError("embed: out= cannot be given for a table that requires grad")
        return _Embed.apply(table, ids, scale, first_row, out_dtype)
    t_stride = dim if table.is_contiguous() else _row_stride("table", table)
    given = out
    if out is None:
        o_code = t_code if out_dtype is None else _TYPES.get(out_dtype)
        if o_code is None:
            raise TypeError(f"out_dtype: expected {', '.join(map(str, _TYPES))}")
        out = torch.empty((*ids.shape, dim), dtype=out_dtype or table.dtype, device=table.device)
        o_stride = dim
    else:
        o_code = _code("out", out, _TYPES, index)
        if out.shape != ids.shape + (dim,) or (out_dtype is not None and out.dtype != out_dtype):
            raise ValueError(f"out: expected shape {(*ids.shape, dim)} and out_dtype's type")
        o_stride = _row_stride("out", out)
    _enqueue(index, _lib.load().train_embed, table.data_ptr(), t_code, rows, dim, t_stride,
             ids.data_ptr(), i_code, ids.numel(), first_row, scale, out.data_ptr(), o_code,
             o_stride)
    if given is not None:
        _wrote((given,))
    return out


def embed_grad(grad_out: torch.Tensor, ids: torch.Tensor, *, n_rows: int | None = None,
               scale: float = 1.0, first_row: int = 0, padding_id: int = -1,
               accumulate: bool = False, out: torch.Tensor | None = None,
               dtype: torch.dtype | None = None) -> torch.Tensor:
    """Gradient of ``embed`` with respect to its table.

    ``grad_out`` is ``ids.shape + (dim,)``.  The result, ``[n_rows, dim]`` in
    ``dtype`` (default: ``grad_out``'s), or ``out``, is the sum of the rows of
    ``grad_out`` of each token times ``scale``: in fp32, in an order that only
    the ids fix, rounded once.  Rows without a token become zero, or with
    ``accumulate`` the sums are added to what ``out`` holds and those rows stay
    as they are.  Tokens outside the slice that starts at ``first_row``, and
    ``padding_id`` (negative: none), add nothing.  The result has no history.
    """
    try:
        g_code, i_code = _TYPES[grad_out.dtype], _ID_TYPES[ids.dtype]
        dim = grad_out.shape[-1]
        index = grad_out.get_device()
        fine = index >= 0 and ids.get_device() == index and ids.is_contiguous()
    except (AttributeError, KeyError, IndexError):
        fine = False
    if not fine:
        _refuse("grad_out", grad_out, ids)
    _fits("first_row", first_row)
    _fits("padding_id", padding_id)
    g_stride = dim if grad_out.is_contiguous() else _row_stride("grad_out", grad_out)
    if grad_out.shape[:-1] != ids.shape:
        raise ValueError("grad_out: expected ids.shape + (dim,)")
    given = out
    if out is None:
        if n_rows is None:
            raise ValueError("n_rows or out must be given")
        if accumulate:
            raise ValueError("accumulate needs out")
        o_code = g_code if dtype is None else _TYPES.get(dtype)
        if o_code is None:
            raise TypeError(f"dtype: expected {', '.join(map(str, _TYPES))}")
        out = torch.empty((n_rows, dim), dtype=dtype or grad_out.dtype, device=grad_out.device)
        o_stride = dim
    else:
        o_code = _code("out", out, _TYPES, index)
        if (out.dim() != 2 or out.shape[1] != dim or n_rows not in (None, out.shape[0])
                or (dtype is not None and out.dtype != dtype)):
            raise ValueError("out: expected [n_rows, dim] of dtype's type")
        o_stride = _row_stride("out", out)
    n_ids, rows = ids.numel(), out.shape[0]
    need = _workspace_bytes(n_ids, rows, dim)
    workspace = (torch.empty(need, dtype=torch.uint8, device=grad_out.device) if need
                 else None)
    _enqueue(index, _lib.load().train_embed_grad, grad_out.data_ptr(), g_code, g_stride,
             ids.data_ptr(), i_code, n_ids, first_row, padding_id, scale, 1 if accumulate else 0,
             out.data_ptr(), o_code, rows, dim, o_stride,
             workspace.data_ptr() if need else None, need)
    if given is not None:
        _wrote((given,))
    return out


__all__ = ["embed", "embed_grad"]
