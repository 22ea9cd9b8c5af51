"""Global gradient norm over many tensors, and clipping: marshalling of torch
tensors to the ``train_clip_*`` calls of ``include/train_ops.h``."""
from __future__ import annotations

import ctypes
from typing import Sequence

import numpy as np
import torch

from . import _lib
from ._lib import check
from .embedding import _TYPES


def _arrays(name, tensors, device):
    """Sizes, type codes and addresses of tensors, after their checks."""
    rows = []
    for i, t in enumerate(tensors):
        code = _TYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
        if code is None:
            raise TypeError(f"{name}[{i}]: expected a bfloat16, float16 or float32 tensor")
        if t.device != device:
            raise ValueError(f"{name}[{i}]: on {t.device}, expected {device}")
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}]: must be contiguous")
        rows.append((t.numel(), code, t.data_ptr()))
    table = np.array(rows, dtype=np.uint64).reshape(len(rows), 3).T
    return table[0].astype(np.int64), table[1].astype(np.int32), table[2].copy()


class GradClip:
    """The global norm of a fixed list of grads, and clipping by it.

    ``grads``: contiguous CUDA tensors on one device, bfloat16, float16 and
    float32 in any mix and of any size.  ``out`` (default: the grads
    themselves): tensors of the same sizes that receive the clipped grads,
    each of any of the three types.  No two tensors may overlap, but an output
    may be its own grad: a grad that is shared is listed once.  ``stream`` defaults to the current torch
    stream at construction; every call runs on it and returns without waiting.

    ``poison``: what ``clip`` and ``finish`` leave in the outputs when a grad is
    inf or NaN.  False: what they held.  True: NaN in every output.  A step that
    reads outputs in other tensors needs True, unless the program looks at
    ``stats`` first: ``Lamb`` skips when it finds inf or NaN in its grads, and
    would else apply the clipped grads of the step before again.  So do steps on
    grads clipped in place over several ranks without the split step.

    The calls return ``stats``, a float32 CUDA tensor that the next call
    overwrites: the norm of ``g / loss_scale`` (inf if a grad is inf or NaN),
    the factor that the grads are multiplied by (0 then), and 1.0 if a grad is
    inf or NaN, else 0.0.
    """

    def __init__(self, grads: Sequence[torch.Tensor],
                 out: Sequence[torch.Tensor] | None = None, stream=None, *,
                 poison: bool = False):
        self._lib = _lib.load()
        self._h = None
        grads = list(grads)
        for i, t in enumerate(grads[:1]):
            if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
                raise ValueError("grads must live on a CUDA device")
        self.device = grads[0].device if grads else torch.device("cuda",
                                                                 torch.cuda.current_device())
        n = len(grads)
        sizes, types, ptrs = _arrays("grads", grads, self.device)
        out_types = out_ptrs = None
        if out is not None:
            out = list(out)
            if len(out) != n:
                raise ValueError(f"out: expected {n} tensors, got {len(out)}")
            out_sizes, out_types, out_ptrs = _arrays("out", out, self.device)
            for i in np.flatnonzero(out_sizes != sizes):
                raise ValueError(f"out[{i}]: expected {sizes[i]} elements")
        self._keep = (grads, out)
        address = lambda a: None if a is None else a.ctypes.data
        with torch.cuda.device(self.device):
            self.stream = stream if stream is not None else torch.cuda.current_stream()
            with torch.cuda.stream(self.stream):
                self.stats = torch.zeros(3, dtype=torch.float32, device=self.device)
            h = ctypes.c_void_p()
            check(self._lib.train_clip_create(
                ctypes.byref(h), n, address(sizes), address(types), address(ptrs),
                address(out_ptrs), address(out_types),
                ctypes.c_void_p(self.stream.cuda_stream)))
        self._h = h
        check(self._lib.train_clip_set_poison(h, 1 if poison else 0))
        self._stats_ptr = self.stats.data_ptr()

    def _handle(self):
        if self._h is None:
            raise RuntimeError("handle is closed")
        return self._h

    def norm(self, loss_scale: float = 1.0) -> torch.Tensor:
        """The norm alone; the factor in ``stats`` is ``1 / loss_scale``."""
        check(self._lib.train_clip_norm(self._handle(), loss_scale, self._stats_ptr))
        return self.stats

    def clip(self, max_norm: float, loss_scale: float = 1.0) -> torch.Tensor:
        """Divides the grads by ``loss_scale`` and clips their global norm to
        ``max_norm`` (<= 0: no clipping), rounding once.  If a grad is inf or
        NaN the outputs stay as they are, or all become NaN (``poison``).

        A step that reads the outputs takes ``loss_scale=1``.  While ``Lamb``'s
        dynamic loss scaler is on, its steps divide by their own scale S in any
        case: then call ``clip(max_norm * S)`` with ``S = opt.next_loss_scale``
        as of the backward pass, which leaves S in the outputs (and in the norm)
        for the step to take off."""
        check(self._lib.train_clip_grads(self._handle(), max_norm, loss_scale, self._stats_ptr))
        return self.stats

    def _exchange(self, exchange):
        if (not isinstance(exchange, torch.Tensor) or exchange.dtype != torch.float64
                or exchange.device != self.device or exchange.numel() != 2
                or not exchange.is_contiguous()):
            raise ValueError(f"exchange: need a contiguous float64 tensor of 2 elements on "
                             f"{self.device}")
        return exchange.data_ptr()

    def partial(self, exchange: torch.Tensor) -> torch.Tensor:
        """This rank's ``{sum of g^2, 1 if a grad is inf or NaN}`` into
        ``exchange``, to be summed over the ranks before ``finish``."""
        check(self._lib.train_clip_partial(self._handle(), self._exchange(exchange)))
        return exchange

    def finish(self, exchange: torch.Tensor, max_norm: float,
               loss_scale: float = 1.0) -> torch.Tensor:
        """``clip`` by the norm that the summed ``exchange`` gives."""
        check(self._lib.train_clip_finish(self._handle(), self._exchange(exchange), max_norm,
                                          loss_scale, self._stats_ptr))
        return self.stats

    def close(self) -> None:
        if self._h is not None:
            h, self._h = self._h, None
            check(self._lib.train_clip_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()


__all__ = ["GradClip"]
