"""Tensors of a clip that overlap are refused when the handle is made: a grad that
is listed twice would count twice, and two CTAs would scale it at once.  The
addresses are never read."""
import ctypes

import numpy as np
import pytest

import optimizer_step_gb300 as og
from optimizer_step_gb300 import _lib

P = 1 << 20
BF16, FP32 = _lib.TRAIN_BF16, _lib.TRAIN_FP32


def create(grads, outs=None):
    """(code, message); each tensor is (address, elements, type)."""
    lib, h = og.load(), ctypes.c_void_p()
    n = len(grads)
    sizes = np.array([g[1] for g in grads], np.int64)
    types = np.array([g[2] for g in grads], np.int32)
    out_types = None if outs is None else np.array([o[1] for o in outs], np.int32)
    at = lambda tensors: (ctypes.c_void_p * n)(*[t[0] for t in tensors])
    rc = lib.train_clip_create(ctypes.byref(h), n, sizes.ctypes.data, types.ctypes.data, at(grads),
                               None if outs is None else at(outs),
                               None if outs is None else out_types.ctypes.data, None)
    message = lib.lamb_last_error().decode()
    if h.value:
        lib.train_clip_destroy(h)
    return rc, message


OVERLAPPING = {
    "listed twice": ([(P, 100, FP32), (P, 100, FP32)], None),
    "listed twice, among others": ([(P + 400 * i, 100, FP32) for i in range(50)] + [(P, 1, FP32)],
                                   None),
    "last element": ([(P, 100, FP32), (P + 396, 100, FP32)], None),
    "in the middle of a long one": ([(P, 100_000, BF16), (P + 300, 1, BF16), (P + 302, 5, BF16)],
                                    None),
    "same memory, two types": ([(P, 100, FP32), (P, 100, BF16)], None),
    "an output of two": ([(P, 8, FP32), (2 * P, 8, FP32)], [(3 * P, BF16), (3 * P, BF16)]),
    "outputs that meet": ([(P, 8, FP32), (2 * P, 8, FP32)], [(3 * P, FP32), (3 * P + 16, BF16)]),
    "another's grad as output": ([(P, 8, FP32), (2 * P, 8, FP32)], [(2 * P, FP32), (P, FP32)]),
    "an output in another's grad": ([(P, 8, FP32), (2 * P, 800, FP32)],
                                    [(2 * P + 1600, BF16), (4 * P, BF16)]),
    "an output behind its own start": ([(P, 8, FP32)], [(P + 4, FP32)]),
    "an output in front of its own start": ([(P, 8, BF16)], [(P - 16, FP32)]),
    "a long output": ([(P, 8, BF16), (P + 16, 8, BF16)], [(2 * P, FP32), (2 * P + 16, FP32)]),
    "a list without outputs of its own but one": ([(P, 8, FP32), (2 * P, 8, FP32)],
                                                  [(P, FP32), (P + 16, BF16)]),
}


@pytest.mark.parametrize("case", OVERLAPPING)
def test_overlapping_tensors_are_refused(case):
    for flip in (False, True):
        grads, outs = OVERLAPPING[case]
        if flip:
            grads, outs = grads[::-1], outs and outs[::-1]
        rc, message = create(grads, outs)
        assert rc == _lib.LAMB_ERR_INVALID and "overlap" in message
        assert "grads[" in message or "outs[" in message


@pytest.mark.parametrize("grads,outs", [
    ([(P, 100, FP32), (P + 400, 100, FP32)], None),
    ([(P, 100, FP32), (P, 0, FP32), (P + 200, 0, BF16), (P + 400, 1, BF16)], None),
    ([(P, 8, FP32), (2 * P, 8, FP32)], [(P, FP32), (2 * P, FP32)]),
    ([(P, 8, FP32), (P + 32, 8, FP32)], [(P, FP32), (P + 64, BF16)]),
    ([(P, 8, FP32), (P + 48, 8, FP32)], [(P + 32, BF16), (P + 80, BF16)]),
])
def test_neighbours_and_tensors_in_place_are_not(grads, outs):
    """Without a GPU the call fails behind the checks."""
    rc, message = create(grads, outs)
    assert rc != _lib.LAMB_ERR_INVALID and "overlap" not in message
