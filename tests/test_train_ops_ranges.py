"""Sizes and token numbers that no call can hold are refused before anything is
enqueued.  Nothing here reaches a GPU: the addresses are never read."""
import pytest

import optimizer_step_gb300 as og
from optimizer_step_gb300 import _lib
from test_train_ops_abi import INVALID, embed_args, grad_args

LAST = 2 ** 63 - 1


@pytest.mark.parametrize("first_row,n_rows", [(LAST, 2), (LAST - 2, 4), (LAST, 2 ** 31 - 1)])
def test_rows_behind_the_last_token_number_are_refused(first_row, n_rows):
    """Their numbers would be those of negative ids."""
    lib = og.load()
    assert lib.train_embed(*embed_args(first_row=first_row, n_rows=n_rows)) == INVALID
    assert lib.train_embed_grad(*grad_args(first_row=first_row, n_rows=n_rows)) == INVALID


def test_a_slice_may_end_at_the_last_token_number():
    lib = og.load()
    assert lib.train_embed(*embed_args(first_row=LAST - 3, n_rows=4, n_ids=0)) == _lib.LAMB_OK
    assert lib.train_embed(*embed_args(first_row=LAST, n_rows=0, n_ids=0)) == _lib.LAMB_OK
    assert lib.train_embed_grad(*grad_args(first_row=LAST - 3, n_rows=4, n_ids=0,
                                           accumulate=1)) == _lib.LAMB_OK


@pytest.mark.parametrize("n_ids,n_rows,dim", [
    (2 ** 31 - 1, 100, 2 ** 20),         # more blocks of sums than a launch has CTAs
    (2 ** 31 - 1, 100, 2 ** 31 - 1),
    (100, 2 ** 31 - 1, 2 ** 20),         # more zero rows than are counted
    (5000, 2 ** 31 - 1, 2 ** 31 - 1),
])
def test_a_gradient_beyond_any_memory_is_refused_before_anything_is_enqueued(n_ids, n_rows, dim):
    lib = og.load()
    sizes = dict(n_ids=n_ids, n_rows=n_rows, dim=dim, grad_out_stride=dim, grad_stride=dim,
                 workspace_bytes=2 ** 62)
    for accumulate in (0, 1):
        rc = lib.train_embed_grad(*grad_args(accumulate=accumulate, **sizes))
        assert rc == INVALID and "too large" in lib.lamb_last_error().decode()
