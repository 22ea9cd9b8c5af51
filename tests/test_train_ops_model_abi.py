"""Host-side tests of layer norm's and the distillation loss's entry points: bad
arguments are refused before anything touches a GPU."""
import ctypes
import math

import pytest
import torch

import optimizer_step_gb300 as og
from optimizer_step_gb300 import _lib

INVALID, ALIGN, OK = _lib.LAMB_ERR_INVALID, _lib.LAMB_ERR_ALIGN, _lib.LAMB_OK
P = 4096  # an address that the checks accept and nothing reads


def norm_args(**change):
    a = dict(x=P, x_dtype=0, x_stride=8, n_rows=2, dim=8, weight=P, bias=P, param_dtype=0,
             eps=1e-5, y=P, y_dtype=0, y_stride=8, stats=P, stream=None)
    assert set(change) <= set(a)
    return list({**a, **change}.values())


@pytest.mark.parametrize("change,code", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x_dtype=3), INVALID),
    (dict(y_dtype=-1), INVALID), (dict(param_dtype=3), INVALID), (dict(n_rows=-1), INVALID),
    (dict(n_rows=1 << 31), INVALID), (dict(dim=-1), INVALID), (dict(dim=0), INVALID),
    (dict(dim=1 << 31, x_stride=1 << 31, y_stride=1 << 31), INVALID), (dict(x_stride=7), INVALID),
    (dict(y_stride=7), INVALID), (dict(eps=-1e-9), INVALID), (dict(eps=math.inf), INVALID),
    (dict(eps=math.nan), INVALID), (dict(x=P + 1), ALIGN), (dict(y=P + 1), ALIGN),
    (dict(x=P + 2, x_dtype=2), ALIGN), (dict(weight=P + 1), ALIGN), (dict(bias=P + 1), ALIGN),
    (dict(bias=P + 2, param_dtype=2), ALIGN), (dict(stats=P + 2), ALIGN),
])
def test_layer_norm_refuses(change, code):
    lib = og.load()
    assert lib.train_layer_norm(*norm_args(**change)) == code
    assert lib.lamb_last_error()


def test_layer_norm_of_no_rows_is_done():
    assert og.load().train_layer_norm(*norm_args(n_rows=0, x=None, y=None)) == OK


def grad_args(**change):
    a = dict(grad_out=P, grad_out_dtype=0, grad_out_stride=8, x=P, x_dtype=0, x_stride=8, n_rows=2,
             dim=8, weight=P, weight_dtype=0, stats=P, x_grad=P, x_grad_stride=8, weight_grad=P,
             bias_grad=P, param_grad_dtype=0, accumulate=0, workspace=P, workspace_bytes=1 << 40,
             stream=None)
    assert set(change) <= set(a)
    return list({**a, **change}.values())


@pytest.mark.parametrize("change,code", [
    (dict(grad_out=None), INVALID), (dict(x=None), INVALID), (dict(stats=None), INVALID),
    (dict(grad_out_dtype=3), INVALID), (dict(x_dtype=3), INVALID), (dict(weight_dtype=-1), INVALID),
    (dict(param_grad_dtype=3), INVALID), (dict(accumulate=2), INVALID), (dict(n_rows=-1), INVALID),
    (dict(dim=0), INVALID), (dict(grad_out_stride=7), INVALID), (dict(x_stride=7), INVALID),
    (dict(x_grad_stride=7), INVALID), (dict(n_rows=1 << 20, workspace=None), INVALID),
    (dict(n_rows=1 << 20, workspace_bytes=-1), INVALID),
    (dict(n_rows=1 << 20, workspace_bytes=0), INVALID),
    (dict(n_rows=1 << 30, dim=1 << 20, grad_out_stride=1 << 20, x_stride=1 << 20,
          x_grad_stride=1 << 20, workspace_bytes=1 << 62), INVALID),
    (dict(grad_out=P + 1), ALIGN), (dict(x=P + 1), ALIGN), (dict(x_grad=P + 1), ALIGN),
    (dict(weight=P + 1), ALIGN), (dict(weight_grad=P + 1), ALIGN), (dict(bias_grad=P + 1), ALIGN),
    (dict(stats=P + 2), ALIGN), (dict(n_rows=1 << 20, workspace=P + 8), ALIGN),
    (dict(weight_grad=P + 2, param_grad_dtype=2), ALIGN),
])
def test_layer_norm_grad_refuses(change, code):
    lib = og.load()
    assert lib.train_layer_norm_grad(*grad_args(**change)) == code
    assert lib.lamb_last_error()


def test_layer_norm_grad_with_nothing_to_do():
    lib = og.load()
    assert lib.train_layer_norm_grad(*grad_args(x_grad=None, weight_grad=None, bias_grad=None,
                                                workspace=None, workspace_bytes=0)) == OK
    assert lib.train_layer_norm_grad(*grad_args(n_rows=0, accumulate=1, stats=None)) == OK


def test_layer_norm_grad_workspace():
    lib, need = og.load(), ctypes.c_int64()
    call = lib.train_layer_norm_grad_workspace
    assert call(1000, 64, None) == INVALID
    for bad in ((-1, 8), (8, -1), (8, 0), (1 << 31, 8), (8, 1 << 31), (1 << 30, 1 << 20)):
        assert call(*bad, ctypes.byref(need)) == INVALID
    for n, dim in ((0, 8), (1, 1), (8192, 4096), (2 ** 31 - 1, 512), (1, 2 ** 31 - 1)):
        assert call(n, dim, ctypes.byref(need)) == OK and need.value >= 0
        if need.value:
            sizes = dict(n_rows=n, dim=dim, grad_out_stride=dim, x_stride=dim, x_grad_stride=dim)
            assert lib.train_layer_norm_grad(
                *grad_args(workspace_bytes=need.value - 1, **sizes)) == INVALID


def distill_args(**change):
    a = dict(logits=P, logits_dtype=0, logits_stride=8, n_rows=2, vocab=8, top_ids=P,
             top_ids_dtype=1, top_ids_stride=3, top_logits=P, top_logits_dtype=0,
             top_logits_stride=3, top_k=3, labels=P, labels_dtype=1, ignore_id=-100,
             temperature=1.0, soft_weight=1.0, hard_weight=1.0, loss=P, row_grad=P, scale=1.0,
             grad=P, grad_dtype=0, grad_stride=8, stream=None)
    assert set(change) <= set(a)
    return list({**a, **change}.values())


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), INVALID), (dict(logits_dtype=3), INVALID), (dict(grad_dtype=3), INVALID),
    (dict(logits_stride=7), INVALID), (dict(grad_stride=7), INVALID), (dict(n_rows=-1), INVALID),
    (dict(n_rows=1 << 31), INVALID), (dict(vocab=0), INVALID), (dict(vocab=-1), INVALID),
    (dict(vocab=1 << 31, logits_stride=1 << 31, grad_stride=1 << 31), INVALID),
    (dict(top_k=-1), INVALID),
    (dict(top_k=1025, top_ids_stride=1025, top_logits_stride=1025), INVALID),
    (dict(top_ids=None), INVALID), (dict(top_logits=None), INVALID),
    (dict(top_ids_dtype=2), INVALID), (dict(top_logits_dtype=3), INVALID),
    (dict(top_ids_stride=2), INVALID), (dict(top_logits_stride=2), INVALID),
    (dict(labels=None), INVALID), (dict(labels_dtype=-1), INVALID),
    (dict(temperature=0.0), INVALID), (dict(temperature=-2.0), INVALID),
    (dict(temperature=math.inf), INVALID), (dict(temperature=math.nan), INVALID),
    (dict(temperature=1e-40), INVALID), (dict(soft_weight=math.inf), INVALID),
    (dict(hard_weight=math.nan), INVALID),
    (dict(logits=P + 1), ALIGN), (dict(grad=P + 1), ALIGN), (dict(top_ids=P + 4), ALIGN),
    (dict(top_logits=P + 1), ALIGN), (dict(labels=P + 4), ALIGN), (dict(loss=P + 2), ALIGN),
    (dict(row_grad=P + 2), ALIGN),
])
def test_distill_refuses(change, code):
    lib = og.load()
    assert lib.train_distill(*distill_args(**change)) == code
    assert lib.lamb_last_error()


def test_distill_with_nothing_to_do():
    lib = og.load()
    assert lib.train_distill(*distill_args(loss=None, grad=None)) == OK
    assert lib.train_distill(*distill_args(n_rows=0, logits=None, grad=None, top_ids=None,
                                           top_logits=None, labels=P)) == OK


def test_python_refuses_tensors_that_are_not_on_a_gpu():
    x = torch.zeros(3, 8)
    with pytest.raises(ValueError):
        og.layer_norm(x)
    with pytest.raises(ValueError):
        og.layer_norm_grad(x, x, None, torch.zeros(2, 3))
    with pytest.raises(ValueError):
        og.distill_loss(x, torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2))
    with pytest.raises(ValueError):
        og.distill_loss_grad(x, torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2))
    for call in (og.layer_norm, lambda v: og.distill_loss(v, None, None)):
        with pytest.raises(TypeError):
            call(None)
