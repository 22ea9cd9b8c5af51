"""Results that lie partly over what their call still reads, or over one another, are
refused before anything touches a GPU.  The addresses are never read."""
import pytest

import optimizer_step_gb300 as og
from optimizer_step_gb300 import _lib

BF16, FP16, FP32 = _lib.TRAIN_BF16, _lib.TRAIN_FP16, _lib.TRAIN_FP32
A, B, C, D, E, F, G = (k << 24 for k in range(1, 8))   # far apart


def refuses(call, args):
    lib = og.load()
    assert getattr(lib, call)(*args) == _lib.LAMB_ERR_INVALID
    return b"overlap" in lib.lamb_last_error()


def norm(**change):
    a = dict(x=A, x_dtype=BF16, x_stride=100, n_rows=50, dim=64, weight=B, bias=C,
             param_dtype=BF16, eps=1e-5, y=D, y_dtype=BF16, y_stride=100, stats=E, stream=None)
    assert set(change) <= set(a)
    return list({**a, **change}.values())


@pytest.mark.parametrize("change", [
    dict(y=A + 2), dict(y=A - 2), dict(y=A + 200), dict(y=A - 49 * 200), dict(y=A + 63 * 2),
    dict(y=A, y_stride=101), dict(y=A, y_dtype=FP16), dict(y=A, y_dtype=FP32),
    dict(y=A, y_dtype=FP32, y_stride=64), dict(y=A + 49 * 200 + 63 * 2),
    dict(y=A - 49 * 200 - 63 * 2), dict(y=A, x_stride=64, y_stride=128),
    dict(y=A + 126, n_rows=1), dict(y=A, y_dtype=FP32, n_rows=1),
    dict(y=B), dict(y=C - 126), dict(y=B - 30 * 200), dict(y=E), dict(y=E + 396),
    dict(stats=A), dict(stats=A + 49 * 200), dict(stats=B), dict(stats=C + 124),
    dict(x=2 << 40, y=(2 << 40) + (1 << 33), x_stride=1 << 32, y_stride=1 << 32,
         n_rows=(1 << 31) - 1),
])
def test_layer_norm_refuses(change):
    assert refuses("train_layer_norm", norm(**change))


def grad(**change):
    a = dict(grad_out=A, grad_out_dtype=BF16, grad_out_stride=100, x=B, x_dtype=BF16, x_stride=100,
             n_rows=5000, dim=64, weight=C, weight_dtype=FP32, stats=D, x_grad=E,
             x_grad_stride=100, weight_grad=F, bias_grad=F + 256, param_grad_dtype=FP32,
             accumulate=0, workspace=G, workspace_bytes=1 << 22, stream=None)
    assert set(change) <= set(a)
    return list({**a, **change}.values())


@pytest.mark.parametrize("change", [
    dict(x_grad=A + 2), dict(x_grad=B + 200), dict(x_grad=A, x_grad_stride=64),
    dict(x_grad=A, grad_out_dtype=FP32), dict(x_grad=B + 4000 * 200, x_grad_stride=200),
    dict(x_grad=C), dict(x_grad=D - 4000 * 200), dict(x_grad=F), dict(x_grad=F + 384),
    dict(x_grad=G), dict(bias_grad=F), dict(bias_grad=F + 252), dict(bias_grad=F - 252),
    dict(workspace=A), dict(workspace=B + 16 * 1000), dict(workspace=C), dict(workspace=D),
    dict(workspace=E), dict(workspace=F), dict(bias_grad=F, n_rows=5),
    dict(bias_grad=F, x_grad=None),
])
def test_layer_norm_grad_refuses(change):
    assert refuses("train_layer_norm_grad", grad(**change))


def distill(**change):
    a = dict(logits=A, logits_dtype=FP32, logits_stride=100, n_rows=50, vocab=64, top_ids=B,
             top_ids_dtype=1, top_ids_stride=3, top_logits=C, top_logits_dtype=BF16,
             top_logits_stride=3, top_k=3, labels=D, labels_dtype=1, ignore_id=-100,
             temperature=1.0, soft_weight=1.0, hard_weight=1.0, loss=E, row_grad=F, scale=1.0,
             grad=G, grad_dtype=FP32, grad_stride=100, stream=None)
    assert set(change) <= set(a)
    return list({**a, **change}.values())


@pytest.mark.parametrize("change", [
    dict(grad=A + 4), dict(grad=A, grad_stride=64), dict(grad=A, grad_dtype=BF16),
    dict(grad=A, grad_dtype=BF16, grad_stride=200), dict(grad=A - 400),
    dict(grad=B), dict(grad=B + 49 * 24 + 16), dict(grad=C), dict(grad=D), dict(grad=E),
    dict(grad=F), dict(grad=F - 30 * 400), dict(loss=A), dict(loss=A + 252), dict(loss=B),
    dict(loss=C), dict(loss=D), dict(loss=F + 4),
    dict(loss=F - 196),
])
def test_distill_refuses(change):
    assert refuses("train_distill", distill(**change))
