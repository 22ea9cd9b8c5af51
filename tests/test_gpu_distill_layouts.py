"""The distillation loss where logits and gradient begin differently, and in place of
logits whose rows are copied ahead."""
import math

import pytest
import torch

import optimizer_step_gb300 as og
from test_gpu_distill import BF16, FP16, FP32, Data, near, reference

pytestmark = pytest.mark.gpu


def placed(n, vocab, stride, shift, dtype, values=None):
    """Rows `stride` apart, `shift` elements off the allocation's alignment; 7 between."""
    store = torch.full((shift + n * stride + 64,), 7.0, dtype=dtype, device="cuda")
    rows = store[shift:shift + n * stride].view(n, stride)[:, :vocab]
    if values is not None:
        rows.copy_(values)
    return store, rows


def with_ends(n, vocab, top, dtype):
    """Rows left out in different ways, and entries and labels at both ends of a row."""
    data = Data(n, vocab, top, dtype)
    data.ids[::3, 0], data.ids[::3, 1] = 0, vocab - 1
    data.ids[1::3, 0], data.ids[1::3, 1] = vocab - 2, 1
    data.ids[2::3, 2:] = -1
    data.labels[::4], data.labels[1::4] = vocab - 1, 0
    data.labels[5::17] = -100
    data.row_grad[6::13] = 0.0
    data.ids[7::19] = -1
    return data


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (BF16, FP32), (FP16, BF16), (FP32, FP32),
                                       (FP32, FP16)])
@pytest.mark.parametrize("n,vocab", [(30, 9), (5000, 40), (4000, 1003), (2500, 4096),
                                     (700, 32000), (230, 131071)])
@pytest.mark.parametrize("pads,shifts", [((0, 1), (0, 0)), ((3, 0), (0, 0)), ((0, 0), (0, 1)),
                                         ((5, 2), (3, 1))])
def test_a_gradient_that_begins_differently(dtype, out, n, vocab, pads, shifts):
    data = with_ends(n, vocab, 6, dtype)
    _, data.logits = placed(n, vocab, vocab + pads[0], shifts[0], dtype, data.logits)
    store, grad = placed(n, vocab, vocab + pads[1], shifts[1], out)
    how = dict(temperature=2.0, soft_weight=0.6, hard_weight=0.4, row_grad=data.row_grad)
    loss, got = og.distill_loss_grad(*data.args(), out=grad, **how)
    assert got is grad
    want = reference(data, 2.0, 0.6, 0.4, row_grad=data.row_grad)
    near(loss, *want[:2], "loss")
    near(got, *want[2:], "grad")
    # The values do not depend on where they go.
    alike = torch.empty_strided(grad.shape, data.logits.stride(), dtype=out, device="cuda")
    again = og.distill_loss_grad(*data.args(), out=alike, **how)
    assert torch.equal(again[0], loss) and torch.equal(again[1], got)
    grad.fill_(7.0)
    assert bool((store == 7.0).all())


@pytest.mark.parametrize("n,vocab", [(3000, 1003), (300, 32000)])
def test_broken_rows_of_a_gradient_that_begins_differently(n, vocab):
    data = with_ends(n, vocab, 6, BF16)
    broken = torch.zeros(n, dtype=torch.bool, device="cuda")
    broken[3::29] = True
    broken &= (data.labels >= 0) & (data.row_grad != 0)
    data.logits[broken, vocab // 2] = math.inf
    _, grad = placed(n, vocab, vocab + 1, 0, BF16)
    loss, got = og.distill_loss_grad(*data.args(), hard_weight=0.5, row_grad=data.row_grad,
                                     out=grad)
    assert bool(loss[broken].isnan().all()) and bool(got[broken].isnan().all())
    assert bool(loss[~broken].isfinite().all()) and bool(got[~broken].isfinite().all())


@pytest.mark.parametrize("n,vocab,pad", [(6000, 64, 0), (2500, 4096, 0), (2500, 4099, 2),
                                         (1000, 32001, 0), (500, 131071, 0)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_in_place_of_many_rows(n, vocab, pad, dtype):
    """Each CTA or cluster has many rows, the next on its way while one is overwritten."""
    data = with_ends(n, vocab, 12, dtype)
    _, data.logits = placed(n, vocab, vocab + pad, 0, dtype, data.logits)
    alike = torch.empty_strided((n, vocab), data.logits.stride(), dtype=dtype, device="cuda")
    how = dict(temperature=2.0, soft_weight=0.5, hard_weight=0.5, row_grad=data.row_grad)
    loss, grad = og.distill_loss_grad(*data.args(), out=alike, **how)
    again, into = og.distill_loss_grad(*data.args(), out=data.logits, **how)
    assert torch.equal(again, loss) and torch.equal(into, grad)
