"""The clip at the ends of its scales."""
import math

import pytest
import torch

import optimizer_step_gb300 as og

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("loss_scale", [2.0 ** -149, 2.0 ** -130, 2.0 ** -128])
def test_a_loss_scale_without_a_reciprocal_in_fp32_is_refused(loss_scale):
    """The factor would be inf, and zeros times it NaN."""
    grads = [torch.zeros(100, device="cuda")]
    with og.GradClip(grads) as clipper:
        with pytest.raises(og.LambError):
            clipper.norm(loss_scale)
        with pytest.raises(og.LambError):
            clipper.clip(1.0, loss_scale)
        with pytest.raises(og.LambError):
            clipper.finish(torch.zeros(2, dtype=torch.float64, device="cuda"), 1.0, loss_scale)


@pytest.mark.parametrize("loss_scale", [2.0 ** -127, 2.0 ** -126, 2.0 ** 127])
def test_the_outermost_loss_scales(loss_scale):
    grads = [torch.full((4,), 2.0 ** -140 if loss_scale < 1 else 2.0 ** 100, device="cuda"),
             torch.zeros(9, device="cuda")]
    norm = 2.0 * float(grads[0][0]) / loss_scale
    want = grads[0].double() / loss_scale
    with og.GradClip(grads) as clipper:
        assert clipper.clip(0.0, loss_scale).tolist() == [norm, 1.0 / loss_scale, 0.0]
    assert torch.equal(grads[0].double(), want) and not grads[1].any()
