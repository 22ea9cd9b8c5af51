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


@pytest.mark.parametrize("to", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value,max_norm,loss_scale", [
    (3e38, 1.0, 1.0), (3e38, 1e-3, 1.0), (1e38, 1e-30, 1.0), (2e38, 1.0, 1e38), (1.0, 0.0, 3e38),
    (3e38, 1e-38, 3e38), (1e30, 1e-3, 1e-3), (3e38, 2.0 ** -149, 1.0)])
def test_factors_below_the_normal_range_of_fp32(value, max_norm, loss_scale, to):
    """Exploded but finite grads: the factor alone would be a number of few bits,
    or zero, where the products are ordinary ones.  Tolerance: the norm's 33
    additions of fp32 squares, halved by the root, the factor's rounding and the
    product's (all 2^-24 each), the rounding to the type (u) and half a subnormal."""
    u = 2.0 ** -8 if to == torch.bfloat16 else 2.0 ** -24
    sub = 2.0 ** -134 if to == torch.bfloat16 else 2.0 ** -150
    values = torch.linspace(0.5, 1.0, 10_001, device="cuda") * value
    grads = [values.clone(), -values[:9].clone(), torch.zeros(3, device="cuda")]
    before = [x.double() for x in grads]
    out = None if to is None else [torch.ones_like(x, dtype=to) for x in grads]
    norm = math.sqrt(sum(float((x / loss_scale).square().sum()) for x in before))
    c = max_norm / norm if 0 < max_norm < norm else 1.0
    with og.GradClip(grads, out) as clipper:
        stats = clipper.clip(max_norm, loss_scale).tolist()
    assert stats[2] == 0.0
    assert abs(stats[1] - c / loss_scale) <= 4e-6 * c / loss_scale + 2.0 ** -150
    assert stats[0] == math.inf if norm > 3.5e38 else abs(stats[0] - norm) <= 4e-6 * norm
    for x, b in zip(out or grads, before):
        want = b * (c / loss_scale)
        tol = (19 * 2.0 ** -24 + u) * 1.01 * want.abs() + sub
        assert bool(((x.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n", [7, 4096, 100_003, 5_000_000])
def test_the_norm_within_what_its_additions_allow(dtype, n):
    """A thread adds 64 squares of 16 bits (32 of fp32) in two chains and then the
    chains, fp64 from there: 33 roundings of positive sums, halved by the root,
    and the norm's own.  33 / 2 + 1 times 2^-24 is 1.05e-6."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    grads = [torch.randn(n, generator=gen, device="cuda").to(dtype).abs_()]
    want = float(grads[0].double().square().sum()) ** 0.5
    with og.GradClip(grads) as clipper:
        assert abs(float(clipper.norm()[0]) - want) <= 1.05e-6 * want
