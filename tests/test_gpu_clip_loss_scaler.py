"""The clip in front of a step whose dynamic loss scaler is on: the step divides by
its own scale, so the clip leaves the scale in the grads."""
import math

import pytest
import torch

import optimizer_step_gb300 as og

pytestmark = pytest.mark.gpu

SIZES = [4096, 70_001, 33]


class Run:
    def __init__(self, seed, grad_dtype=torch.bfloat16):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        new = lambda dtype: [torch.zeros(n, dtype=dtype, device="cuda") for n in SIZES]
        self.w, self.m, self.v, self.w16 = (new(torch.float32), new(torch.float32),
                                            new(torch.float32), new(torch.bfloat16))
        for w in self.w:
            w.copy_(torch.randn(w.numel(), generator=gen, device="cuda"))
        self.sums, self.grads = new(torch.float32), new(grad_dtype)
        self.clipper = og.GradClip(self.sums, out=self.grads, poison=True)
        self.opt = og.Lamb(self.w, self.m, self.v, self.w16, [1, 0, 1], grad_dtype=grad_dtype)

    def backward(self, seed, scale):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        for s in self.sums:
            s.copy_(torch.randn(s.numel(), generator=gen, device="cuda") * scale)

    def state(self):
        return self.w + self.m + self.v + self.w16

    def close(self):
        self.clipper.close()
        self.opt.close()


@pytest.mark.parametrize("max_norm", [0.0, 1.0, 1e6])
def test_clipped_steps_equal_those_without_a_scaler(max_norm):
    """Scales are powers of two and no grad is subnormal, so the bits agree."""
    scaled, plain = Run(1), Run(1)
    scaled.opt.set_loss_scaler(init_scale=1024.0, growth_interval=2)
    plain.opt.set_step(1)
    scaled.opt.set_step(1)
    used = []
    for k in range(5):
        s = scaled.opt.next_loss_scale
        used.append(s)
        scaled.backward(k, s)
        plain.backward(k, 1.0)
        a = scaled.clipper.clip(max_norm * s)
        b = plain.clipper.clip(max_norm)
        assert float(a[0]) == s * float(b[0]) and float(a[1]) == float(b[1])
        _, norm, _ = scaled.opt.result(scaled.opt.step_async(lr=0.01, grads=scaled.grads))
        _, want, _ = plain.opt.result(plain.opt.step_async(lr=0.01, grads=plain.grads))
        assert norm == want
        assert all(torch.equal(x, y) for x, y in zip(scaled.state(), plain.state()))
    assert used == [1024.0, 1024.0, 2048.0, 2048.0, 4096.0]
    scaled.close()
    plain.close()


def test_an_overflow_skips_the_step_and_backs_the_scale_off():
    run = Run(2)
    run.opt.set_loss_scaler(init_scale=1024.0)
    run.opt.set_step(1)
    for k in range(2):
        run.backward(k, 1024.0)
        run.clipper.clip(1024.0)
        assert not run.opt.result(run.opt.step_async(lr=0.01, grads=run.grads))[0]
    before = [x.clone() for x in run.state()]
    run.backward(3, 1024.0)
    run.sums[1][70_000] = math.inf
    run.clipper.clip(1024.0)
    assert run.opt.result(run.opt.step_async(lr=0.01, grads=run.grads))[0]
    assert run.opt.next_loss_scale == 512.0
    assert all(torch.equal(a, b) for a, b in zip(run.state(), before))
    run.close()
