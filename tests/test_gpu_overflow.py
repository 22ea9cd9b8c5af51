"""An inf or NaN grad on its way through the clip to the optimizer step: the step
must skip, whatever the clip's outputs held before."""
import math

import pytest
import torch

import optimizer_step_gb300 as og
import test_gpu_training_example as example

pytestmark = pytest.mark.gpu


def state(model):
    return [x.clone() for group in (model.weights, model.w16, *model.opt.state_buffers())
            for x in group]


@pytest.mark.parametrize("clean_steps", [0, 2])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_the_example_skips_a_step_whose_sums_overflow(bad, clean_steps):
    """Behind clean steps the clip's outputs hold grads that have been applied;
    before the first one they are zero, which would still decay the weights."""
    ex = example.load()

    class Overflowing(ex.TiedLM):
        plant = False

        def micro_batch(self, *args):
            loss = super().micro_batch(*args)
            if self.plant:
                self.sum_views[1][5] = bad
            return loss

    model = Overflowing(vocab=300, width=64)
    batch = ex.make_batch(6, 40, 300, seed=3)
    for _ in range(clean_steps):
        _, _, seq = model.step(batch, lr=0.01)
        assert not model.opt.result(seq)[0]
    before = state(model)
    model.plant = True
    _, stats, seq = model.step(batch, lr=0.01)
    skipped, _, t = model.opt.result(seq)
    assert skipped and stats.tolist() == [math.inf, 0.0, 1.0]
    assert all(torch.equal(a, b) for a, b in zip(state(model), before))
    model.plant = False
    _, stats, seq = model.step(batch, lr=0.01)
    skipped, _, t_next = model.opt.result(seq)
    assert not skipped and t_next == t and float(stats[2]) == 0.0
    assert not torch.equal(model.weights[0], before[0])
    model.close()


BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
SIZES = [5, 4097, 0, 70_003, 16, 1]


def tensors(types, seed):
    """Tensors one element off the alignment in a buffer of 7.0 each."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    buffers = [torch.full((n + 9,), 7.0, dtype=t, device="cuda") for n, t in zip(SIZES, types)]
    found = [b[1:1 + n] for b, n in zip(buffers, SIZES)]
    for x in found:
        x.copy_(torch.randn(x.numel(), generator=gen, device="cuda"))
    return found, buffers


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("to", [BF16, FP16, FP32, "in place"])
@pytest.mark.parametrize("types", [[BF16] * 6, [FP16] * 6, [FP32] * 6, [BF16, FP32, FP16] * 2])
def test_poison_turns_every_output_to_nan_and_nothing_else(types, to, bad):
    grads, buffers = tensors(types, 1)
    out, others = (None, buffers) if to == "in place" else tensors([to] * 6, 2)
    with og.GradClip(grads, out, poison=True) as clipper:
        out = grads if out is None else out
        stats = clipper.clip(1.0, loss_scale=2.0)   # clean: as without poison
        assert float(stats[2]) == 0.0 and all(bool(x.isfinite().all()) for x in out)
        grads[3][33_333] = bad
        assert clipper.norm().tolist() == [math.inf, 0.0, 1.0]   # the norm writes no output
        assert all(bool(x.isfinite().all()) for i, x in enumerate(out) if i != 3)
        assert clipper.clip(0.0).tolist() == [math.inf, 0.0, 1.0]
        assert all(bool(x.isnan().all()) for x in out)
        for x, b in zip(out, others):
            assert float(b[0]) == 7.0 and bool((b[1 + x.numel():] == 7.0).all())
        if to != "in place":   # the next clean call writes them all again
            grads[3][33_333] = 1.0
            assert float(clipper.clip(1.0)[2]) == 0.0
            assert all(bool(x.isfinite().all()) for x in out)


@pytest.mark.parametrize("in_place", [False, True])
def test_poison_reaches_the_ranks_whose_own_grads_are_clean(in_place):
    grads, _ = tensors([FP32] * 6, 3)
    grads[0][2] = math.inf
    out = grads if in_place else tensors([BF16] * 6, 4)[0]
    ex = [torch.zeros(2, dtype=torch.float64, device="cuda") for _ in range(2)]
    make = lambda k: og.GradClip(grads[k], None if in_place else out[k], poison=True)
    with make(slice(0, 2)) as a, make(slice(2, 6)) as b:
        total = a.partial(ex[0]) + b.partial(ex[1])
        for clipper in (a, b):
            assert clipper.finish(total, 1.0).tolist() == [math.inf, 0.0, 1.0]
    assert all(bool(x.isnan().all()) for x in out)


@pytest.mark.parametrize("in_place", [False, True])
def test_without_poison_outputs_keep_what_they_held(in_place):
    grads, _ = tensors([FP32] * 6, 5)
    out = None if in_place else tensors([BF16] * 6, 6)[0]
    grads[1][7] = math.nan
    kept = [x.clone() for x in (out or grads)]
    with og.GradClip(grads, out) as clipper:
        clipper.clip(1.0)
        assert all(torch.equal(a.nan_to_num(9.0), b.nan_to_num(9.0))
                   for a, b in zip(out or grads, kept))


def test_poison_is_refused_if_it_is_neither_0_nor_1():
    from optimizer_step_gb300 import _lib
    lib = og.load()
    assert lib.train_clip_set_poison(None, 1) == _lib.LAMB_ERR_INVALID
    with og.GradClip(tensors([FP32] * 6, 7)[0]) as clipper:
        assert lib.train_clip_set_poison(clipper._handle(), 2) == _lib.LAMB_ERR_INVALID
