"""The weights that a step updates through their addresses count as changed for autograd:
a graph that saved them refuses its backward pass instead of going on with what stands
there now."""
import pytest
import torch

import optimizer_step_gb300 as og

pytestmark = pytest.mark.gpu

SIZES = [64, 4096]


def flat(dtype):
    """Weights as slices of one buffer."""
    buffer = torch.randn(sum(SIZES), device="cuda").to(dtype)
    return list(buffer.split(SIZES))


def apart(dtype):
    return [torch.randn(n, device="cuda").to(dtype) for n in SIZES]


def make(place, **how):
    weights, w16 = place(torch.float32), place(torch.bfloat16)
    zeros = lambda: [torch.zeros(n, device="cuda") for n in SIZES]
    grads = [torch.randn(n, device="cuda").to(torch.bfloat16) for n in SIZES]
    return og.Lamb(weights, zeros(), zeros(), w16, [0, 1], **how), weights, w16, grads


def step(opt, grads):
    opt.step(0.1, 1, grads=grads)


def step_async(opt, grads):
    opt.set_step(1)
    opt.result(opt.step_async(0.1, grads=grads))


def step_speculative(opt, grads):
    second = [[torch.zeros(n, device="cuda") for n in SIZES] for _ in range(2)]
    opt.set_speculative(*second)
    opt.set_step(1)
    opt.result(opt.step_async(0.1, grads=grads))
    opt.close()


def step_split(opt, grads):
    opt.result(opt.split_step(0.1, t=1, grads=grads))


@pytest.mark.parametrize("run", [step, step_async, step_speculative, step_split],
                         ids=lambda f: f.__name__)
@pytest.mark.parametrize("place", [flat, apart], ids=lambda f: f.__name__)
@pytest.mark.parametrize("which", ["weight", "rounded"])
def test_a_graph_that_saved_the_weights_refuses(run, place, which):
    how = {}
    if run is step_split:
        buffers = [torch.zeros(2, dtype=torch.float64, device="cuda") for _ in range(2)]
        how = dict(exchange_slots=[-1, 0], norm_exchange=buffers[0], tensor_exchange=buffers[1])
    opt, weights, w16, grads = make(place, **how)
    used = (weights if which == "weight" else w16)[0]
    x = torch.randn(5, SIZES[0], device="cuda", requires_grad=True)
    y = og.layer_norm(x, used)
    read = [g._version for g in grads]
    run(opt, grads)
    assert [g._version for g in grads] == read
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    og.layer_norm(x, used).sum().backward()   # a graph behind the step
    opt.close()


def test_weights_of_inference_mode_step_as_before():
    with torch.inference_mode():
        opt, weights, w16, grads = make(apart)
    was = [w.clone() for w in weights]
    step(opt, grads)
    assert not any(torch.equal(a, b) for a, b in zip(weights, was))
    opt.close()
