"""The example that runs the lookup, its gradient, the clip and the step
together: its grads against autograd's, and its loss falls."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "tied_embedding_lm.py")


def load():
    spec = importlib.util.spec_from_file_location("tied_embedding_lm", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_grads_of_the_example_match_autograd():
    """In fp64 from the same bf16 weights.  The activations between are bf16
    (unit roundoff 2^-8); some ten of them lie on a path, so the grads as a
    whole agree to 10 * 2^-8 of their size."""
    ex = load()
    model = ex.TiedLM(vocab=300, width=64)
    batch = ex.make_batch(6, 40, 300, seed=3)
    loss, stats, seq = model.step(batch, lr=0.0, max_norm=0.0, micro_batches=1)
    assert not model.opt.result(seq)[0]
    table = model.weights[0].to(torch.bfloat16).double().view(300, 64).requires_grad_()
    hidden = model.weights[1].to(torch.bfloat16).double().view(64, 64).requires_grad_()
    ids, targets = batch[:, :-1], batch[:, 1:]
    x = table[ids] * 8.0
    logits = (x + torch.tanh(x @ hidden)) @ table.t()
    want = torch.nn.functional.cross_entropy(logits.reshape(-1, 300), targets.reshape(-1),
                                             ignore_index=0)
    want.backward()
    want = float(want.detach())
    assert abs(float(loss) - want) <= 10 * 2.0 ** -8 * want
    norm = math.sqrt(sum(float(g.square().sum()) for g in (table.grad, hidden.grad)))
    for got, ref in zip(model.grads, (table.grad, hidden.grad)):
        assert float((got.double() - ref.reshape(-1)).norm()) <= 10 * 2.0 ** -8 * norm
    assert abs(float(stats[0]) - norm) <= 10 * 2.0 ** -8 * norm
    model.close()


def test_the_loss_of_the_example_falls():
    losses = load().train(steps=40, report=0)
    assert losses[0] > 0.8 * math.log(512)
    assert losses[-1] < 0.5 * losses[0], losses[::8]
