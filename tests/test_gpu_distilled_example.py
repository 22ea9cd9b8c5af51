"""The lookup, layer norm, the distillation loss, their backward passes, the clip and the
step run together: an example's grads against autograd's in 64 bits, the same through
autograd, and training steps as one captured graph."""
import importlib.util
import math
import os

import pytest
import torch

import optimizer_step_gb300 as og

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "distilled_lm.py")


def load():
    spec = importlib.util.spec_from_file_location("distilled_lm", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def loss_in_64_bits(ex, leaves, batch, vocab, width):
    """The mean loss of the formulas."""
    table, hidden, gain1, shift1, gain2, shift2 = leaves
    table, hidden = table.view(vocab, width), hidden.view(width, width)

    def norm(x, gain, shift):
        c = x - x.mean(-1, keepdim=True)
        return c / torch.sqrt(c.square().mean(-1, keepdim=True) + 1e-5) * gain + shift

    ids, targets, top_ids, top_logits = batch
    x = table[ids]
    x = x + torch.tanh(norm(x, gain1, shift1) @ hidden)
    z = norm(x, gain2, shift2) @ table.t()
    p = torch.softmax(top_logits.double() / 2.0, -1)
    q = torch.log_softmax(z / 2.0, -1).gather(-1, top_ids)
    s = torch.log_softmax(z, -1).gather(-1, targets.clamp(min=0)[..., None])[..., 0]
    rows = 0.5 * 4.0 * (p * (p.log() - q)).sum(-1) - 0.5 * s
    used = targets != ex.IGNORE
    return (rows * used).sum() / used.sum()


def test_grads_of_the_example_match_autograd():
    """From the same bf16 weights.  The activations between are bf16 (half a step is 2^-8
    of the value); some twelve of them lie on a path, so the grads as a whole agree to
    12 * 2^-8 of their size."""
    ex = load()
    vocab, width = 300, 64
    model = ex.DistilledLM(vocab, width)
    for k in range(2, 6):   # norms that are not the identity
        model.w16[k].add_(0.1 * torch.randn(width, device="cuda").to(torch.bfloat16))
    batch = ex.make_batch(6, 40, vocab, 7, seed=3)
    leaves = [w.double().requires_grad_() for w in model.w16]
    loss, stats, seq = model.step(batch, lr=0.0, max_norm=0.0, micro_batches=1)
    assert not model.opt.result(seq)[0]
    want = loss_in_64_bits(ex, leaves, batch, vocab, width)
    want.backward()
    want = float(want.detach())
    assert abs(float(loss) - want) <= 12 * 2.0 ** -8 * abs(want)
    norm = math.sqrt(sum(float(w.grad.square().sum()) for w in leaves))
    for got, leaf in zip(model.grads, leaves):
        assert float((got.double() - leaf.grad).norm()) <= 12 * 2.0 ** -8 * norm
    assert abs(float(stats[0]) - norm) <= 12 * 2.0 ** -8 * norm
    model.close()


def test_the_same_model_through_autograd():
    """With fp32 weights, where autograd calls the operators: fp32 rounding, amplified by
    a path of a few products and two norms, stays below 1e-4 of the grads' size."""
    ex = load()
    vocab, width = 200, 48
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    leaves = [rand(vocab * width) / 7, rand(width * width) / 7, 1 + 0.1 * rand(width),
              0.1 * rand(width), 1 + 0.1 * rand(width), 0.1 * rand(width)]
    batch = ex.make_batch(5, 30, vocab, 6, seed=2)
    ids, targets, top_ids, top_logits = batch
    mine = [w.clone().requires_grad_() for w in leaves]
    table, hidden = mine[0].view(vocab, width), mine[1].view(width, width)
    x = og.embed(table, ids.contiguous())
    x = x + torch.tanh(og.layer_norm(x, mine[2], mine[3]) @ hidden)
    z = og.layer_norm(x, mine[4], mine[5]) @ table.t()
    rows = og.distill_loss(z, top_ids, top_logits, targets.contiguous(), temperature=2.0,
                           soft_weight=0.5, hard_weight=0.5, ignore_id=ex.IGNORE)
    loss = rows.sum() / (targets != ex.IGNORE).sum()
    loss.backward()
    ref = [w.double().requires_grad_() for w in leaves]
    want = loss_in_64_bits(ex, ref, batch, vocab, width)
    want.backward()
    loss, want = float(loss.detach()), float(want.detach())
    assert abs(loss - want) <= 1e-4 * abs(want)
    norm = math.sqrt(sum(float(w.grad.square().sum()) for w in ref))
    for a, b in zip(mine, ref):
        assert float((a.grad.double() - b.grad).norm()) <= 1e-4 * norm


def test_micro_batches_add_up():
    ex = load()
    grads = []
    for parts in (1, 3):
        model = ex.DistilledLM(300, 64)
        batch = ex.make_batch(6, 40, 300, 7, seed=3)
        # Equal numbers of positions that count in each part.
        batch = (batch[0], batch[0], *batch[2:])
        model.step(batch, lr=0.0, max_norm=0.0, micro_batches=parts)
        grads.append(model.sums.clone())
        model.close()
    assert float((grads[0] - grads[1]).norm()) <= 12 * 2.0 ** -8 * float(grads[0].norm())


def test_a_captured_training_step():
    ex = load()
    vocab, width = 512, 128
    model, same = ex.DistilledLM(vocab, width), ex.DistilledLM(vocab, width)
    batch = [t.contiguous() for t in ex.make_batch(4, 32, vocab, 8, seed=0)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # the first calls of the products, outside the graph
        model.micro_batch(*batch[:2], batch[2].flatten(0, 1), batch[3].flatten(0, 1), 1.0)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        model.sums.zero_()
        loss = model.micro_batch(*batch[:2], batch[2].flatten(0, 1), batch[3].flatten(0, 1), 1.0)
    for k in range(3):
        for held, new in zip(batch, ex.make_batch(4, 32, vocab, 8, seed=k)):
            held.copy_(new)
        graph.replay()
        same.sums.zero_()
        want = same.micro_batch(*batch[:2], batch[2].flatten(0, 1), batch[3].flatten(0, 1), 1.0)
        assert torch.equal(loss, want) and torch.equal(model.sums, same.sums)
    model.close()
    same.close()


def test_a_captured_autograd_step():
    """Forwards and backwards captured together, with leaves that no eager graph holds."""
    n, dim, vocab, top = 96, 64, 500, 6
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    ids = torch.randint(vocab, (n, top), generator=gen, device="cuda")
    x, teacher, head = rand(n, dim), rand(n, top), rand(vocab, dim) / 8

    def passes(x, weight, bias):
        z = og.layer_norm(x, weight, bias) @ head.t()
        og.distill_loss(z, ids, teacher, temperature=2.0).sum().backward()

    def leaves():
        return (rand(n, dim).requires_grad_(), rand(dim).requires_grad_(),
                rand(dim).requires_grad_())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        passes(*leaves())
    torch.cuda.current_stream().wait_stream(side)
    captured = leaves()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        passes(*captured)
    for _ in range(2):
        new = leaves()
        with torch.no_grad():
            for a, b in zip(captured, new):
                a.copy_(b)
        for a in captured:
            a.grad.zero_()   # the captured pass adds to it
        graph.replay()
        passes(*new)
        for a, b in zip(captured, new):
            assert float((a.grad - b.grad).norm()) <= 1e-5 * float(b.grad.norm())


def test_the_example_runs():
    losses = load().train(steps=5, report=0)
    assert len(losses) == 5 and all(math.isfinite(x) for x in losses)
