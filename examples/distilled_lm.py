"""A small language model that learns from a larger one's most likely tokens.

Embedding, layer norm, a hidden layer on the residual stream, layer norm, and the
embedding again as the output head.  The loss weighs the teacher's top logits at a
temperature against the true next token.  Everything but the matrix products is the
framework's: the lookup, both layer norms, the loss with its gradient, their backward
passes, the clip and the LAMB step.  The norms' weights and biases take no weight decay.
Nothing waits for the GPU within a step.

    python examples/distilled_lm.py [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from optimizer_step_gb300 import (GradClip, Lamb, distill_loss_grad, embed,  # noqa: E402
                                  embed_grad, layer_norm, layer_norm_grad)

ALIGN = 64  # elements between tensor starts
IGNORE = -100


def flat(sizes, dtype, device):
    """Zeroed tensors at aligned offsets of one buffer."""
    offsets, at = [], 0
    for n in sizes:
        offsets.append(at)
        at += (n + ALIGN - 1) // ALIGN * ALIGN
    buffer = torch.zeros(at, dtype=dtype, device=device)
    return buffer, [buffer[o:o + n] for o, n in zip(offsets, sizes)]


class DistilledLM:
    """x = embedding; x = x + tanh(norm(x) W); logits = norm(x) against the embedding."""

    def __init__(self, vocab, width, temperature=2.0, soft_weight=0.5, hard_weight=0.5,
                 device="cuda", seed=0):
        self.vocab, self.width = vocab, width
        self.how = dict(temperature=temperature, soft_weight=soft_weight,
                        hard_weight=hard_weight, ignore_id=IGNORE)
        # The table, the hidden matrix, and weight and bias of the two norms.
        sizes = [vocab * width, width * width] + [width] * 4
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        _, self.weights = flat(sizes, torch.float32, device)
        _, self.w16 = flat(sizes, torch.bfloat16, device)
        for k, w in enumerate(self.weights):
            if k < 2:
                w.copy_(torch.randn(w.numel(), generator=gen, device=device) / width ** 0.5)
            else:
                w.fill_(1.0 if k % 2 == 0 else 0.0)
            self.w16[k].copy_(w)
        self.sums, self.sum_views = flat(sizes, torch.float32, device)
        _, self.grads = flat(sizes, torch.bfloat16, device)
        _, exp_avg = flat(sizes, torch.float32, device)
        _, exp_avg_sq = flat(sizes, torch.float32, device)
        self.clipper = GradClip(self.sum_views, out=self.grads, poison=True)
        self.opt = Lamb(self.weights, exp_avg, exp_avg_sq, self.w16, [1, 1, 0, 0, 0, 0])
        self.opt.set_step(1)

    def micro_batch(self, ids, targets, top_ids, top_logits, weight):
        """Adds the grads of weight * (mean loss) to the fp32 sums; returns the mean loss.
        Positions whose target is IGNORE count nothing."""
        table, hidden = self.w16[0].view(self.vocab, self.width), self.w16[1].view(
            self.width, self.width)
        gain1, shift1, gain2, shift2 = self.w16[2:]
        d_table = self.sum_views[0].view(self.vocab, self.width)
        d_hidden = self.sum_views[1].view(self.width, self.width)
        ids, targets = ids.reshape(-1), targets.reshape(-1)
        # Forwards.
        x0 = embed(table, ids)
        n1, stats1 = layer_norm(x0, gain1, shift1, stats=True)
        h = torch.tanh(n1 @ hidden)
        x1 = x0 + h
        n2, stats2 = layer_norm(x1, gain2, shift2, stats=True)
        logits = n2 @ table.t()
        used = targets != IGNORE
        count = used.sum().clamp(min=1)
        losses, d_logits = distill_loss_grad(logits, top_ids, top_logits, targets,
                                             row_grad=used * (weight / count), out=logits,
                                             **self.how)
        # Backwards.
        d_table += d_logits.t() @ n2
        d_x1, _, _ = layer_norm_grad(d_logits @ table, x1, gain2, stats2,
                                     weight_grad=self.sum_views[4],
                                     bias_grad=self.sum_views[5], accumulate=True)
        d_h = (d_x1.float() * (1.0 - h.float().square())).to(torch.bfloat16)
        d_hidden += n1.t() @ d_h
        d_x0, _, _ = layer_norm_grad(d_h @ hidden.t(), x0, gain1, stats1,
                                     weight_grad=self.sum_views[2],
                                     bias_grad=self.sum_views[3], accumulate=True)
        embed_grad(d_x0 + d_x1, ids, out=d_table, accumulate=True)
        return losses.sum() / count

    def step(self, batch, lr, max_norm=1.0, micro_batches=2):
        """One optimizer step on (ids, targets, top ids, top logits), each [n, length, ...];
        returns (mean loss, the clip's stats, the step's sequence number), without waiting."""
        self.sums.zero_()
        loss = 0.0
        for parts in zip(*(t.chunk(micro_batches) for t in batch)):
            ids, targets, top_ids, top_logits = (t.contiguous() for t in parts)
            loss = loss + self.micro_batch(ids, targets, top_ids.flatten(0, 1),
                                           top_logits.flatten(0, 1),
                                           1.0 / micro_batches) / micro_batches
        stats = self.clipper.clip(max_norm)
        seq = self.opt.step_async(lr=lr, grads=self.grads)
        return loss, stats, seq

    def close(self):
        self.clipper.close()
        self.opt.close()


def make_batch(n, length, vocab, top, seed, device="cuda"):
    """Counting sequences and a teacher that knows the rule: token t is followed by
    (3 t + 1) mod vocab, nearly always.  Some sequences end early."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    ids = torch.empty(n, length + 1, dtype=torch.int64, device=device)
    ids[:, 0] = torch.randint(vocab, (n,), generator=gen, device=device)
    for k in range(length):
        ids[:, k + 1] = (3 * ids[:, k] + 1) % vocab
    following = ids[:, 1:]
    ends = torch.randint(length // 2, length + 1, (n, 1), generator=gen, device=device)
    targets = following.masked_fill(torch.arange(length, device=device) >= ends, IGNORE)
    # The teacher's tokens, the right one first.
    order = torch.arange(top, device=device)
    top_ids = (following[..., None] + order * (vocab // top)) % vocab
    top_logits = torch.where(order == 0, 6.0, 0.0) + torch.randn(
        n, length, top, generator=gen, device=device)
    return ids[:, :-1], targets, top_ids, top_logits.to(torch.bfloat16)


def train(steps=60, vocab=512, width=256, n=16, length=64, top=8, lr=0.03, report=10):
    """Trains and returns the losses."""
    model = DistilledLM(vocab, width)
    losses = []
    for k in range(steps):
        loss, stats, seq = model.step(make_batch(n, length, vocab, top, seed=k), lr)
        losses.append(loss)
        if report and (k % report == 0 or k == steps - 1):
            skipped, _, t = model.opt.result(seq)
            norm, factor, _ = stats.tolist()
            print(f"step {t}: loss {float(loss):.3f}  grad norm {norm:.3f}  "
                  f"factor {factor:.3f}{'  skipped' if skipped else ''}")
    model.close()
    return [float(x) for x in losses]


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=60)
    train(parser.parse_args().steps)
