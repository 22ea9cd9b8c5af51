"""A small language model trained with the operators around the LAMB step.

Next-token prediction with a tied embedding: the lookup starts the forward
pass, one hidden layer follows, and the table is the output head too, whose
logits the loss turns into their gradient.  Every
step sums the grads of a few micro-batches in fp32, where the table gets two
contributions: the head's product, and on top of it the lookup's gradient by
sorted tokens.  GradClip takes the fp32 sums to the bf16 grads that the step
reads, clipped by their global norm, and Lamb updates the weights.  Nothing
waits for the GPU within a step: when the sums overflow, the clip leaves NaN in
the step's grads and the step skips.

    python examples/tied_embedding_lm.py [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from optimizer_step_gb300 import (GradClip, Lamb, distill_loss_grad, embed,  # noqa: E402
                                  embed_grad)

ALIGN = 64  # elements between tensor starts


def flat(sizes, dtype, device):
    """Zeroed tensors at aligned offsets of one buffer."""
    offsets, at = [], 0
    for n in sizes:
        offsets.append(at)
        at += (n + ALIGN - 1) // ALIGN * ALIGN
    buffer = torch.zeros(at, dtype=dtype, device=device)
    return buffer, [buffer[o:o + n] for o, n in zip(offsets, sizes)]


class TiedLM:
    """embedding -> tanh(x W) + x -> logits against the embedding."""

    def __init__(self, vocab, width, padding_id=0, device="cuda", seed=0):
        self.vocab, self.width, self.padding_id = vocab, width, padding_id
        sizes = [vocab * width, width * width]
        self.scale = width ** 0.5
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        _, self.weights = flat(sizes, torch.float32, device)
        _, self.w16 = flat(sizes, torch.bfloat16, device)
        for w, w16 in zip(self.weights, self.w16):
            w.copy_(torch.randn(w.numel(), generator=gen, device=device) * (0.5 / self.scale))
            w16.copy_(w)
        self.sums, self.sum_views = flat(sizes, torch.float32, device)
        _, self.grads = flat(sizes, torch.bfloat16, device)
        _, exp_avg = flat(sizes, torch.float32, device)
        _, exp_avg_sq = flat(sizes, torch.float32, device)
        self.clipper = GradClip(self.sum_views, out=self.grads, poison=True)
        self.opt = Lamb(self.weights, exp_avg, exp_avg_sq, self.w16, [1, 1])
        self.opt.set_step(1)

    def micro_batch(self, ids, targets, weight):
        """Adds the grads of weight * (mean loss) to the fp32 sums; returns the
        mean loss.  Positions whose target is the padding count nothing."""
        table = self.w16[0].view(self.vocab, self.width)
        hidden_w = self.w16[1].view(self.width, self.width)
        x = embed(table, ids, scale=self.scale)
        h = torch.tanh((x @ hidden_w).float())
        y = (x.float() + h).to(torch.bfloat16)
        logits = y @ table.t()
        # The loss and its gradient, in place of the logits.
        used = targets != self.padding_id
        count = used.sum().clamp(min=1)
        losses, d_logits = distill_loss_grad(
            logits, None, None, targets, hard_weight=1.0, ignore_id=self.padding_id,
            row_grad=used * (weight / count), out=logits)
        loss = losses.sum() / count
        # Backwards through the head, the hidden layer and the lookup.
        rows = d_logits.reshape(-1, self.vocab)
        flat_x, flat_y = x.reshape(-1, self.width), y.reshape(-1, self.width)
        d_y = (rows @ table).float()
        d_z = (d_y * (1.0 - h.reshape(-1, self.width).square())).to(torch.bfloat16)
        d_x = (d_y + (d_z @ hidden_w.t()).float()).to(torch.bfloat16)
        d_table = self.sum_views[0].view(self.vocab, self.width)
        d_table += rows.t() @ flat_y
        self.sum_views[1].view(self.width, self.width).add_(flat_x.t() @ d_z)
        embed_grad(d_x.view(*ids.shape, self.width), ids, out=d_table, scale=self.scale,
                   accumulate=True)
        return loss

    def step(self, batch, lr, max_norm=1.0, micro_batches=2):
        """One optimizer step on ids [n, length + 1]; returns (mean loss, the
        clip's stats, the step's sequence number), all without waiting."""
        self.sums.zero_()
        loss = 0.0
        for part in batch.chunk(micro_batches):
            loss = loss + self.micro_batch(part[:, :-1].contiguous(), part[:, 1:].contiguous(),
                                           1.0 / micro_batches) / micro_batches
        stats = self.clipper.clip(max_norm)
        seq = self.opt.step_async(lr=lr, grads=self.grads)
        return loss, stats, seq

    def close(self):
        self.clipper.close()
        self.opt.close()


def make_batch(n, length, vocab, seed, device="cuda"):
    """Counting sequences: token t is followed by (3 t + 1) mod (vocab - 1), plus
    one; token 0 is the padding that ends some of them."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    ids = torch.empty(n, length + 1, dtype=torch.int64, device=device)
    ids[:, 0] = torch.randint(1, vocab, (n,), generator=gen, device=device)
    for k in range(length):
        ids[:, k + 1] = (3 * ids[:, k] + 1) % (vocab - 1) + 1
    ends = torch.randint(length // 2, length + 2, (n, 1), generator=gen, device=device)
    return ids.masked_fill(torch.arange(length + 1, device=device) >= ends, 0)


def train(steps=60, vocab=512, width=256, n=16, length=64, lr=0.03, report=10):
    """Trains and returns the losses."""
    model = TiedLM(vocab, width)
    losses = []
    for k in range(steps):
        loss, stats, seq = model.step(make_batch(n, length, vocab, seed=k), lr)
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
