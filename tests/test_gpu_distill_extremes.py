"""The distillation loss where a teacher's logits lie further apart than fp32's largest
number, and at the temperatures next to those that are refused."""
import math

import pytest
import torch

import optimizer_step_gb300 as og

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,vocab", [(20, 5), (20, 4096), (2500, 4096), (3, 1_300_000)])
def test_an_entry_without_a_share_adds_nothing_to_the_loss(n, vocab):
    """Masked by the type's lowest value next to a logit of 1e38: the difference is past
    fp32 and the entry's probability 0, so its term is 0, as p log p is."""
    z = torch.randn(n, vocab, device="cuda")
    ids = torch.tensor([[1, 2, 3]], device="cuda").expand(n, 3).contiguous()
    teacher = torch.tensor([[1e38, torch.finfo(torch.float32).min, 1e38]],
                           device="cuda").expand(n, 3).contiguous()
    alone = ids[:, ::2].contiguous(), teacher[:, ::2].contiguous()
    want, want_grad = og.distill_loss_grad(z, *alone)
    assert bool(want.isfinite().all())
    loss, grad = og.distill_loss_grad(z, ids, teacher)
    assert torch.equal(loss, want) and torch.equal(grad, want_grad)
    assert torch.equal(og.distill_loss(z, ids, teacher), og.distill_loss(z, *alone))


@pytest.mark.parametrize("n,vocab", [(20, 5), (20, 4096), (2500, 4096), (3, 1_300_000)])
def test_named_tokens_further_from_the_largest_than_fp32_reaches(n, vocab):
    """The student's logits are 1e38 and the lowest value, 4.4e38 apart; a share of 0.18 of
    that is a loss that fp32 holds: soft T p (the difference), with log sizes of at most 13
    lost beside it."""
    lowest = torch.finfo(torch.float32).min
    z = torch.zeros(n, vocab, device="cuda")
    z[:, 1], z[:, 2] = 1e38, lowest
    apart = 1e38 - lowest
    ids = torch.tensor([[1, 2]], device="cuda").expand(n, 2).contiguous()
    teacher = torch.tensor([[1.5, 0.0]], device="cuda").expand(n, 2).contiguous()
    share = 1.0 / (1.0 + math.exp(1.5))
    labels = torch.full((n,), 2, device="cuda")
    for args, want, how in (((ids, teacher), share * apart, {}),
                            ((None, None, labels), 0.3 * apart, dict(hard_weight=0.3)),
                            ((ids, teacher, labels), (0.5 * share + 0.25) * apart,
                             dict(soft_weight=0.5, hard_weight=0.25))):
        # A few roundings of products, and of the share's exponential.
        for got in (og.distill_loss(z, *args, **how), og.distill_loss_grad(z, *args, **how)[0]):
            assert bool(((got.double() - want).abs() <= 16 * 2.0 ** -24 * want).all())


@pytest.mark.parametrize("vocab", [5, 4096])
@pytest.mark.parametrize("temperature", [1e-30, 1e30, 3e38])
def test_the_farthest_temperatures(vocab, temperature):
    """At the low end only the largest logits have a share, at the high end all alike."""
    n = 8
    z = torch.randn(n, vocab, device="cuda")
    ids = torch.arange(4, device="cuda").expand(n, 4).contiguous()
    teacher = torch.randn(n, 4, device="cuda")
    loss, grad = og.distill_loss_grad(z, ids, teacher, temperature=temperature,
                                      soft_weight=1.0 / temperature
                                      if temperature > 1 else 1.0)
    if temperature < 1:
        want = torch.zeros(n, vocab, device="cuda")
        rows = torch.arange(n, device="cuda")
        want[rows, z.argmax(1)] += 1.0
        want[rows, ids[rows, teacher.argmax(1)]] -= 1.0
        want *= temperature
    else:
        want = torch.full((n, vocab), 1.0 / vocab, device="cuda")
        want[:, :4] -= 0.25
    tol = 1e-5 * want.abs().max()
    assert bool(((grad - want).abs() <= tol).all())
    assert not bool(loss.isnan().any())
