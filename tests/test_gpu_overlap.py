"""Results next to what their call reads, in one buffer, are taken; results partly over
it are refused."""
import pytest
import torch

import optimizer_step_gb300 as og
from optimizer_step_gb300 import LambError

pytestmark = pytest.mark.gpu

N, DIM = 300, 64


def check(x, out, into):
    """A normal call into `into`, which lies beside `x`."""
    keep = x.clone()
    want = og.layer_norm(keep, out_dtype=out.dtype)
    got = og.layer_norm(x, out=into)
    assert torch.equal(got, want) and torch.equal(x, keep)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_results_beside_what_is_read(dtype):
    base = torch.randn(3 * N, 3 * DIM, device="cuda").to(dtype)
    left, right = base[:N, :DIM], base[:N, DIM:2 * DIM]
    check(left, left, right)                                  # columns of one matrix
    check(right, right, left)
    check(base[:2 * N:2, :DIM], left, base[1:2 * N:2, :DIM])  # every other row
    check(base[:N], base[:N], base[N:2 * N])                  # one behind the other
    check(base[N:2 * N], base[:N], base[:N])
    check(base[:N:2, :DIM], left, base[1:2 * N:4, 4:4 + DIM])  # at two strides, never meeting
    both = torch.randn(N, 2 * DIM, device="cuda")              # two types in one buffer
    half = both.view(torch.bfloat16)[:, 2 * DIM:3 * DIM]
    check(both[:, :DIM], half, half)


def test_shapes_of_one_row_and_gradients_beside_one_another():
    row = torch.randn(1, 3 * DIM, device="cuda")
    check(row[:, :DIM], row, row[:, DIM:2 * DIM])
    assert torch.equal(og.layer_norm(row[:, :DIM], out=row[:, :DIM]), row[:, :DIM])
    x, dy = torch.randn(N, DIM, device="cuda"), torch.randn(N, DIM, device="cuda")
    _, stats = og.layer_norm(x, stats=True)
    sums = torch.empty(2 * DIM, device="cuda")
    got = og.layer_norm_grad(dy, x, None, stats, weight_grad=sums[:DIM], bias_grad=sums[DIM:])
    want = og.layer_norm_grad(dy, x, None, stats)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_partly_over_is_refused():
    base = torch.randn(2 * N, 2 * DIM, device="cuda")
    x = base[:N, :DIM]
    dy = torch.randn(N, DIM, device="cuda")
    _, stats = og.layer_norm(x, stats=True)
    weight = base[N - 1, DIM:]
    ids, teacher = torch.zeros(N, 2, dtype=torch.int64, device="cuda"), torch.zeros(
        N, 2, device="cuda")
    keep = base.clone()
    bad = [
        lambda: og.layer_norm(x, out=base[:N, 1:DIM + 1]),
        lambda: og.layer_norm(x, out=base[1:N + 1, :DIM]),
        lambda: og.layer_norm(x, out=base[::2, :DIM]),
        lambda: og.layer_norm(x, out=base.view(torch.bfloat16)[:N, :DIM]),
        lambda: og.layer_norm(x, weight, out=base[:N, DIM:]),
        lambda: og.layer_norm_grad(dy, x, None, stats, x_grad=base[1:N + 1, :DIM]),
        lambda: og.layer_norm_grad(dy, x, weight, stats, x_grad=base[:N, DIM:]),
        lambda: og.layer_norm_grad(dy, x, None, stats, weight_grad=base[0, :DIM],
                                   bias_grad=base[0, 4:DIM + 4]),
        lambda: og.distill_loss_grad(x, ids, teacher, out=base[:N, 2:DIM + 2]),
        lambda: og.distill_loss_grad(x, ids, teacher, out=base.view(torch.bfloat16)[:N, :DIM]),
    ]
    for call in bad:
        with pytest.raises(LambError, match="overlap"):
            call()
    assert torch.equal(base, keep)


@pytest.mark.parametrize("n,vocab", [(40, 5), (3000, 4096), (600, 131071), (5, 700_000)])
def test_losses_in_place_of_their_row_grads(n, vocab):
    """Through the C entry point, which takes the address."""
    z = torch.randn(n, vocab, device="cuda").to(torch.bfloat16)
    labels = torch.randint(vocab, (n,), device="cuda")
    row_grad = torch.rand(n, device="cuda")
    want, want_grad = og.distill_loss_grad(z, None, None, labels, hard_weight=1.0,
                                           row_grad=row_grad)
    grad = torch.empty_like(z)
    rc = og.load().train_distill(
        z.data_ptr(), 0, vocab, n, vocab, None, 0, 0, None, 0, 0, 0, labels.data_ptr(), 1, -100,
        1.0, 1.0, 1.0, row_grad.data_ptr(), row_grad.data_ptr(), 1.0, grad.data_ptr(), 0, vocab,
        torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(row_grad, want) and torch.equal(grad, want_grad)
