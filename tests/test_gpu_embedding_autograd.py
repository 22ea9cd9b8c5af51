"""The lookup of a table that requires grad: its gradient reaches the table.

Tolerance: as for the gradient itself, any order of adding n fp32 terms and the
product with the scale, (n + 2) 2^-24 |scale| sum|x|, and one rounding to the
table's type (unit roundoff u, half a subnormal h) of the result."""
import pytest
import torch

import optimizer_step_gb300 as og

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
ROUND = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24}
HALF_SUB = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -150}


def randn(shape, dtype, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def randint(high, shape, seed, dtype=torch.int64):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(high, shape, generator=gen, device="cuda", dtype=dtype)


def check(grad, dy, ids, scale, first_row, rows):
    """Against the sum over tokens in 64 bits."""
    flat, x = ids.reshape(-1).long() - first_row, dy.reshape(-1, dy.shape[-1]).double()
    held = (flat >= 0) & (flat < rows)
    zeros = torch.zeros(rows, x.shape[1], dtype=torch.float64, device="cuda")
    ref = scale * zeros.index_add(0, flat[held], x[held])
    size = abs(scale) * zeros.index_add(0, flat[held], x[held].abs())
    n = torch.bincount(flat[held], minlength=rows).double()[:, None]
    tol = 1.01 * ((n + 2) * 2.0 ** -24 * size + ROUND[grad.dtype] * ref.abs()) \
        + HALF_SUB[grad.dtype]
    assert bool(((grad.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("tin,tout", [(BF16, BF16), (FP32, BF16), (FP16, FP32), (FP32, FP32)])
@pytest.mark.parametrize("shape,dim", [((), 8), ((0,), 8), ((7,), 5), ((3, 40), 64),
                                       ((4, 1500), 129)])
def test_backward_through_the_lookup(tin, tout, shape, dim):
    table = randn((300, dim), tin, 1).requires_grad_()
    ids = randint(900, shape, 2, torch.int32)
    out = og.embed(table, ids, scale=1.5, first_row=350, out_dtype=tout)
    assert out.requires_grad and out.dtype == tout
    assert torch.equal(out, og.embed(table.detach(), ids, scale=1.5, first_row=350,
                                     out_dtype=tout))
    dy = randn(shape + (dim,), tout, 3)
    out.backward(dy)
    assert table.grad.dtype == tin and table.grad.shape == table.shape
    check(table.grad, dy, ids, 1.5, 350, 300)


def test_backward_of_grads_without_rows_of_their_own():
    """A sum's gradient is one number for all; a transposed one steps oddly."""
    table = randn((30, 16), FP32, 1).requires_grad_()
    ids = randint(30, (4, 50), 2)
    og.embed(table, ids).sum().backward()
    check(table.grad, torch.ones(4, 50, 16, device="cuda"), ids, 1.0, 0, 30)
    table.grad = None
    weight = randn((50, 16, 4), FP32, 3)
    (og.embed(table, ids, scale=2.0).permute(1, 2, 0) * weight).sum().backward()
    check(table.grad, weight.permute(2, 0, 1).contiguous(), ids, 2.0, 0, 30)


def test_backward_matches_differences():
    """Linear, with values of few bits: every difference is exact."""
    table = (randint(128, (6, 5), 1) - 64).float() / 16
    ids, weight = randint(6, (11,), 2), (randint(128, (11, 5), 3) - 64).float() / 8
    leaf = table.clone().requires_grad_()
    (og.embed(leaf, ids, scale=4.0) * weight).sum().backward()
    loss = lambda t: float((og.embed(t, ids, scale=4.0).double() * weight.double()).sum())
    for v in range(6):
        for d in range(5):
            step = torch.zeros_like(table)
            step[v, d] = 0.25
            assert float(leaf.grad[v, d]) == (loss(table + step) - loss(table - step)) / 0.5


def test_a_table_used_twice_gets_both_gradients():
    table = randn((40, 24), FP32, 1).requires_grad_()
    a, b = randint(40, (500,), 2), randint(40, (60,), 3)
    (og.embed(table, a).sum() + 3.0 * og.embed(table, b).sum()).backward()
    want = torch.bincount(a, minlength=40) + 3 * torch.bincount(b, minlength=40)
    assert torch.equal(table.grad, want.float()[:, None].expand(40, 24))


def test_no_history_where_none_is_asked_for():
    table = randn((40, 24), FP32, 1).requires_grad_()
    ids = randint(40, (9,), 2)
    with torch.no_grad():
        assert not og.embed(table, ids).requires_grad
        out = torch.empty(9, 24, device="cuda")
        assert og.embed(table, ids, out=out) is out and not out.requires_grad
    with torch.inference_mode():
        assert not og.embed(table, ids).requires_grad
    assert not og.embed(table.detach(), ids).requires_grad


def test_refusals_of_what_has_no_gradient():
    table = randn((40, 24), FP32, 1).requires_grad_()
    ids = randint(40, (9,), 2)
    with pytest.raises(RuntimeError):   # as torch refuses out= of what requires grad
        og.embed(table, ids, out=torch.empty(9, 24, device="cuda"))
    out = og.embed(table, ids)
    with pytest.raises(RuntimeError):   # once only
        torch.autograd.grad(torch.autograd.grad(out.square().sum(), table,
                                                create_graph=True)[0].sum(), table)
    out = og.embed(table, ids)
    ids.add_(1)
    with pytest.raises(RuntimeError):   # ids changed since
        out.sum().backward()
