"""Layer norm and its backward pass in place of rows that are copied ahead, and the
widest rows on chip in each pair of types."""
import pytest
import torch

import optimizer_step_gb300 as og
from test_gpu_layer_norm import BF16, FP16, FP32, both, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [24, 64, 256, 1023, 4096, 12288])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("pad", [0, 8])
def test_in_place_of_many_rows(dim, dtype, pad):
    """Each group has many rows, the next on their way while one is overwritten."""
    n = 5003 if dim > 100 else 60_001
    x, dy = (randn((n, dim + pad), dtype, k)[:, :dim] for k in (1, 2))
    weight, bias = randn((dim,), dtype, 3), randn((dim,), dtype, 4)
    alike = lambda t: torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
    y, stats = og.layer_norm(x, weight, bias, stats=True, out=alike(x))
    z = alike(x).copy_(x)
    assert og.layer_norm(z, weight, bias, out=z) is z and torch.equal(z, y)
    want = og.layer_norm_grad(dy, x, weight, stats, x_grad=alike(x))
    for into in (0, 1):
        args = [alike(t).copy_(t) for t in (dy, x)]
        got = og.layer_norm_grad(*args, weight, stats, x_grad=args[into])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("tx", [BF16, FP16, FP32])
@pytest.mark.parametrize("ty", [BF16, FP16, FP32])
@pytest.mark.parametrize("dim", [8200, 9001, 10752, 10756, 12288])
def test_the_widest_rows_on_chip(tx, ty, dim):
    x, dy = randn((310, dim), tx, 1, 2.0, 0.5), randn((310, dim), ty, 2)
    weight, bias = randn((dim,), tx, 3, 0.3, 1.0), randn((dim,), tx, 4)
    both(x, weight, bias, dy, out_dtype=ty)
