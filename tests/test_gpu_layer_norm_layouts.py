"""Layer norm and its backward pass in place of rows that are copied ahead, and the
widest rows on chip in each pair of types."""
import pytest
import torch

import optimizer_step_gb300 as og
from test_gpu_layer_norm import BF16, FP16, FP32, both, check_backward, randn

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


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,dim", [(4096, 1), (4097, 1), (4096, 9), (4097, 9), (14000, 9),
                                   (26214, 5), (4096, 32), (4097, 32), (8192, 8), (16384, 8),
                                   (3971, 33), (128, 1024), (129, 1024), (512, 256), (513, 256),
                                   (127, 1025), (3, 1025)])
def test_sizes_next_to_those_that_one_cluster_takes(n, dim, dtype):
    x, dy = randn((n, dim), dtype, 1, 2.0, 0.5), randn((n, dim), dtype, 2)
    weight, bias = randn((dim,), dtype, 3, 0.3, 1.0), randn((dim,), dtype, 4)
    both(x, weight, bias, dy)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 7, 15, 16, 17, 33])
@pytest.mark.parametrize("dim,pad", [(8, 0), (9, 0), (64, 0), (255, 0), (257, 0), (300, 3),
                                     (1000, 1), (1023, 0), (1024, 0), (1024, 1)])
def test_fewer_rows_than_a_cluster_has_ctas(n, dim, pad, dtype):
    x, dy = (randn((n, dim + pad), dtype, k)[:, :dim] for k in (1, 2))
    weight = randn((dim,), dtype, 3, 0.3, 1.0)
    alike = torch.empty_strided(x.shape, x.stride(), dtype=dtype, device="cuda")
    y, stats = og.layer_norm(x, weight, stats=True)
    for into in (True, alike):
        old = [randn((dim,), FP32, k) for k in (5, 6)]
        sums = [t.clone() for t in old]
        got = og.layer_norm_grad(dy, x, weight, stats, x_grad=into, weight_grad=sums[0],
                                 bias_grad=sums[1], accumulate=True)
        check_backward(dy, x, weight, stats, got, old)
