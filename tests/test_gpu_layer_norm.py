"""Layer norm and its backward pass on the GPU against 64-bit forms.

Tolerances.  u = 2^-24 is half a step of fp32, r that of the stored type, h half
its smallest subnormal.  A row's sum runs through chains of at most L = 72 +
dim / 256 additions, so it is off by at most L u times the sum of magnitudes.
- mean: dm = L u mean|x| + u |mean|;
- var: the differences x - mean sum to zero, so an error of the mean enters
  squared: dv = dm^2 + (L + 4) u var; rstd is off by dv / 2 (var + eps) + 3 u of
  itself (sum, root and quotient round once each);
- y: the difference is off by dm + u |x - mean|; two products and a sum follow;
- backwards, from given stats: xhat is off by 2 u of itself, g = dy weight by u;
  the two means by (L + 5) u of their magnitudes; then dx as it is written;
- sums over n rows in any order: (n + 5) u of the sum of magnitudes.
Each carries a factor 1.01 for second-order terms and ends with r |result| + h.
"""
import math

import pytest
import torch

import optimizer_step_gb300 as og

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
ROUND = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24}
HALF_SUB = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -150}
U = 2.0 ** -24


def randn(shape, dtype, seed, std=1.0, mean=0.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std + mean).to(dtype)


def chain(dim):
    return 72 + dim / 256


def near(got, ref, tol, what):
    tol = 1.01 * (tol + ROUND[got.dtype] * ref.abs()) + HALF_SUB[got.dtype]
    off = (got.double() - ref).abs()
    assert got.shape == ref.shape, what
    assert bool((off <= tol).all()), (what, float((off / tol).nan_to_num(nan=math.inf).max()))


def check_forward(x, weight, bias, eps, y, stats=None):
    d, x = x.shape[-1], x.reshape(-1, x.shape[-1]).double()
    w = torch.ones(d, device="cuda").double() if weight is None else weight.double()
    b = torch.zeros(d, device="cuda").double() if bias is None else bias.double()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    var = c.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    dm = chain(d) * U * x.abs().mean(1, keepdim=True) + U * mean.abs()
    dr = 0.5 * (dm.square() + (chain(d) + 4) * U * var) / (var + eps) + 3 * U
    xhat = c * rstd
    tol = w.abs() * (rstd * (dm + 2 * U * c.abs()) + xhat.abs() * (dr + 3 * U)) \
        + U * (xhat * w).abs() + U * b.abs()
    near(y.reshape(-1, d), xhat * w + b, tol, "y")
    if stats is not None:
        stats = stats.reshape(2, -1, 1)
        near(stats[0], mean, dm, "mean")
        near(stats[1], rstd, dr * rstd, "rstd")


def check_backward(dy, x, weight, stats, got, old=(None, None)):
    d = x.shape[-1]
    x, dy = x.reshape(-1, d).double(), dy.reshape(-1, d).double()
    n = x.shape[0]
    w = torch.ones(d, device="cuda").double() if weight is None else weight.double()
    mean, rstd = stats.reshape(2, -1, 1).double()
    xhat = (x - mean) * rstd
    g = dy * w
    a, b = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    da = (chain(d) + 5) * U * g.abs().mean(1, keepdim=True)
    db = (chain(d) + 5) * U * (g * xhat).abs().mean(1, keepdim=True)
    dx, dw, dbias = got
    if dx is not None:
        tol = rstd * (da + xhat.abs() * db
                      + 5 * U * (g.abs() + a.abs() + (xhat * b).abs()))
        near(dx.reshape(-1, d), rstd * (g - a - xhat * b), tol, "dx")
    for out, terms, was, what in ((dw, dy * xhat, old[0], "dweight"), (dbias, dy, old[1], "dbias")):
        if out is not None:
            was = torch.zeros(d, device="cuda").double() if was is None else was.double()
            tol = (n + 5) * U * (terms.abs().sum(0) + was.abs())
            near(out, was + terms.sum(0), tol, what)


def both(x, weight, bias, dy, eps=1e-5, out_dtype=None, **how):
    y, stats = og.layer_norm(x, weight, bias, eps=eps, stats=True, out_dtype=out_dtype)
    check_forward(x, weight, bias, eps, y, stats)
    got = og.layer_norm_grad(dy, x, weight, stats, **how)
    check_backward(dy, x, weight, stats, got)
    return y, stats, got


WIDTHS = [1, 2, 3, 7, 8, 31, 33, 64, 96, 100, 128, 255, 256, 257, 512, 513, 768, 1000, 1023, 1024,
          1025, 1536, 2047, 2048, 2056, 4095, 4096, 4100, 5000, 8191, 8192, 12288, 12289, 16384,
          20000, 24576, 32768, 33000, 40001]


@pytest.mark.parametrize("dim", WIDTHS)
@pytest.mark.parametrize("tx,ty", [(BF16, BF16), (FP32, FP32)])
def test_widths(dim, tx, ty):
    n = 37 if dim > 300 else 301
    x = randn((n, dim), tx, dim, 2.0, 0.5)
    weight, bias = randn((dim,), tx, 1, 0.3, 1.0), randn((dim,), tx, 2)
    both(x, weight, bias, randn((n, dim), ty, 3), out_dtype=ty)


@pytest.mark.parametrize("tx", [BF16, FP16, FP32])
@pytest.mark.parametrize("ty", [BF16, FP16, FP32])
@pytest.mark.parametrize("tp", [BF16, FP16, FP32])
@pytest.mark.parametrize("dim", [40, 33, 640, 2048, 2046])
def test_types(tx, ty, tp, dim):
    x = randn((50, dim), tx, 5)
    weight, bias = randn((dim,), tp, 1, 0.3, 1.0), randn((dim,), tp, 2)
    dy = randn((50, dim), ty, 3)
    y, stats, got = both(x, weight, bias, dy, out_dtype=ty)
    assert y.dtype == ty and [t.dtype for t in got] == [tx, tp, tp]
    got = og.layer_norm_grad(dy, x, weight, stats, param_dtype=FP32)
    assert got[1].dtype == FP32
    check_backward(dy, x, weight, stats, got)


@pytest.mark.parametrize("n", [0, 1, 2, 31, 257, 4099, 20011])
@pytest.mark.parametrize("dim", [8, 65, 256, 1024, 2049])
def test_rows(n, dim):
    x, dy = randn((n, dim), BF16, n), randn((n, dim), BF16, n + 1)
    weight, bias = randn((dim,), FP32, 1, 0.3, 1.0), randn((dim,), FP32, 2)
    both(x, weight, bias, dy)


def test_many_short_rows():
    x, dy = randn((300_007, 16), BF16, 1), randn((300_007, 16), BF16, 2)
    both(x, None, None, dy)


@pytest.mark.parametrize("dim", [64, 1023, 4096, 40001])
def test_without_parameters_or_with_one(dim):
    x, dy = randn((3, 20, dim), BF16, 1), randn((3, 20, dim), BF16, 2)
    weight, bias = randn((dim,), BF16, 3), randn((dim,), BF16, 4)
    y, stats, got = both(x, None, None, dy)
    assert y.shape == x.shape and stats.shape == (2, 3, 20) and got[1].dtype == FP32
    both(x, weight, None, dy)
    both(x, None, bias, dy)


@pytest.mark.parametrize("dim", [48, 1000, 4096, 40001])
def test_each_gradient_alone(dim):
    x, dy, weight = randn((70, dim), BF16, 1), randn((70, dim), BF16, 2), randn((dim,), BF16, 3)
    _, stats = og.layer_norm(x, weight, stats=True)
    whole = og.layer_norm_grad(dy, x, weight, stats)
    for k in range(3):
        ask = [i == k for i in range(3)]
        got = og.layer_norm_grad(dy, x, weight, stats, x_grad=ask[0], weight_grad=ask[1],
                                 bias_grad=ask[2])
        assert [t is not None for t in got] == ask
        check_backward(dy, x, weight, stats, got)
        assert torch.equal(got[k], whole[k])
    assert og.layer_norm_grad(dy, x, weight, stats, x_grad=False, weight_grad=False,
                              bias_grad=False) == (None, None, None)


@pytest.mark.parametrize("n", [0, 5, 3000])
@pytest.mark.parametrize("dim", [24, 1023, 4096, 40001])
@pytest.mark.parametrize("tp", [BF16, FP32])
def test_accumulate(n, dim, tp):
    n = min(n, 300) if dim > 5000 else n
    x, dy = randn((n, dim), FP16, 1), randn((n, dim), FP16, 2)
    weight = randn((dim,), tp, 3)
    _, stats = og.layer_norm(x, weight, stats=True)
    old = randn((dim,), tp, 4), randn((dim,), tp, 5)
    sums = old[0].clone(), old[1].clone()
    got = og.layer_norm_grad(dy, x, weight, stats, weight_grad=sums[0], bias_grad=sums[1],
                             accumulate=True)
    assert got[1] is sums[0] and got[2] is sums[1]
    check_backward(dy, x, weight, stats, got, old)
    if n == 0:
        assert torch.equal(sums[0], old[0])
    # Without it, what was there is not read.
    junk = torch.full((dim,), float("nan"), dtype=tp, device="cuda")
    got = og.layer_norm_grad(dy, x, weight, stats, weight_grad=junk, bias_grad=False)
    check_backward(dy, x, weight, stats, got)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("dim,stride,shift", [(64, 64, 1), (64, 72, 0), (64, 67, 3), (33, 40, 1),
                                              (1000, 1001, 0), (1024, 1028, 4), (2048, 2050, 2),
                                              (4096, 4104, 8), (9000, 9001, 0), (36000, 36001, 5)])
def test_strides_and_alignment_leave_the_gaps_alone(dtype, dim, stride, shift):
    rows = 41

    def spread(values):
        store = torch.full((rows * stride + shift + 64,), 7.0, dtype=dtype, device="cuda")
        view = store[shift:shift + rows * stride].view(rows, stride)[:, :dim]
        if values is not None:
            view.copy_(values)
        return store, view

    def gaps_hold(store):
        back = store.clone()
        back[shift:shift + rows * stride].view(rows, stride)[:, :dim] = 7.0
        assert bool((back == 7.0).all())

    x, dy = randn((rows, dim), dtype, 1), randn((rows, dim), dtype, 2)
    pstore = randn((2 * dim + shift,), dtype, 3)
    weight, bias = pstore[shift:shift + dim], pstore[shift + dim:]
    (_, xs), (_, dys), (ystore, ys), (dxstore, dxs) = (spread(v) for v in (x, dy, None, None))
    y, stats = og.layer_norm(xs, weight, bias, stats=True, out=ys)
    assert y is ys
    check_forward(x, weight, bias, 1e-5, ys, stats)
    gaps_hold(ystore)
    sums = torch.full((2 * dim + shift + 9,), 7.0, dtype=dtype, device="cuda")
    dw, db = sums[shift:shift + dim], sums[shift + dim:shift + 2 * dim]
    got = og.layer_norm_grad(dys, xs, weight, stats, x_grad=dxs, weight_grad=dw, bias_grad=db)
    check_backward(dy, x, weight, stats, got)
    gaps_hold(dxstore)
    assert bool((sums[:shift] == 7.0).all()) and bool((sums[shift + 2 * dim:] == 7.0).all())


@pytest.mark.parametrize("dim", [16, 100, 1024, 4096, 12289, 40001])
def test_in_place(dim):
    x, dy = randn((65, dim), BF16, 1), randn((65, dim), BF16, 2)
    weight, bias = randn((dim,), BF16, 3), randn((dim,), BF16, 4)
    y, stats = og.layer_norm(x, weight, bias, stats=True)
    z = x.clone()
    assert torch.equal(og.layer_norm(z, weight, bias, out=z), y) and torch.equal(z, y)
    want = og.layer_norm_grad(dy, x, weight, stats)
    for into in (0, 1):
        args = [dy.clone(), x.clone()]
        got = og.layer_norm_grad(args[0], args[1], weight, stats, x_grad=args[into])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dim", [24, 33, 100, 250, 1023, 2048, 12288, 40001])
@pytest.mark.parametrize("dtype,mean,std", [
    (FP32, 1000.0, 1.0), (FP32, -3e4, 0.1), (BF16, 100.0, 3.0), (FP32, 0.0, 1e-6),
    (FP32, 0.0, 1e19), (FP32, 1e30, 1e25), (BF16, 0.0, 2e37), (FP32, 4e37, 1e37), (FP16, 0, 1e4)])
def test_rows_far_from_zero_large_and_small(dim, dtype, mean, std):
    x = randn((40, dim), FP32, 5).clamp(-4, 4).mul(std).add(mean).to(dtype)
    for eps in (1e-5, 1e-12):
        y, stats = og.layer_norm(x, stats=True, eps=eps, out_dtype=FP32)
        check_forward(x, None, None, eps, y, stats)


@pytest.mark.parametrize("dim", [24, 33, 100, 250, 1023, 2048, 12288, 40001])
def test_small_rows_without_eps(dim):
    """Squares below fp32's range count where no eps covers them."""
    x = randn((40, dim), FP32, 5).mul(1e-30)
    y, stats = og.layer_norm(x, stats=True, eps=0.0)
    check_forward(x, None, None, 0.0, y, stats)
    x = randn((40, dim), FP32, 5).mul(1e-24)
    y, stats = og.layer_norm(x, stats=True, eps=1e-46)
    check_forward(x, None, None, float(torch.tensor(1e-46, dtype=FP32)), y, stats)


@pytest.mark.parametrize("dim", [24, 1000, 2048, 12289, 40001])
def test_equal_elements(dim):
    x = torch.full((5, dim), 2.5, device="cuda")
    bias = randn((dim,), FP32, 1)
    y, stats = og.layer_norm(x, None, bias, stats=True)
    assert torch.equal(y, bias.expand(5, dim)) and bool((stats[0] == 2.5).all())
    assert bool(og.layer_norm(x, eps=0.0).isnan().all())


@pytest.mark.parametrize("dim", [24, 1000, 2048, 12289, 40001])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_inf_and_nan_stay_in_their_rows(dim, bad):
    x, dy = randn((9, dim), BF16, 1), randn((9, dim), BF16, 2)
    x[4, dim // 2] = bad
    y, stats = og.layer_norm(x, stats=True)
    keep = torch.arange(9, device="cuda") != 4
    assert bool(y[4].isnan().all()) and bool(stats[1, 4].isnan())
    check_forward(x[keep], None, None, 1e-5, y[keep], stats[:, keep])
    dx, dw, db = og.layer_norm_grad(dy, x, None, stats)
    assert bool(dx[4].isnan().all()) and bool(dw.isnan().all())
    check_backward(dy[keep], x[keep], None, stats[:, keep].contiguous(), (dx[keep], None, None))
    check_backward(dy, x, None, torch.zeros_like(stats), (None, None, db))


@pytest.mark.parametrize("dim", [24, 33, 1023, 4096])
@pytest.mark.parametrize("scale", [1e30, 1e-25])
def test_scaled_rows_among_others(dim, scale):
    """One row in three leaves fp32's squares; its neighbours keep their bits."""
    x = randn((50, dim), FP32, 5)
    plain, _ = og.layer_norm(x, stats=True, eps=1e-30)
    x[::3] *= scale
    y, stats = og.layer_norm(x, stats=True, eps=1e-30)
    check_forward(x, None, None, 1e-30, y, stats)
    keep = torch.arange(50, device="cuda") % 3 != 0
    assert torch.equal(y[keep], plain[keep])


@pytest.mark.parametrize("dim", [24, 33, 1023, 4096, 12288])
@pytest.mark.parametrize("scale", [1e30, 1e-20])
def test_backward_of_large_and_small_rows(dim, scale):
    x, dy = randn((40, dim), FP32, 1).mul(scale), randn((40, dim), FP32, 2)
    _, stats = og.layer_norm(x, stats=True, eps=1e-44)
    got = og.layer_norm_grad(dy, x, None, stats)
    check_backward(dy, x, None, stats, got)


@pytest.mark.parametrize("n", [1, 3, 17, 500, 2000])
@pytest.mark.parametrize("dim,pad", [(1000, 1), (300, 3), (4096, 5), (130, 3), (20, 1), (9000, 2)])
def test_rows_apart_in_each_tensor(n, dim, pad):
    """x, grad_out and x_grad begin differently from row to row."""
    x, dy = randn((n, dim + pad), BF16, 1)[:, :dim], randn((n, dim), BF16, 2)
    weight = randn((dim,), FP32, 3)
    y, stats = og.layer_norm(x, weight, stats=True, out_dtype=FP32)
    check_forward(x, weight, None, 1e-5, y, stats)
    check_backward(dy, x, weight, stats, og.layer_norm_grad(dy, x, weight, stats))
    dx = torch.empty((n, dim + pad), dtype=BF16, device="cuda")[:, :dim]
    both = og.layer_norm_grad(torch.cat([dy, dy], 1)[:, dim:], x, weight, stats, x_grad=dx)
    check_backward(dy, x, weight, stats, both)


@pytest.mark.parametrize("n,dim", [(512, 256), (3000, 1023), (1000, 4096), (90, 40001)])
def test_the_same_bits_every_time(n, dim):
    x, dy, weight = randn((n, dim), BF16, 1), randn((n, dim), BF16, 2), randn((dim,), BF16, 3)
    _, stats = og.layer_norm(x, weight, stats=True)
    first = og.layer_norm_grad(dy, x, weight, stats, param_dtype=FP32)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(
            first, og.layer_norm_grad(dy, x, weight, stats, param_dtype=FP32)))


def test_offsets_past_32_bits():
    n, dim = 600_000, 8192
    x = torch.zeros((n, dim), dtype=BF16, device="cuda")
    rows = torch.tensor([0, 1, n // 2, n - 2, n - 1], device="cuda")
    x[rows] = randn((5, dim), BF16, 1)
    y, stats = og.layer_norm(x, stats=True)
    check_forward(x[rows], None, None, 1e-5, y[rows], stats[:, rows])
    del y
    dy = torch.zeros_like(x)
    dy[rows] = randn((5, dim), BF16, 2)
    got = og.layer_norm_grad(dy, x, None, stats, x_grad=dy.new_empty(0).set_(dy))
    check = [got[0][rows].clone(), got[1], got[2]]
    dy[rows] = randn((5, dim), BF16, 2)
    check_backward(dy[rows], x[rows], None, stats[:, rows].contiguous(), check)


# ------------------------------------------------------------------- autograd
def test_autograd_gives_the_formulas():
    x, dy = randn((4, 9, 200), BF16, 1).requires_grad_(), randn((4, 9, 200), FP32, 2)
    weight, bias = (randn((200,), FP32, s).requires_grad_() for s in (3, 4))
    y, stats = og.layer_norm(x, weight, bias, stats=True, out_dtype=FP32)
    assert y.requires_grad and not stats.requires_grad
    check_forward(x.detach(), weight.detach(), bias.detach(), 1e-5, y.detach(), stats)
    y.backward(dy)
    assert x.grad.dtype == BF16 and weight.grad.dtype == FP32
    check_backward(dy, x.detach(), weight.detach(), stats, (x.grad, weight.grad, bias.grad))


@pytest.mark.parametrize("need", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)])
def test_autograd_of_some(need):
    x, weight, bias = (randn(s, BF16, k) for k, s in enumerate([(30, 72), (72,), (72,)]))
    for t, want in zip((x, weight, bias), need):
        t.requires_grad_(bool(want))
    og.layer_norm(x, weight, bias).sum().backward()   # one number for all rows
    _, stats = og.layer_norm(x.detach(), weight.detach(), stats=True)
    assert [t.grad is not None for t in (x, weight, bias)] == [bool(k) for k in need]
    check_backward(torch.ones(30, 72, device="cuda"), x.detach(), weight.detach(), stats,
                   (x.grad, weight.grad, bias.grad))


def test_autograd_of_a_transposed_gradient():
    x = randn((5, 6, 40), FP32, 1).requires_grad_()
    w = randn((6, 40, 5), FP32, 2)
    (og.layer_norm(x).permute(1, 2, 0) * w).sum().backward()
    _, stats = og.layer_norm(x.detach(), stats=True)
    check_backward(w.permute(2, 0, 1).contiguous(), x.detach(), None, stats, (x.grad, None, None))


def test_gradients_match_differences():
    """Central differences in 64 bits of the plain form; fp32 arithmetic and the
    third derivative, with steps of 2^-10, stay below 1e-4 here."""
    x, weight, bias = (randn(s, FP32, k + 1) for k, s in enumerate([(3, 12), (12,), (12,)]))
    dy = randn((3, 12), FP32, 9)
    leaves = [t.clone().requires_grad_() for t in (x, weight, bias)]
    (og.layer_norm(*leaves) * dy).sum().backward()

    def loss(x, w, b):
        c = x - x.mean(1, keepdim=True)
        return float(((c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w + b) * dy).sum())

    args = [t.double() for t in (x, weight, bias)]
    for k, leaf in enumerate(leaves):
        for i in range(args[k].numel()):
            ends = []
            for sign in (1, -1):
                moved = [t.clone() for t in args]
                moved[k].view(-1)[i] += sign * 2.0 ** -10
                ends.append(loss(*moved))
            assert abs(float(leaf.grad.view(-1)[i]) - (ends[0] - ends[1]) * 2.0 ** 9) < 1e-4


def test_weights_used_twice_get_both_gradients():
    x = [randn((n, 64), FP32, n) for n in (20, 33)]
    weight = randn((64,), FP32, 3).requires_grad_()
    (og.layer_norm(x[0], weight).sum() + og.layer_norm(x[1], weight).sum()).backward()
    _, stats = og.layer_norm(torch.cat(x), stats=True)
    check_backward(torch.ones(53, 64, device="cuda"), torch.cat(x), weight.detach(), stats,
                   (None, weight.grad, None))


def test_refusals():
    x, weight = randn((6, 24), FP32, 1), randn((24,), FP32, 2)
    _, stats = og.layer_norm(x, stats=True)
    bad = [
        (TypeError, lambda: og.layer_norm(x.double())),
        (TypeError, lambda: og.layer_norm(x, out_dtype=torch.float64)),
        (TypeError, lambda: og.layer_norm(x, weight, weight.to(BF16))),
        (ValueError, lambda: og.layer_norm(x, weight[:-1])),
        (ValueError, lambda: og.layer_norm(x, torch.ones(48, device="cuda")[::2])),
        (ValueError, lambda: og.layer_norm(x, weight.cpu())),
        (ValueError, lambda: og.layer_norm(x.t())),
        (ValueError, lambda: og.layer_norm(x[:, :0])),
        (TypeError, lambda: og.layer_norm(x[0, 0])),
        (ValueError, lambda: og.layer_norm(x, out=x[:3])),
        (ValueError, lambda: og.layer_norm(x, out=torch.empty(6, 24, device="cuda"),
                                           out_dtype=BF16)),
        (og.LambError, lambda: og.layer_norm(x, eps=-1.0)),
        (og.LambError, lambda: og.layer_norm(x, eps=math.nan)),
        (ValueError, lambda: og.layer_norm_grad(x[:3], x, weight, stats)),
        (ValueError, lambda: og.layer_norm_grad(x, x, weight, stats[:, :3])),
        (ValueError, lambda: og.layer_norm_grad(x, x, weight, stats.to(BF16))),
        (TypeError, lambda: og.layer_norm_grad(x, x, weight, stats, x_grad=x.to(BF16))),
        (TypeError, lambda: og.layer_norm_grad(x, x, weight, stats, weight_grad=weight.clone(),
                                               bias_grad=weight.to(BF16))),
        (ValueError, lambda: og.layer_norm_grad(x, x, weight, stats, accumulate=True)),
        (RuntimeError, lambda: og.layer_norm(x.clone().requires_grad_(), out=torch.empty_like(x))),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    leaf = x.clone().requires_grad_()
    with pytest.raises(RuntimeError):   # once only
        first, = torch.autograd.grad(og.layer_norm(leaf).square().sum(), leaf, create_graph=True)
        torch.autograd.grad(first.sum(), leaf)
    moved = x.clone()
    y = og.layer_norm(moved, weight.requires_grad_())
    moved.add_(1.0)
    with pytest.raises(RuntimeError):   # x changed since
        y.sum().backward()


# ----------------------------------------------------------- streams and graphs
def test_another_stream_and_a_captured_graph():
    n, dim = 300, 1024
    weight = randn((dim,), BF16, 3)
    x, dy = torch.zeros(n, dim, dtype=BF16, device="cuda"), torch.zeros(n, dim, dtype=BF16,
                                                                          device="cuda")

    def calls():
        y, stats = og.layer_norm(x, weight, stats=True)
        return (y, stats, *og.layer_norm_grad(dy, x, weight, stats, param_dtype=FP32))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = calls()
        graphs.append((graph, outs))
    for k in range(4):
        x.copy_(randn((n, dim), BF16, k))
        dy.copy_(randn((n, dim), BF16, k + 50))
        graph, (y, stats, *grads) = graphs[k % 2]
        graph.replay()
        check_forward(x, weight, None, 1e-5, y, stats)
        check_backward(dy, x, weight, stats, grads)


def test_calls_on_several_streams_at_once():
    cases = [(randn((700, 512), BF16, k), randn((700, 512), BF16, k + 9)) for k in range(4)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for stream, (x, dy) in zip(streams, cases):
            with torch.cuda.stream(stream):
                _, stats = og.layer_norm(x, stats=True)
                got.append((dy, x, stats, og.layer_norm_grad(dy, x, None, stats)))
    torch.cuda.synchronize()
    for dy, x, stats, grads in got:
        check_backward(dy, x, None, stats, grads)
