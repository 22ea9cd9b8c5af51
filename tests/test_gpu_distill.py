"""The loss against a teacher's top logits and true labels, and its gradient, on
the GPU against 64-bit forms.

Tolerances.  u = 2^-24 is half a step of fp32, r that of the stored type, h half
its smallest subnormal.  With d = z - max z (off by u |d|):
- an exponent d / T is off by 4 u |d| / T (difference, two constants, product)
  and the exponential by 4 u of itself, so a term e of a sum S is off by
  (4 |d| / T + 4) u, and S, through chains of at most L = 72 + vocab / 256
  additions, by E = u (sum of e (4 |d| / T + 4) / S + L) of itself;
- q = e / S by (4 |d| / T + 6) u + E of itself; log S by E + 2 u |log S| + u;
  log q by 3 u |d| / T more; the same for the teacher's p and log p;
- a term p (log p - log q) by what its factors are off by and 4 u of the sizes
  that it is put together from; the sum of top_k of them by 72 u of magnitudes;
- the gradient by what q, s and p are off by and 8 u of the magnitudes;
- an exponential below f = 2^-126, fp32's smallest normal number, may become 0 or
  lose bits: it is off by f at most, and as S is at least 1, so are q, s and p.
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
CHAIN = 72
TINY = 2.0 ** -126


class Data:
    """Rows of student and teacher; ids distinct within a row."""

    def __init__(self, n, vocab, top, dtype=BF16, teacher=None, id_type=torch.int64, seed=0,
                 std=2.0, labels=True):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed + n + 7 * vocab + 31 * top)
        rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.logits = (std * rand(n, vocab)).to(dtype)
        start = torch.randint(vocab, (n, 1), generator=gen, device="cuda")
        self.ids = ((start + torch.arange(top, device="cuda") * max(1, vocab // max(1, top)))
                    % vocab).to(id_type)
        self.teacher = (2.0 * rand(n, top)).to(teacher or dtype)
        self.labels = (torch.randint(vocab, (n,), generator=gen, device="cuda").to(id_type)
                       if labels else None)
        self.row_grad = rand(n).abs() + 0.1

    def args(self):
        return self.logits, self.ids, self.teacher, self.labels


def softmax(z, valid, temperature):
    """(probabilities, their relative error, log, its error) where valid."""
    z = torch.where(valid, z.double(), -math.inf)
    top = z.max(1, keepdim=True).values
    d = torch.where(valid & (z > -math.inf), (z - top) / temperature, 0.0)
    live = valid & (z > -math.inf)
    e = torch.where(live, d.exp(), 0.0)
    size = e.sum(1, keepdim=True)
    chain = CHAIN + z.shape[1] / 256
    off = U * ((e * (4 * d.abs() + 4)).sum(1, keepdim=True) / size + chain)
    log = torch.where(live, d - size.log(), -math.inf)
    log_off = 3 * U * d.abs() + off + 2 * U * size.log().abs() + U
    return e / size, U * (4 * d.abs() + 6) + off, log, log_off


def reference(data, temperature, soft, hard, ignore=-100, row_grad=None, scale=1.0):
    """(loss, its tolerance, gradient, its tolerance) in 64 bits."""
    z, T = data.logits.double(), temperature
    n, vocab = z.shape
    zero = torch.zeros(n, dtype=torch.float64, device="cuda")
    loss, loss_tol, grad, grad_tol = zero, zero, torch.zeros_like(z), torch.zeros_like(z)
    live = torch.ones(n, dtype=torch.bool, device="cuda")
    if data.labels is not None:
        labels = data.labels.long()
        live = (labels != ignore) & (labels >= 0) & (labels < vocab)
    up = scale * (torch.ones_like(zero) if row_grad is None else row_grad.double())
    up = torch.where(live, up, 0.0)[:, None]
    every = torch.ones_like(z, dtype=torch.bool)
    if soft and data.ids is not None and data.ids.shape[1]:
        ids, t = data.ids.long(), data.teacher.double()
        valid = (ids >= 0) & (ids < vocab) & (t != -math.inf) & live[:, None]
        some = valid.any(1)
        ids = torch.where(valid, ids, 0)
        p, p_off, log_p, log_p_off = softmax(torch.where(valid, t, 0.0), valid, T)
        q, q_off, log_q, log_q_off = softmax(z, every, T)
        at_q, at_off = log_q.gather(1, ids), log_q_off.gather(1, ids)
        p, log_p = torch.where(valid, p, 0.0), torch.where(valid, log_p, 0.0)
        terms = torch.where(valid, p * (log_p - at_q), 0.0)
        size = p * (log_p.abs() + at_q.abs())
        off = p * (log_p_off + at_off) + size * p_off + 4 * U * size \
            + TINY * torch.where(valid, log_p - at_q, 0.0).abs()
        off = torch.where(valid, off + CHAIN * U * terms.abs(), 0.0).sum(1)
        c = soft * T * T
        loss = loss + torch.where(some, c * terms.sum(1), 0.0)
        loss_tol = loss_tol + torch.where(some, abs(c) * off, 0.0) + 6 * U * loss.abs()
        c = soft * T
        q = torch.where(some[:, None], q, 0.0)
        grad = grad + c * q.scatter_add(1, ids, -p)
        mine = (q * (q_off + 8 * U) + TINY).scatter_add(
            1, ids, torch.where(valid, p * (p_off + (8 + CHAIN) * U) + TINY, 0.0))
        grad_tol = grad_tol + abs(c) * mine
    if hard:
        labels = torch.where(live, labels, 0)[:, None]
        s, s_off, log_s, log_s_off = softmax(z, every, 1.0)
        mine = -hard * log_s.gather(1, labels)[:, 0]
        loss = loss + torch.where(live, mine, 0.0)
        loss_tol = loss_tol + torch.where(
            live, abs(hard) * log_s_off.gather(1, labels)[:, 0] + 6 * U * mine.abs(), 0.0)
        one = torch.full_like(labels, -1.0, dtype=torch.float64)
        grad = grad + hard * s.scatter_add(1, labels, one)
        grad_tol = grad_tol + abs(hard) * (s * (s_off + 8 * U) + TINY).scatter_add(1, labels,
                                                                            -8 * U * one)
    loss = torch.where(live, loss, 0.0)
    grad = torch.where(up != 0, up * grad, 0.0)
    grad_tol = torch.where(up != 0, up.abs() * grad_tol, 0.0)
    return loss, loss_tol, grad, grad_tol


def near(got, ref, tol, what):
    tol = 1.01 * (tol + ROUND[got.dtype] * ref.abs()) + HALF_SUB[got.dtype]
    off = torch.where(got.double() == ref, 0.0, (got.double() - ref).abs())
    assert got.shape == ref.shape, what
    assert bool((off <= tol).all()), (what, float((off / tol).nan_to_num(nan=math.inf).max()))


def check(data, temperature=1.0, soft=1.0, hard=0.0, ignore=-100, row_grad=None, scale=1.0,
          dtype=None, out=None):
    how = dict(temperature=temperature, soft_weight=soft, hard_weight=hard, ignore_id=ignore)
    loss, loss_tol, grad, grad_tol = reference(data, temperature, soft, hard, ignore, row_grad,
                                               scale)
    alone = og.distill_loss(*data.args(), **how)
    near(alone, loss, loss_tol, "loss alone")
    got = og.distill_loss_grad(*data.args(), row_grad=row_grad, scale=scale, dtype=dtype, out=out,
                               **how)
    near(got[0], loss, loss_tol, "loss")
    near(got[1], grad, grad_tol, "grad")
    return got


VOCABS = [1, 2, 3, 7, 8, 31, 32, 33, 100, 128, 255, 512, 1000, 1023, 1024, 2048, 2050, 4096, 5000,
          8192, 10007, 16384, 24580, 32000, 32768, 40001, 65536, 99991, 131071, 131072, 262144]


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_vocabularies(vocab, dtype):
    data = Data(13 if vocab > 2000 else 70, vocab, min(vocab, 20), dtype)
    check(data, 1.0, 1.0, 0.0)
    check(data, 2.0, 0.6, 0.4, row_grad=data.row_grad, scale=0.25)


@pytest.mark.parametrize("vocab", [500_000, 900_001, 1_300_000])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_very_wide_vocabularies(vocab, dtype):
    data = Data(3, vocab, 50, dtype)
    check(data, 1.5, 0.5, 0.5)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("out", [BF16, FP16, FP32])
@pytest.mark.parametrize("teacher", [BF16, FP16, FP32])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_types(dtype, out, teacher, id_type):
    for vocab in (1000, 4097, 32000):
        data = Data(17, vocab, 12, dtype, teacher, id_type)
        _, grad = check(data, 0.7, 0.8, 0.2, row_grad=data.row_grad, dtype=out)
        assert grad.dtype == out


@pytest.mark.parametrize("ids,labels", [(torch.int32, torch.int64), (torch.int64, torch.int32)])
def test_types_of_ids_and_labels(ids, labels):
    data = Data(40, 3000, 12, BF16, FP32, ids)
    data.labels = data.labels.to(labels)
    data.labels[::5] = -7
    check(data, 2.0, 0.5, 0.5, ignore=-7, row_grad=data.row_grad)


@pytest.mark.parametrize("scale", [0.0, -2.0, 1024.0, 1e-30])
def test_scales(scale):
    check(Data(40, 3000, 12, FP32), 2.0, 0.5, 0.5, scale=scale)


def test_more_rows_than_are_held_at_once_with_some_left_out():
    """Each CTA walks through many rows; those left out come anywhere between."""
    for vocab in (64, 1001, 40000):
        n = 9000 if vocab < 2000 else 1500
        data = Data(n, vocab, 3)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(1)
        data.labels[torch.rand(n, generator=gen, device="cuda") < 0.5] = -100
        data.row_grad[torch.rand(n, generator=gen, device="cuda") < 0.3] = 0.0
        data.ids[torch.rand(n, generator=gen, device="cuda") < 0.3] = -1
        check(data, 2.0, 0.5, 0.5, row_grad=data.row_grad)
        check(data, 2.0, 1.0, 0.0, row_grad=data.row_grad)


@pytest.mark.parametrize("n", [0, 1, 2, 150, 153, 1000, 5003])
@pytest.mark.parametrize("vocab", [40, 513, 3000])
def test_rows(n, vocab):
    check(Data(n, vocab, 5), 2.0, 0.5, 0.5)


@pytest.mark.parametrize("n,vocab", [(1, 32000), (64, 32000), (400, 32000), (700, 12001),
                                     (310, 131071)])
def test_rows_wide(n, vocab):
    check(Data(n, vocab, 33), 2.0, 0.5, 0.5)


@pytest.mark.parametrize("top", [0, 1, 2, 31, 32, 33, 64, 127, 256, 257, 1000, 1024])
def test_entries(top):
    data = Data(21, 3001, top)
    check(data, 1.3, 1.0, 0.0)
    check(data, 1.3, 0.5, 0.5)


@pytest.mark.parametrize("soft,hard", [(1.0, 0.0), (0.0, 1.0), (0.3, 0.7), (-0.5, 2.0), (0, 0)])
@pytest.mark.parametrize("temperature", [0.05, 0.7, 1.0, 2.0, 20.0])
@pytest.mark.parametrize("vocab", [100, 8192])
def test_weights_and_temperatures(soft, hard, temperature, vocab):
    check(Data(40, vocab, 9, FP16), temperature, soft, hard)


@pytest.mark.parametrize("vocab", [50, 2048, 40000])
def test_labels_alone(vocab):
    data = Data(60, vocab, 1)
    data.ids = data.teacher = None
    loss, grad = check(data, 1.0, 1.0, 1.0)
    want = torch.nn.functional.cross_entropy(data.logits.double(), data.labels, reduction="none")
    assert float((loss - want).abs().max()) < 1e-4


@pytest.mark.parametrize("vocab", [50, 2048, 40000])
def test_a_teacher_alone(vocab):
    data = Data(60, vocab, 7, labels=False)
    check(data, 2.0, 1.0, 0.0)
    assert not og.distill_loss(data.logits, None, None).any()


@pytest.mark.parametrize("vocab", [60, 2001, 32000])
@pytest.mark.parametrize("hard", [0.0, 0.5])
def test_rows_left_out(vocab, hard):
    data = Data(64, vocab, 10)
    data.labels[::7] = -100
    data.labels[1::7] = vocab
    data.labels[2::7] = -5
    out = (data.labels < 0) | (data.labels >= vocab)
    check(data, 2.0, 1.0, hard)
    # Whatever they hold.
    data.logits[::7] = math.nan
    data.logits[1::7, 3] = math.inf
    data.logits[2::7] = -math.inf
    data.teacher[::7] = math.nan
    loss, grad = og.distill_loss_grad(*data.args(), hard_weight=hard)
    assert not loss[out].any() and not grad[out].any()
    assert bool(loss[~out].isfinite().all()) and bool(grad[~out].isfinite().all())
    # Another id that says so.
    data = Data(64, vocab, 10)
    data.labels[5] = data.labels[9]
    check(data, 1.0, 0.5, 0.5, ignore=int(data.labels[9]))


@pytest.mark.parametrize("vocab", [60, 2001, 32000])
def test_rows_whose_gradient_is_not_wanted(vocab):
    data = Data(50, vocab, 10)
    data.row_grad[::3] = 0.0
    check(data, 2.0, 0.5, 0.5, row_grad=data.row_grad)
    data.logits[::3] = math.nan
    loss, grad = og.distill_loss_grad(*data.args(), row_grad=data.row_grad)
    assert not grad[::3].any() and bool(loss[::3].isnan().all())
    assert bool(grad[1::3].isfinite().all())
    _, grad = og.distill_loss_grad(*data.args(), scale=0.0)
    assert not grad.any()


@pytest.mark.parametrize("vocab", [60, 2001, 32000])
def test_missing_entries(vocab):
    data = Data(64, vocab, 10)
    data.ids[::4, 3:] = -1
    data.ids[1::4] = -1                     # none at all
    data.ids[2::4, ::2] = vocab + 5
    data.teacher[3::4, 1:4] = -math.inf
    data.teacher[7, :] = -math.inf
    data.teacher[::4, 5] = math.nan         # its id is -1
    check(data, 2.0, 1.0, 0.0)
    check(data, 2.0, 0.5, 0.5, row_grad=data.row_grad)
    loss, grad = og.distill_loss_grad(data.logits, data.ids, data.teacher)
    assert not loss[1::4].any() and not grad[1::4].any() and not grad[7].any()


@pytest.mark.parametrize("top", [2, 40, 300])
@pytest.mark.parametrize("vocab", [500, 32000])
def test_a_token_named_again(vocab, top):
    data = Data(30, vocab, top)
    data.ids[:10, 1::2] = data.ids[:10, :1]
    data.ids[10:20] = data.ids[10:20, :1]
    data.labels[::2] = data.ids[::2, 0]
    check(data, 2.0, 0.5, 0.5)
    check(data, 1.0, 1.0, 0.0)


@pytest.mark.parametrize("top", [3, 40, 100, 256, 1000, 1024])
@pytest.mark.parametrize("n,vocab,range_", [(600, 700, 700), (400, 4100, 4100), (400, 4100, 90),
                                            (40, 131071, 131071), (40, 131071, 2000)])
def test_tokens_named_any_number_of_times(n, vocab, range_, top):
    data = Data(n, vocab, 0)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    data.ids = torch.randint(range_, (n, top), generator=gen, device="cuda")
    data.teacher = torch.randn(n, top, generator=gen, device="cuda")
    data.ids[torch.rand(n, top, generator=gen, device="cuda") < 0.05] = -1
    data.labels[::2] = data.ids[::2, top // 2]
    data.ids[3] = -1
    data.labels[3] = 8
    first = check(data, 2.0, 0.5, 0.5)
    check(data, 1.0, 1.0, 0.0)
    again = og.distill_loss_grad(*data.args(), temperature=2.0, soft_weight=0.5, hard_weight=0.5)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("vocab", [60, 2001, 32000])
def test_masked_logits(dtype, vocab):
    """Tokens masked with -inf and with the type's lowest value."""
    data = Data(40, vocab, 4, dtype)
    data.ids[:] = torch.arange(4, device="cuda")
    data.labels[:] = 5
    data.logits[:, 8::2] = -math.inf
    data.logits[:, 9::2] = torch.finfo(dtype).min
    loss, grad = check(data, 2.0, 0.5, 0.5)
    assert not grad[:, 8:].any()
    data.logits[3, 6:] = -math.inf
    data.logits[3, :5] = -math.inf
    data.logits[3, 5] = torch.finfo(dtype).min   # one token left
    loss, grad = og.distill_loss_grad(data.logits, None, None, data.labels, hard_weight=1.0)
    assert float(loss[3]) == 0.0 and not grad[3].any()
    # A masked token that is named: an infinite loss, a finite gradient.
    data.labels[4] = 8
    loss, grad = og.distill_loss_grad(data.logits, None, None, data.labels, hard_weight=1.0)
    assert float(loss[4]) == math.inf and bool(grad[4].isfinite().all())
    data.ids[6, 2] = 8
    loss, grad = og.distill_loss_grad(data.logits, data.ids, data.teacher)
    assert float(loss[6]) == math.inf and bool(grad[6].isfinite().all())


@pytest.mark.parametrize("vocab", [60, 2001, 32000])
@pytest.mark.parametrize("bad", [math.inf, math.nan, None])
def test_broken_rows_stay_alone(vocab, bad):
    data = Data(30, vocab, 6)
    if bad is None:
        data.logits[11] = -math.inf
    else:
        data.logits[11, vocab // 2] = bad
    for soft, hard in ((1.0, 0.0), (0.0, 1.0), (0.5, 0.5)):
        loss, grad = og.distill_loss_grad(*data.args(), soft_weight=soft, hard_weight=hard)
        assert bool(loss[11].isnan()) and bool(grad[11].isnan().all())
        keep = torch.arange(30, device="cuda") != 11
        assert bool(loss[keep].isfinite().all()) and bool(grad[keep].isfinite().all())
    data = Data(30, vocab, 6)
    data.teacher[5, 2] = math.nan if bad is None else bad
    loss, grad = og.distill_loss_grad(*data.args())
    assert bool(loss[5].isnan()) and bool(grad[5].isnan().any())
    assert bool(loss[6:].isfinite().all())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [64, 2000, 32000])
def test_large_logits(dtype, vocab):
    data = Data(20, vocab, 6, dtype, std=1e4)
    check(data, 1.0, 0.5, 0.5)
    data = Data(20, vocab, 6, dtype, std=1e30)
    check(data, 1.0, 0.5, 0.5)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab,stride,shift", [(64, 64, 1), (64, 72, 0), (64, 67, 3), (33, 40, 1),
                                                (1000, 1001, 0), (2048, 2056, 8), (4100, 4102, 2),
                                                (32000, 32064, 0), (32000, 32001, 5),
                                                (131071, 131072, 0), (131072, 131073, 3)])
def test_strides_and_alignment_leave_the_gaps_alone(dtype, vocab, stride, shift):
    rows = 19
    data = Data(rows, vocab, 12, dtype)
    stores = []
    for values in (data.logits, None):
        store = torch.full((rows * stride + shift + 64,), 7.0, dtype=dtype, device="cuda")
        view = store[shift:shift + rows * stride].view(rows, stride)[:, :vocab]
        if values is not None:
            view.copy_(values)
        stores.append((store, view))
    wide = torch.zeros(rows, 15, dtype=data.ids.dtype, device="cuda")
    wide[:, 2:14] = data.ids
    data.ids = wide[:, 2:14]
    wide = torch.zeros(rows, 17, dtype=dtype, device="cuda")
    wide[:, 1:13] = data.teacher
    data.teacher = wide[:, 1:13]
    data.logits = stores[0][1]
    check(data, 2.0, 0.5, 0.5, row_grad=data.row_grad, out=stores[1][1])
    store = stores[1][0]
    store[shift:shift + rows * stride].view(rows, stride)[:, :vocab] = 7.0
    assert bool((store == 7.0).all())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab", [33, 64, 2000, 12007, 32000, 131071, 262144, 700_001])
def test_in_place(dtype, vocab):
    data = Data(9, vocab, 12, dtype)
    data.ids[4, 3:] = data.ids[4, 2]
    how = dict(temperature=2.0, soft_weight=0.5, hard_weight=0.5, row_grad=data.row_grad)
    loss, grad = og.distill_loss_grad(*data.args(), **how)
    again, into = og.distill_loss_grad(*data.args(), out=data.logits, **how)
    assert into is data.logits and torch.equal(into, grad) and torch.equal(loss, again)


def test_leading_dimensions():
    data = Data(24, 300, 5)
    loss, grad = og.distill_loss_grad(*data.args())
    shaped = [t.view(2, 3, 4, *t.shape[1:]) for t in data.args()]
    got = og.distill_loss_grad(*shaped)
    assert torch.equal(got[0], loss.view(2, 3, 4)) and torch.equal(got[1].view(24, 300), grad)
    one = og.distill_loss(*(t[0] for t in data.args()))
    assert one.shape == () and torch.equal(one, loss[0])


@pytest.mark.parametrize("n,vocab", [(300, 700), (40, 32000), (8, 131071)])
def test_the_same_bits_every_time(n, vocab):
    data = Data(n, vocab, 30)
    data.ids[:, 20:] = data.ids[:, :10]
    first = og.distill_loss_grad(*data.args(), hard_weight=0.5, temperature=2.0)
    for _ in range(5):
        again = og.distill_loss_grad(*data.args(), hard_weight=0.5, temperature=2.0)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_offsets_past_32_bits():
    n, vocab = 80_000, 65536
    rows = torch.tensor([0, 1, n // 2, n - 2, n - 1], device="cuda")
    data = Data(5, vocab, 9)
    logits = torch.zeros((n, vocab), dtype=BF16, device="cuda")
    logits[rows] = data.logits
    ids = torch.full((n, 9), -1, device="cuda")
    ids[rows] = data.ids
    teacher = torch.zeros((n, 9), dtype=BF16, device="cuda")
    teacher[rows] = data.teacher
    labels = torch.full((n,), -100, device="cuda")
    labels[rows] = data.labels
    loss, grad = og.distill_loss_grad(logits, ids, teacher, labels, hard_weight=0.5, out=logits)
    want = reference(data, 1.0, 1.0, 0.5)
    near(loss[rows], *want[:2], "loss")
    near(grad[rows], *want[2:], "grad")


# ------------------------------------------------------------------- autograd
@pytest.mark.parametrize("vocab", [50, 3001, 32000])
def test_autograd_gives_the_formulas(vocab):
    data = Data(30, vocab, 8, FP32)
    how = dict(temperature=2.0, soft_weight=0.5, hard_weight=0.5)
    _, _, grad, tol = reference(data, 2.0, 0.5, 0.5, row_grad=data.row_grad)
    data.logits.requires_grad_()
    loss = og.distill_loss(*data.args(), **how)
    (loss * data.row_grad).sum().backward()
    near(data.logits.grad, grad, tol, "grad")
    data.logits.grad = None
    og.distill_loss(*data.args(), **how).sum().backward()   # one number for all rows
    _, _, grad, tol = reference(Detached(data), 2.0, 0.5, 0.5)
    near(data.logits.grad, grad, tol, "grad of a sum")


class Detached(Data):
    def __init__(self, data):
        self.__dict__.update(data.__dict__)
        self.logits = data.logits.detach()


def test_autograd_through_a_slice_of_the_logits():
    """A head wider than its vocabulary; the loss of one row in two."""
    data = Data(20, 128, 8, FP32)
    data.logits.requires_grad_()
    part = Detached(data)
    part.logits = data.logits[:, :100]
    part.ids, part.labels = data.ids % 100, data.labels % 100
    og.distill_loss(*part.args(), hard_weight=0.5)[::2].sum().backward()
    part.logits = part.logits.detach().contiguous()
    picked = torch.zeros(20, device="cuda")
    picked[::2] = 1.0
    _, _, grad, tol = reference(part, 1.0, 1.0, 0.5, row_grad=picked)
    near(data.logits.grad[:, :100].contiguous(), grad, tol, "grad")
    assert not data.logits.grad[:, 100:].any()


def test_gradients_match_differences():
    """Central differences in 64 bits of the plain form; fp32 arithmetic and the
    third derivative, with steps of 2^-10, stay below 1e-5 here."""
    data = Data(4, 11, 5, FP32)
    data.ids[1, 2] = data.ids[1, 0]
    data.ids[2, 1] = -1
    data.logits.requires_grad_()
    og.distill_loss(*data.args(), temperature=1.5, soft_weight=0.6,
                    hard_weight=0.4).sum().backward()
    for i in range(4):
        for j in range(11):
            ends = []
            for sign in (1, -1):
                moved = Detached(data)
                moved.logits = data.logits.detach().double()
                moved.logits[i, j] += sign * 2.0 ** -10
                ends.append(float(reference(moved, 1.5, 0.6, 0.4)[0].sum()))
            assert abs(float(data.logits.grad[i, j]) - (ends[0] - ends[1]) * 2.0 ** 9) < 1e-5


def test_refusals():
    data = Data(6, 50, 4)
    z, ids, t, y = data.args()
    f = og.distill_loss
    bad = [
        (TypeError, lambda: f(z.double(), ids, t)),
        (TypeError, lambda: f(z, ids.float(), t)),
        (TypeError, lambda: f(z, ids, t.double())),
        (TypeError, lambda: f(z, ids, None)),
        (TypeError, lambda: f(z, None, t)),
        (TypeError, lambda: f(None, ids, t)),
        (ValueError, lambda: f(z, ids[:3], t)),
        (ValueError, lambda: f(z, ids, t[:, :3])),
        (ValueError, lambda: f(z, ids, t, y[:3])),
        (ValueError, lambda: f(z, ids, t, y[:, None])),
        (ValueError, lambda: f(z, ids.cpu(), t)),
        (ValueError, lambda: f(z.t(), ids, t)),
        (ValueError, lambda: f(z[:, :0], ids, t)),
        (ValueError, lambda: f(z, ids, t, ignore_id=2 ** 63)),
        (og.LambError, lambda: f(z, ids, t, temperature=0.0)),
        (og.LambError, lambda: f(z, ids, t, temperature=-1.0)),
        (og.LambError, lambda: f(z, ids, t, temperature=math.inf)),
        (og.LambError, lambda: f(z, ids, t, temperature=math.nan)),
        (og.LambError, lambda: f(z, ids, t, soft_weight=math.nan)),
        (og.LambError, lambda: f(z, ids, t, y, hard_weight=math.inf)),
        (og.LambError, lambda: f(z, ids, t, hard_weight=0.5)),      # no labels
        (og.LambError, lambda: f(z, ids[:, :1].expand(6, 1025).contiguous(),
                                 t[:, :1].expand(6, 1025).contiguous())),
        (ValueError, lambda: og.distill_loss_grad(z, ids, t, row_grad=data.row_grad[:3])),
        (ValueError, lambda: og.distill_loss_grad(z, ids, t, row_grad=data.row_grad.to(BF16))),
        (ValueError, lambda: og.distill_loss_grad(z, ids, t, out=z[:3])),
        (TypeError, lambda: og.distill_loss_grad(z, ids, t, dtype=torch.float64)),
        (RuntimeError, lambda: f(z, ids, t.clone().requires_grad_())),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    leaf = data.logits.float().requires_grad_()
    with pytest.raises(RuntimeError):   # once only
        first, = torch.autograd.grad(f(leaf, ids, t).sum(), leaf, create_graph=True)
        torch.autograd.grad(first.sum(), leaf)


# ----------------------------------------------------------- streams and graphs
@pytest.mark.parametrize("vocab", [4096, 131071])
def test_another_stream_and_captured_graphs(vocab):
    data = Data(200, vocab, 16)

    def calls():
        return og.distill_loss_grad(*data.args(), hard_weight=0.5, row_grad=data.row_grad)

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
        new = Data(200, vocab, 16, seed=k + 1)
        for name in ("logits", "ids", "teacher", "labels", "row_grad"):
            getattr(data, name).copy_(getattr(new, name))
        graph, (loss, grad) = graphs[k % 2]
        graph.replay()
        want = reference(new, 1.0, 1.0, 0.5, row_grad=new.row_grad)
        near(loss, *want[:2], "loss")
        near(grad, *want[2:], "grad")


def test_calls_on_several_streams_at_once():
    cases = [Data(100, 9000, 8, seed=k) for k in range(4)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for stream, data in zip(streams, cases):
            with torch.cuda.stream(stream):
                got.append((data, og.distill_loss_grad(*data.args())))
    torch.cuda.synchronize()
    for data, (loss, grad) in got:
        want = reference(data, 1.0, 1.0, 0.0)
        near(loss, *want[:2], "loss")
        near(grad, *want[2:], "grad")


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,vocab", [(20, 5), (20, 4096), (2500, 4096), (2, 1_300_000)])
@pytest.mark.parametrize("temperature", [0.5, 1.0, 2.0])
def test_a_loss_near_the_largest_number_is_finite(dtype, n, vocab, temperature):
    """All of the teacher's weight on tokens of the type's lowest value."""
    data = Data(n, vocab, 4, dtype)
    data.ids[:] = torch.arange(4, device="cuda")
    data.logits[:, :4] = torch.finfo(dtype).min
    # soft T^2 sum of p 3.4e38 / T: 0.4 or 0.8 of the largest number.
    loss, tol, _, _ = reference(data, temperature, 0.4, 0.0)
    for got in (og.distill_loss(*data.args(), temperature=temperature, soft_weight=0.4),
                og.distill_loss_grad(*data.args(), temperature=temperature, soft_weight=0.4)[0]):
        near(got, loss, tol, "loss")


# ------------------------------------------- the loss alone, of more rows than are held
def check_loss(data, temperature=1.0, soft=1.0, hard=0.0, ignore=-100):
    loss, tol, _, _ = reference(data, temperature, soft, hard, ignore)
    got = og.distill_loss(*data.args(), temperature=temperature, soft_weight=soft,
                          hard_weight=hard, ignore_id=ignore)
    # A token of the type's lowest value that is named: soft T^2 times 3.4e38 / T, say, is
    # past fp32's largest number at T = 2, and rounds to infinity.
    past = (loss + 1.01 * tol > torch.finfo(FP32).max) & (got == math.inf)
    near(got, torch.where(past, math.inf, loss), tol, "loss")
    return got


@pytest.mark.parametrize("n,vocab", [(3700, 2047), (3700, 2048), (2400, 4096), (2500, 5001),
                                     (1300, 12007), (1000, 16384), (700, 32000), (1100, 32001),
                                     (500, 50001), (200, 131071), (160, 262144)])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
def test_the_loss_of_many_rows(n, vocab, dtype):
    data = Data(n, vocab, 11, dtype)
    data.labels[::9] = -100
    data.labels[3::11] = vocab
    data.ids[5::7, 4:] = -1
    data.ids[6::8] = vocab
    data.logits[1::13, 7:vocab // 2] = -math.inf
    data.logits[2::13, vocab // 2:vocab - 9] = torch.finfo(dtype).min
    data.ids[1::13] = torch.arange(11, device="cuda") % 7
    data.labels[1::13] = 6
    for temperature, soft, hard in ((1.0, 0.7, 0.3), (2.0, 0.7, 0.3), (3.0, 0.7, 0.3),
                                    (2.0, 1.0, 0.0), (2.0, 0.0, 1.0)):
        check_loss(data, temperature, soft, hard)


@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_the_loss_of_the_longest_rows(n, dtype):
    check_loss(Data(n, 3_000_001, 20, dtype), 2.0, 0.5, 0.5)


@pytest.mark.parametrize("top", [0, 31, 33, 127, 257, 1024])
def test_the_loss_of_many_rows_with_many_entries(top):
    check_loss(Data(2500, 4096, top), 2.0, 0.5, 0.5)
    check_loss(Data(700, 32000, top), 1.0, 0.5, 0.5)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vocab,stride,shift", [(4096, 4096, 1), (4096, 4104, 0), (4096, 4099, 3),
                                                (4099, 4101, 1), (4099, 4099, 2)])
def test_the_loss_of_many_rows_anywhere(dtype, vocab, stride, shift):
    n = 2500
    data = Data(n, vocab, 9, dtype)
    held = torch.full((shift + n * stride,), math.nan, dtype=dtype, device="cuda")
    rows = held[shift:].view(n, stride)[:, :vocab]
    rows.copy_(data.logits)
    data.logits = rows
    check_loss(data, 2.0, 0.5, 0.5)


@pytest.mark.parametrize("n,vocab", [(2500, 4096), (2000, 9001), (1000, 32000)])
@pytest.mark.parametrize("bad", [math.inf, math.nan, -math.inf])
def test_broken_rows_among_many_stay_alone(n, vocab, bad):
    data = Data(n, vocab, 6)
    how = dict(temperature=2.0, soft_weight=0.5, hard_weight=0.5)
    whole = og.distill_loss(*data.args(), **how)
    broken = torch.zeros(n, dtype=torch.bool, device="cuda")
    broken[7::97] = True
    if bad == -math.inf:
        data.logits[broken] = bad
    else:
        data.logits[broken, vocab // 3] = bad
    loss = og.distill_loss(*data.args(), **how)
    assert bool(loss[broken].isnan().all())
    assert torch.equal(loss[~broken], whole[~broken])


@pytest.mark.parametrize("n,vocab", [(2500, 4096), (1000, 32000), (200, 131071)])
def test_the_loss_of_many_rows_on_streams_and_in_graphs(n, vocab):
    how = dict(temperature=2.0, soft_weight=0.5, hard_weight=0.5)
    sets = [Data(n, vocab, 9, seed=k) for k in range(2)]
    want = [og.distill_loss(*d.args(), **how) for d in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for d, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(og.distill_loss(*d.args(), **how))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caught = og.distill_loss(*sets[0].args(), **how)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(caught, want[0])
    for to, other in zip(sets[0].args(), sets[1].args()):
        to.copy_(other)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(caught, want[1])
