"""The embedding lookup and its gradient on the GPU against plain 64-bit sums.

Tolerances.  With u the unit roundoff of the stored type (bf16 2^-8, fp16
2^-11, fp32 2^-24) and h half its smallest subnormal:
- lookup: one fp32 product and one rounding: (2^-24 + u) |x| + h;
- gradient: any order of adding n fp32 terms is off by at most
  (n - 1) 2^-24 sum|x| to first order; the product with the scale and the sum
  with the old value round once more each, then comes the rounding to the
  stored type: (n + 2) 2^-24 (|scale| sum|x| + |old|) + u |result| + h.
Both carry a factor of 1.01 for the terms of second order.
"""
import math

import pytest
import torch

import optimizer_step_gb300 as og

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
ROUND = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24}
HALF_SUB = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -150}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).to(dtype)


def make_ids(n, vocab, spread, seed, dtype=torch.int64):
    u = torch.rand(n, generator=gen(seed), device="cuda", dtype=torch.float64)
    if spread == "zipf":
        ids = torch.exp(u * math.log(vocab + 1)).long() - 1
    elif spread == "uniform":
        ids = (u * vocab).long()
    else:
        ids = torch.full((n,), int(spread), device="cuda", dtype=torch.int64)
    return ids.to(dtype)


def embed_reference(table, ids, scale, first_row):
    flat = ids.reshape(-1).long()
    held = (flat >= first_row) & (flat < first_row + table.shape[0])
    out = torch.zeros(flat.numel(), table.shape[1], dtype=torch.float64, device=table.device)
    out[held] = table.double()[flat[held] - first_row] * scale
    return out.reshape(*ids.shape, table.shape[1])


def check_embed(out, table, ids, scale=1.0, first_row=0):
    ref = embed_reference(table, ids, scale, first_row)
    assert out.shape == ref.shape
    tol = 1.01 * (2.0 ** -24 + ROUND[out.dtype]) * ref.abs() + HALF_SUB[out.dtype]
    diff = (out.double() - ref).abs()
    assert bool((diff <= tol).all()), float((diff - tol).max())


@pytest.mark.parametrize("dim", [1, 2, 3, 7, 8, 12, 64, 100, 513, 1023, 1024, 4096, 12289])
@pytest.mark.parametrize("tin,tout", [(BF16, BF16), (FP32, BF16), (FP16, FP32)])
def test_embed_widths(dim, tin, tout):
    table = randn((37, dim), tin, dim)
    ids = make_ids(101, 37, "uniform", 1)
    check_embed(og.embed(table, ids, scale=3.7, out_dtype=tout), table, ids, 3.7)


@pytest.mark.parametrize("tin", [BF16, FP16, FP32])
@pytest.mark.parametrize("tout", [BF16, FP16, FP32])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_embed_types(tin, tout, id_type):
    for dim in (40, 33):
        table = randn((500, dim), tin, 3)
        ids = make_ids(1000, 500, "zipf", 2, id_type)
        out = og.embed(table, ids, scale=0.3, out_dtype=tout)
        assert out.dtype == tout
        check_embed(out, table, ids, 0.3)


@pytest.mark.parametrize("n", [0, 1, 2, 31, 257, 4099, 70001])
def test_embed_lengths(n):
    table = randn((1000, 72), BF16, 5)
    ids = make_ids(n, 1000, "zipf", n)
    check_embed(og.embed(table, ids), table, ids)


def test_embed_default_scale_copies_bits():
    table = randn((50, 96), BF16, 5)
    ids = make_ids(300, 50, "uniform", 6)
    assert torch.equal(og.embed(table, ids).view(torch.int16), table[ids].view(torch.int16))


@pytest.mark.parametrize("dim", [16, 17, 1023])
def test_embed_slice_of_a_vocabulary(dim):
    table = randn((300, dim), FP32, 5)
    ids = make_ids(2000, 1000, "uniform", 6)
    ids[:8] = torch.tensor([-1, -2**63, 2**63 - 1, 449, 450, 749, 750, -450])
    out = og.embed(table, ids, first_row=450, scale=2.0)
    check_embed(out, table, ids, 2.0, 450)
    assert not out[ids >= 750].any() and not out[ids < 450].any()


def test_embed_slices_add_up_to_the_whole():
    table = randn((300, 24), FP32, 5)
    ids = make_ids(500, 300, "uniform", 6).view(4, 125)
    whole = og.embed(table, ids, scale=1.5)
    parts = [og.embed(table[a:b], ids, scale=1.5, first_row=a) for a, b in ((0, 99), (99, 300))]
    assert torch.equal(parts[0] + parts[1], whole)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("dim,stride,shift", [(64, 64, 1), (64, 72, 0), (64, 67, 3), (33, 40, 1),
                                              (5, 8, 0), (1000, 1001, 0), (8, 8, 4)])
def test_embed_strides_and_alignment_leave_the_gaps_alone(dtype, dim, stride, shift):
    rows, n = 41, 77
    store = randn((rows * stride + shift + 8,), dtype, 9)
    table = store[shift:shift + rows * stride].view(rows, stride)[:, :dim]
    ids = make_ids(n, rows, "uniform", 3)
    back = torch.full((n * stride + shift + 64,), 7.0, dtype=dtype, device="cuda")
    out = back[shift:shift + n * stride].view(n, stride)[:, :dim]
    assert og.embed(table, ids, out=out, scale=1.25) is out
    check_embed(out, table, ids, 1.25)
    gaps = back.clone()
    gaps[shift:shift + n * stride].view(n, stride)[:, :dim] = 7.0
    assert bool((gaps == 7.0).all())


def test_embed_infinities_and_nan_stay_in_their_rows():
    table = randn((10, 130), BF16, 1)
    table[3, 5], table[3, 6], table[3, 7] = float("inf"), float("-inf"), float("nan")
    ids = torch.tensor([3, 2, 3, 12, -1], device="cuda")
    out = og.embed(table, ids, scale=0.5)
    assert out[0, 5] == float("inf") and out[2, 6] == float("-inf") and out[0, 7].isnan()
    assert bool(torch.isfinite(out[1]).all()) and not out[3:].any()
    assert bool(og.embed(table, ids, scale=0.0)[0, 5].isnan())


def test_embed_offsets_past_32_bits():
    """Tables and outputs of more than 2^32 bytes, rows at both ends."""
    rows, dim = 600_000, 4096
    table = torch.empty((rows, dim), dtype=BF16, device="cuda")
    table[:3] = randn((3, dim), BF16, 1)
    table[-3:] = randn((3, dim), BF16, 2)
    ids = torch.tensor([0, 1, 2, rows - 1, rows - 2, rows - 3], device="cuda").repeat(100_000)
    out = og.embed(table, ids)
    for k in (0, 5, 299_999, 599_998, 599_999):
        assert torch.equal(out[k], table[ids[k]]), k


def test_embed_refusals():
    table = randn((10, 16), BF16, 1)
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad in (ids.float(), ids.to(torch.int16)):
        with pytest.raises(TypeError):
            og.embed(table, bad)
    with pytest.raises(TypeError):
        og.embed(table.double(), ids)
    with pytest.raises(TypeError):
        og.embed(table[0], ids)
    with pytest.raises(ValueError):
        og.embed(table, ids.cpu())
    with pytest.raises(ValueError):
        og.embed(table, torch.zeros(4, 2, dtype=torch.int64, device="cuda")[:, 0])
    with pytest.raises(ValueError):
        og.embed(table.t(), ids)
    with pytest.raises(ValueError):
        og.embed(table, ids, out=torch.empty(4, 15, dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        og.embed(table, ids, out=torch.empty(4, 16, dtype=BF16, device="cuda"), out_dtype=FP32)
    with pytest.raises(ValueError):
        og.embed(table, ids, out=torch.empty(16, 4, dtype=BF16, device="cuda").t())
    with pytest.raises(ValueError):   # every row is the same memory
        og.embed(table, ids, out=torch.empty(1, 16, dtype=BF16, device="cuda").expand(4, 16))
    with pytest.raises(og.LambError):
        og.embed(table, ids, first_row=-1)


# ------------------------------------------------------------------ gradient
def grad_reference(dy, ids, rows, scale, first_row, padding, old):
    """(result, sum of magnitudes, count) a row in 64 bits."""
    flat = ids.reshape(-1).long()
    x = dy.reshape(-1, dy.shape[-1]).double()
    held = (flat >= first_row) & (flat < first_row + rows) & (flat != padding)
    at = flat[held] - first_row
    total = torch.zeros(rows, x.shape[1], dtype=torch.float64, device=x.device)
    total.index_add_(0, at, x[held])
    size = torch.zeros_like(total).index_add_(0, at, x[held].abs())
    count = torch.bincount(at, minlength=rows).double()
    result = scale * total
    if old is not None:
        result = result + old.double()
        size = abs(scale) * size + old.double().abs()
    else:
        size = abs(scale) * size
    return result, size, count


def check_grad(out, dy, ids, scale=1.0, first_row=0, padding=-1, old=None):
    ref, size, count = grad_reference(dy, ids, out.shape[0], scale, first_row, padding, old)
    tol = 1.01 * ((count[:, None] + 2) * 2.0 ** -24 * size + ROUND[out.dtype] * ref.abs()) \
        + HALF_SUB[out.dtype]
    diff = (out.double() - ref).abs()
    assert bool((diff <= tol).all()), float((diff - tol).max())
    idle = count == 0
    if old is None:
        assert not out[idle].any()
    else:
        assert torch.equal(out[idle], old[idle])


@pytest.mark.parametrize("dim", [1, 2, 3, 8, 12, 64, 100, 255, 513, 1024, 2049, 4096])
@pytest.mark.parametrize("tin,tout", [(BF16, BF16), (FP16, FP32), (FP32, BF16)])
def test_grad_widths(dim, tin, tout):
    ids = make_ids(700, 90, "zipf", dim)
    dy = randn((700, dim), tin, 2)
    check_grad(og.embed_grad(dy, ids, n_rows=90, scale=1.7, dtype=tout), dy, ids, 1.7)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("tin", [BF16, FP16, FP32])
@pytest.mark.parametrize("tout", [BF16, FP16, FP32])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_grad_types(tin, tout, id_type, accumulate):
    for dim in (48, 31):
        ids = make_ids(3000, 2000, "uniform", 4, id_type)
        dy = randn((3000, dim), tin, 5, 0.01)
        out = randn((2000, dim), tout, 6, 0.01)
        old = out.clone() if accumulate else None
        og.embed_grad(dy, ids, out=out, scale=0.7, accumulate=accumulate)
        check_grad(out, dy, ids, 0.7, old=old)


@pytest.mark.parametrize("spread", ["zipf", "uniform", "5"])
@pytest.mark.parametrize("n", [0, 1, 2, 33, 63, 64, 65, 1000, 1025, 2047, 2049, 4097, 8193, 16385,
                               40000, 131073])
def test_grad_lengths(n, spread):
    rows, dim = 1003, 40
    ids = make_ids(n, rows, spread, n)
    dy = randn((n, dim), BF16, n + 1)
    for accumulate in (False, True):
        out = randn((rows, dim), FP32, 6)
        old = out.clone() if accumulate else None
        og.embed_grad(dy, ids, out=out, accumulate=accumulate)
        check_grad(out, dy, ids, old=old)


@pytest.mark.parametrize("n", [15, 16, 17, 255, 257, 512, 513, 2048, 2049, 16384, 16385, 32769, 65537])
@pytest.mark.parametrize("dim", [8, 129, 520])
def test_grad_where_the_ways_of_working_change(n, dim):
    """Lengths beside each limit of the sort and of the cut into blocks, with
    runs that end in, at and behind the ends of blocks."""
    rows = 97
    u = torch.arange(n, device="cuda")
    for ids in ((u * u) % 89 % rows, torch.where(u % 3 == 0, 11, (u // 7) % rows), u * rows // n):
        dy = randn((n, dim), BF16, n)
        out = randn((rows, dim), FP32, 3)
        old = out.clone()
        og.embed_grad(dy, ids, out=out, accumulate=True, scale=0.5)
        check_grad(out, dy, ids, 0.5, old=old)
        check_grad(og.embed_grad(dy, ids, n_rows=rows), dy, ids)


@pytest.mark.parametrize("n,dim", [(40_000, 3), (40_000, 21), (9000, 4100), (131_073, 12)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_of_one_token_throughout(n, dim, accumulate):
    ids = torch.full((n,), 6, device="cuda", dtype=torch.int32)
    ids[n // 2] = 3
    dy = randn((n, dim), FP16, 1)
    out = randn((9, dim), FP32, 2)
    old = out.clone() if accumulate else None
    og.embed_grad(dy, ids, out=out, accumulate=accumulate)
    check_grad(out, dy, ids, old=old)


@pytest.mark.parametrize("rows", [1, 2, 255, 256, 257, 65535, 65537, 150_001])
def test_grad_row_counts(rows):
    for n in (50, 5000, 30_000):
        ids = make_ids(n, rows, "uniform", rows + n)
        ids[0], ids[-1] = rows - 1, 0
        dy = randn((n, 24), FP32, 3)
        check_grad(og.embed_grad(dy, ids, n_rows=rows, dtype=FP32), dy, ids)


@pytest.mark.parametrize("n", [300, 6000, 50_000])
def test_grad_slice_padding_and_foreign_tokens(n):
    """NaN and infinities in the grads of masked tokens do not come through."""
    ids = make_ids(n, 3000, "uniform", 8)
    ids[:6] = torch.tensor([-1, -2**63, 2**63 - 1, 999, 2000, -1500], device="cuda")
    dy = randn((n, 72), BF16, 9)
    masked = (ids < 1000) | (ids >= 2000) | (ids == 1234)
    dy[masked] = float("nan")
    dy[torch.nonzero(masked)[::2].flatten()] = float("inf")
    clean = torch.where(masked[:, None], torch.zeros_like(dy), dy)
    for accumulate in (False, True):
        out = randn((1000, 72), BF16, 10)
        old = out.clone() if accumulate else None
        og.embed_grad(dy, ids, out=out, first_row=1000, padding_id=1234, accumulate=accumulate,
                      scale=2.0)
        check_grad(out, clean, ids, 2.0, 1000, 1234, old)


@pytest.mark.parametrize("n", [200, 20_000])
def test_grad_with_every_token_masked(n):
    dy = torch.full((n, 33), float("nan"), dtype=BF16, device="cuda")
    ids = torch.full((n,), 7, device="cuda")
    assert not og.embed_grad(dy, ids, n_rows=20, padding_id=7).any()
    assert not og.embed_grad(dy, ids, n_rows=20, first_row=8).any()
    out = randn((20, 33), FP32, 1)
    old = out.clone()
    og.embed_grad(dy, ids, out=out, padding_id=7, accumulate=True)
    assert torch.equal(out, old)


def test_grad_nan_stays_in_its_row():
    ids = make_ids(9000, 500, "uniform", 3)
    dy = randn((9000, 64), BF16, 4)
    dy[17] = float("nan")
    out = og.embed_grad(dy, ids, n_rows=500)
    named = torch.zeros(500, dtype=torch.bool, device="cuda")
    named[ids[17]] = True
    assert torch.equal(out.isnan().all(1), named) and torch.equal(out.isnan().any(1), named)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("dim,stride,shift", [(64, 64, 1), (64, 72, 0), (64, 67, 3), (33, 40, 1),
                                              (5, 8, 0), (1000, 1001, 0), (8, 8, 4)])
@pytest.mark.parametrize("n", [60, 9000])
def test_grad_strides_and_alignment_leave_the_gaps_alone(dtype, dim, stride, shift, n):
    rows = 300
    store = randn((n * stride + shift + 8,), dtype, 9)
    dy = store[shift:shift + n * stride].view(n, stride)[:, :dim]
    ids = make_ids(n, rows, "zipf", 3)
    for accumulate in (False, True):
        back = torch.full((rows * stride + shift + 64,), 7.0, dtype=dtype, device="cuda")
        out = back[shift:shift + rows * stride].view(rows, stride)[:, :dim]
        old = out.clone() if accumulate else None
        assert og.embed_grad(dy, ids, out=out, accumulate=accumulate) is out
        check_grad(out, dy, ids, old=old)
        back[shift:shift + rows * stride].view(rows, stride)[:, :dim] = 7.0
        assert bool((back == 7.0).all())


def test_grad_gives_the_same_bits_every_time():
    for n, rows in ((900, 50), (12_000, 700), (60_000, 32_000)):
        ids = make_ids(n, rows, "zipf", 1)
        dy = randn((n, 136), BF16, 2)
        first = og.embed_grad(dy, ids, n_rows=rows, dtype=FP32)
        for fill in (0, 255, 77):
            # What the workspace held before must not matter.
            del_me = torch.full((1 << 24,), fill, dtype=torch.uint8, device="cuda")
            del del_me
            assert torch.equal(og.embed_grad(dy, ids, n_rows=rows, dtype=FP32), first)


def test_grad_offsets_past_32_bits():
    """More than 2^31 grads of outputs and of the table."""
    n, rows, dim = 300_001, 280_000, 8192
    dy = torch.zeros((n, dim), dtype=BF16, device="cuda")
    ids = torch.arange(n, device="cuda") % 1000
    for k, v in ((0, 5), (150_000, rows - 1), (n - 1, rows - 1), (n - 2, 0)):
        ids[k] = v
        dy[k] = randn((dim,), BF16, k)
    out = og.embed_grad(dy, ids, n_rows=rows)
    last = (dy[150_000].double() + dy[n - 1].double())
    assert torch.equal(out[5], dy[0]) and torch.equal(out[0], dy[n - 2])
    assert bool(((out[rows - 1].double() - last).abs()
                 <= 1.01 * (2.0 ** -8 + 2.0 ** -22) * last.abs() + 2.0 ** -22).all())
    assert int(out.any(1).sum()) == 3


def test_grad_matches_differences_of_the_lookup():
    """The lookup is linear, and with a power of two as scale and values of few
    bits every difference is exact."""
    rows, dim, n, h = 6, 5, 11, 0.25
    table = torch.randint(-64, 64, (rows, dim), generator=gen(1), device="cuda").float() / 16
    ids = torch.randint(0, rows, (n,), generator=gen(2), device="cuda")
    weight = torch.randint(-64, 64, (n, dim), generator=gen(3), device="cuda").float() / 8

    def loss(t):
        return float((og.embed(t, ids, scale=4.0).double() * weight.double()).sum())

    out = og.embed_grad(weight, ids, n_rows=rows, scale=4.0, padding_id=-1)
    for v in range(rows):
        for d in range(dim):
            step = torch.zeros_like(table)
            step[v, d] = h
            assert float(out[v, d]) == (loss(table + step) - loss(table - step)) / (2 * h)


def test_calls_follow_the_current_stream():
    side = torch.cuda.Stream()
    table, ids = randn((400, 256), BF16, 1), make_ids(5000, 400, "zipf", 2)
    dy = randn((5000, 256), BF16, 3)
    want, want_grad = og.embed(table, ids), og.embed_grad(dy, ids, n_rows=400)
    late_table, late_dy = torch.zeros_like(table), torch.zeros_like(dy)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late_table.copy_(table)
        late_dy.copy_(dy)
        got, got_grad = og.embed(late_table, ids), og.embed_grad(late_dy, ids, n_rows=400)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(got_grad, want_grad)


def test_calls_can_be_captured_into_a_graph():
    table, ids = randn((400, 256), BF16, 1), make_ids(5000, 400, "zipf", 2)
    dy = randn((5000, 256), BF16, 3)
    out, grad = torch.empty_like(dy), torch.empty((400, 256), dtype=FP32, device="cuda")
    og.embed(table, ids, out=out)
    og.embed_grad(dy, ids, out=grad)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og.embed(table, ids, out=out, scale=2.0)
        og.embed_grad(dy, ids, out=grad, scale=2.0)
    ids.copy_(make_ids(5000, 400, "uniform", 20))
    dy.copy_(randn((5000, 256), BF16, 30))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check_embed(out, table, ids, 2.0)
    check_grad(grad, dy, ids, 2.0)


def test_a_graph_with_copies_and_fills_between_the_calls():
    """Copies and fills in front of and between the calls keep their order."""
    table, ids = randn((600, 136), BF16, 1), make_ids(6000, 600, "zipf", 2)
    dy, few = randn((6000, 136), BF16, 3), make_ids(40, 600, "uniform", 4)
    table_in, ids_in, dy_in = torch.zeros_like(table), torch.zeros_like(ids), torch.zeros_like(dy)
    out, grad = torch.empty_like(dy), torch.empty((600, 136), dtype=FP32, device="cuda")
    small = torch.empty((600, 136), dtype=FP32, device="cuda")

    def work():
        table_in.copy_(table)
        ids_in.copy_(ids)
        og.embed(table_in, ids_in, out=out)
        dy_in.copy_(out)
        grad.fill_(1.0)
        og.embed_grad(dy_in, ids_in, out=grad, accumulate=True)
        dy_in.zero_()
        small.copy_(grad)
        og.embed_grad(out[:40], few, out=small, accumulate=True)
        out.zero_()

    work()
    torch.cuda.synchronize()
    want, want_small = grad.clone(), small.clone()
    check_grad(want, table[ids], ids, old=torch.ones_like(grad))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for _ in range(3):
        grad.fill_(-5.0)
        small.fill_(-5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(grad, want) and torch.equal(small, want_small)


def test_calls_on_several_streams_at_once():
    cases = []
    for k, n in enumerate((300, 9000, 40_000, 150_000)):
        ids = make_ids(n, 5000, "zipf", k)
        dy = randn((n, 200), BF16, k + 10)
        cases.append((dy, ids, og.embed_grad(dy, ids, n_rows=5000), og.embed(dy[:5000], ids)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(10):
        for (dy, ids, _, _), stream in zip(cases, streams):
            with torch.cuda.stream(stream):
                got.append((og.embed_grad(dy, ids, n_rows=5000), og.embed(dy[:5000], ids)))
    torch.cuda.synchronize()
    for i, (grad, out) in enumerate(got):
        assert torch.equal(grad, cases[i % 4][2]) and torch.equal(out, cases[i % 4][3])


def test_grad_refusals():
    dy = randn((4, 16), BF16, 1)
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    out = torch.zeros(9, 16, device="cuda")
    with pytest.raises(ValueError):
        og.embed_grad(dy, ids)
    with pytest.raises(ValueError):
        og.embed_grad(dy, ids, n_rows=9, accumulate=True)
    with pytest.raises(ValueError):
        og.embed_grad(dy[:3], ids, n_rows=9)
    with pytest.raises(ValueError):
        og.embed_grad(dy, ids, n_rows=8, out=out)
    with pytest.raises(ValueError):
        og.embed_grad(dy, ids, out=out, dtype=BF16)
    with pytest.raises(ValueError):
        og.embed_grad(dy, ids, out=out[:, :15])
    with pytest.raises(TypeError):
        og.embed_grad(dy.double(), ids, out=out)
    with pytest.raises(TypeError):
        og.embed_grad(dy, ids.float(), out=out)
    with pytest.raises(ValueError):
        og.embed_grad(dy, ids, out=torch.zeros(16, 9, device="cuda").t())
    with pytest.raises(og.LambError):
        og.embed_grad(dy, ids, out=out, first_row=-5)


@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
def test_ids_at_any_offset(id_type, shift):
    for n in (5, 700, 5001):
        ids = make_ids(n + shift, 60, "uniform", n, id_type)[shift:]
        dy = randn((n, 520), BF16, 1)
        table = randn((60, 520), BF16, 2)
        check_embed(og.embed(table, ids), table, ids)
        check_grad(og.embed_grad(dy, ids, n_rows=60, padding_id=3), dy, ids, padding=3)


def test_embed_takes_ids_of_any_shape():
    table = randn((50, 40), BF16, 1)
    for shape in ((), (3,), (2, 3), (2, 0, 3), (2, 3, 4)):
        ids = make_ids(math.prod(shape), 50, "uniform", 2).view(shape)
        out = og.embed(table, ids)
        assert out.shape == shape + (40,)
        assert torch.equal(out, table[ids])
        grad = og.embed_grad(out, ids, n_rows=50, dtype=FP32)
        check_grad(grad, out, ids)
    # A batch-first view of a sequence-first output: rows do not step evenly.
    with pytest.raises(ValueError):
        og.embed(table, make_ids(6, 50, "uniform", 2).view(2, 3),
                 out=torch.empty(3, 2, 40, dtype=BF16, device="cuda").transpose(0, 1))
