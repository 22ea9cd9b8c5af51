"""Dense gradients so large that their zero rows are written by several kernels:
some beside the sort, most by CTAs behind the sums, the rest beside the join.
What was there before is NaN, so a row that is missed, or written by none of
them, shows; so do the gaps between rows.

Tolerance: any order of adding n fp32 terms, the product with the scale, one
rounding: (n + 2) 2^-24 |scale| sum|x| + u |result| + half a subnormal."""
import pytest
import torch

import optimizer_step_gb300 as og
from test_gpu_embedding import BF16, FP16, FP32, HALF_SUB, ROUND, make_ids, randn

pytestmark = pytest.mark.gpu


def check(out, dy, ids, scale, first_row=0, padding=-1):
    """Rows without a token are zero, the others are checked in 64 bits."""
    rows = out.shape[0]
    flat = ids.long() - first_row
    held = torch.nonzero((flat >= 0) & (flat < rows) & (ids != padding)).flatten()
    named, at = torch.unique(flat[held], return_inverse=True)
    idle = torch.ones(rows, dtype=torch.bool, device="cuda")
    idle[named] = False
    for part in torch.nonzero(idle).flatten().split(4096):
        assert not out[part].any()   # a NaN counts as not zero
    x = dy[held].double()
    ref = torch.zeros(named.numel(), x.shape[1], dtype=torch.float64, device="cuda")
    size = torch.zeros_like(ref).index_add_(0, at, x.abs())
    ref.index_add_(0, at, x)
    n = torch.bincount(at, minlength=named.numel()).double()[:, None]
    ref, size = scale * ref, abs(scale) * size
    tol = 1.01 * ((n + 2) * 2.0 ** -24 * size + ROUND[out.dtype] * ref.abs()) \
        + HALF_SUB[out.dtype]
    assert bool(((out[named].double() - ref).abs() <= tol).all())


def run(n, rows, dim, tin, tout, spread, gap=0, shift=0, id_type=torch.int64, **how):
    vocab = rows + 2 * how.get("first_row", 0)
    ids = make_ids(n, vocab, spread, n + rows, id_type)
    dy = randn((n, dim), tin, 3)
    back = torch.full((shift + rows * (dim + gap) + 8,), float("nan"), dtype=tout, device="cuda")
    out = back[shift:shift + rows * (dim + gap)].view(rows, dim + gap)[:, :dim]
    og.embed_grad(dy, ids, out=out, scale=0.75, **how)
    check(out, dy, ids, 0.75, how.get("first_row", 0), how.get("padding_id", -1))
    first = out.clone() if out.numel() < 1 << 28 else None
    out.fill_(float("nan"))
    assert bool(back.isnan().all())   # nothing outside the rows was written
    if first is not None:             # and the same bits every time
        og.embed_grad(dy, ids, out=out, scale=0.75, **how)
        assert torch.equal(out, first)


# Rows a CTA of the first kernel looks at: 128, 96, 352, 512 or 32; the last one has
# fewer in all but the first case.
@pytest.mark.parametrize("spread", ["zipf", "uniform", "77"])
@pytest.mark.parametrize("n,rows,dim,tin,tout", [
    (8192, 32000, 4096, BF16, BF16),
    (9000, 20011, 1023, FP16, FP32),
    (8192, 20011, 2560, FP32, BF16),
    (20_000, 100_003, 520, BF16, FP16),
    (131_072, 150_001, 264, BF16, FP32),
    (2049, 9001, 4104, BF16, BF16),
])
def test_zero_rows_behind_the_sums_and_the_join(n, rows, dim, tin, tout, spread):
    run(n, rows, dim, tin, tout, spread)


@pytest.mark.parametrize("gap,shift", [(0, 3), (8, 0), (5, 1)])
@pytest.mark.parametrize("dim", [2560, 2557])
def test_zero_rows_with_gaps_and_off_the_alignment(dim, gap, shift):
    run(8192, 12_007, dim, BF16, BF16, "zipf", gap, shift, torch.int32)


def test_zero_rows_of_a_slice_with_padding():
    run(9000, 20_011, 1280, BF16, FP32, "uniform", first_row=5000, padding_id=5077)


@pytest.mark.parametrize("n,rows,dim", [(5, 1100, 300_001), (9, 1101, 400_008)])
def test_few_tokens_of_very_wide_rows(n, rows, dim):
    """No run is long, so the last kernel only writes zeros."""
    run(n, rows, dim, BF16, BF16, "uniform")


@pytest.mark.parametrize("dim", [600_008, 600_001])
def test_grads_so_large_that_no_zero_row_is_written_beside_the_sort(dim):
    """The part for that time is less than a row of each CTA's range."""
    run(13, 2100, dim, BF16, BF16, "uniform")


def test_every_token_masked():
    ids = torch.full((6000,), 12, device="cuda")
    out = torch.full((20_011, 1280), float("nan"), device="cuda")
    og.embed_grad(torch.full((6000, 1280), float("nan"), device="cuda"), ids, out=out,
                  padding_id=12)
    assert not out.any()
