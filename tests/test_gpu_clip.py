"""The global gradient norm and clipping on the GPU against plain 64-bit sums.

Tolerances.  Squares are added in fp32 at most 128 at a time, so the sum of
squares is off by at most 130 * 2^-24 of itself (7.8e-6), the norm and the
factor by half of that and one fp32 rounding: 4e-6 covers both.  A clipped
grad carries the factor's error, the product's rounding and the rounding to
its type (unit roundoff u, half a subnormal h): (4e-6 + 2^-24 + u) |x| + h.
"""
import math

import pytest
import torch

import optimizer_step_gb300 as og
import workloads as W
from optimizer_step_gb300 import Lamb

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
ROUND = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24}
HALF_SUB = {BF16: 2.0 ** -134, FP16: 2.0 ** -25, FP32: 2.0 ** -150}
RTOL = 4e-6


def make(sizes, types, seed=0, std=1.0, shift=0, gap=0):
    """Tensors one after another in a flat buffer a type, shift elements off
    the alignment, gap elements apart; the gaps hold NaN."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    found, flats = [None] * len(sizes), []
    for dt in sorted(set(types), key=str):
        mine = [i for i, t in enumerate(types) if t == dt]
        flat = torch.full((shift + sum(sizes[i] + gap for i in mine) + 8,), float("nan"),
                          dtype=dt, device="cuda")
        at = shift
        for i in mine:
            found[i] = flat[at:at + sizes[i]]
            found[i].copy_(torch.randn(sizes[i], generator=g, device="cuda") * std)
            at += sizes[i] + gap
        flats.append(flat)
    return found, flats


def reference(grads, max_norm, loss_scale):
    square = sum(float(x.double().square().sum()) for x in grads)
    if not math.isfinite(square):
        return math.inf, 0.0, 1.0
    norm = math.sqrt(square) / loss_scale
    c = max_norm / norm if max_norm > 0 and norm > max_norm else 1.0
    return norm, c / loss_scale, 0.0


def check_stats(stats, want):
    got = stats.tolist()
    assert got[2] == want[2]
    for a, b in zip(got[:2], want[:2]):
        assert a == b or abs(a - b) <= RTOL * abs(b), (got, want)


def check_out(out, before, factor):
    for i, (a, b) in enumerate(zip(out, before)):
        ref = b.double() * factor
        tol = (RTOL + 2.0 ** -24 + ROUND[a.dtype]) * ref.abs() + HALF_SUB[a.dtype]
        assert bool(((a.double() - ref).abs() <= tol).all()), i


MIXES = {"bf16": [BF16], "fp16": [FP16], "fp32": [FP32], "mixed": [BF16, FP32, FP16]}
SIZES = {
    "none": [], "empty": [0, 0], "one": [1], "small": [1, 2, 3, 5, 7, 8, 9, 31, 33],
    "edges": [4095, 4096, 4097, 0, 16383, 16384, 16385, 1],
    "many": [(i * 37) % 301 for i in range(3000)], "large": [3_000_001, 5, 1_234_567],
}


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("shift,gap", [(0, 0), (1, 0), (3, 5)])
def test_norm_and_clip_into_other_tensors(sizes, mix, shift, gap):
    sizes = SIZES[sizes]
    types = [MIXES[mix][i % len(MIXES[mix])] for i in range(len(sizes))]
    grads, flats = make(sizes, types, 1, 0.5, shift, gap)
    before = [f.clone() for f in flats]
    for to in (BF16, FP32):
        out, back = make(sizes, [to] * len(sizes), 2, 1.0, 2, gap)
        with og.GradClip(grads, out) as clipper:
            check_stats(clipper.norm(), reference(grads, 0.0, 1.0))
            want = reference(grads, 0.25, 2.0)
            check_stats(clipper.clip(0.25, loss_scale=2.0), want)
            check_out(out, grads, want[1])
        if gap and sizes:
            lost = back[0].clone()
            for x in out:
                start = x.storage_offset()
                lost[start:start + x.numel()] = float("nan")
            assert bool(lost.isnan().all())
    assert all(torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())
               for a, b in zip(flats, before))


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("max_norm,loss_scale", [(0.5, 1.0), (1e9, 1.0), (0.0, 1.0), (-1.0, 4.0),
                                                 (0.5, 1024.0), (0.0, 0.125)])
def test_clip_in_place(mix, max_norm, loss_scale):
    sizes = [5, 4097, 0, 70_003, 16]
    types = [MIXES[mix][i % len(MIXES[mix])] for i in range(len(sizes))]
    grads, flats = make(sizes, types, 3, 0.5, 1, 3)
    before = [x.clone() for x in grads]
    want = reference(grads, max_norm, loss_scale)
    with og.GradClip(grads) as clipper:
        check_stats(clipper.clip(max_norm, loss_scale), want)
    if want[1] == 1.0:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    else:
        check_out(grads, before, want[1])
    for f in flats:  # the gaps are untouched
        assert int(f.isnan().sum()) == f.numel() - sum(
            x.numel() for x in grads if x.dtype == f.dtype)


def test_clip_of_some_in_place_and_some_elsewhere():
    grads, _ = make([100, 5000, 33], [FP32, BF16, FP32], 3)
    before = [x.clone() for x in grads]
    out = [grads[0], torch.zeros(5000, device="cuda"), torch.zeros(33, dtype=FP16, device="cuda")]
    with og.GradClip(grads, out) as clipper:
        stats = clipper.clip(1.0)
        check_stats(stats, reference(before, 1.0, 1.0))
        check_out(out, before, reference(before, 1.0, 1.0)[1])
    assert torch.equal(grads[1], before[1]) and torch.equal(grads[2], before[2])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("where", [(0, 0), (1, 4096), (2, 299_999), (3, 2)])
@pytest.mark.parametrize("mix", MIXES)
def test_a_bad_grad_stops_the_write(bad, where, mix):
    sizes = [9, 4097, 300_000, 3]
    types = [MIXES[mix][i % len(MIXES[mix])] for i in range(len(sizes))]
    grads, _ = make(sizes, types, 4)
    grads[where[0]][where[1]] = bad
    before = [x.clone() for x in grads]
    out, _ = make(sizes, [BF16] * 4, 5)
    kept = [x.clone() for x in out]
    with og.GradClip(grads, out) as elsewhere, og.GradClip(grads) as in_place:
        for clipper in (elsewhere, in_place):
            assert clipper.clip(1.0, loss_scale=2.0).tolist() == [math.inf, 0.0, 1.0]
            assert clipper.norm().tolist() == [math.inf, 0.0, 1.0]
        assert all(torch.equal(a, b) for a, b in zip(out, kept))
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
                   for a, b in zip(grads, before))
        grads[where[0]][where[1]] = 1.0  # the next call starts afresh
        check_stats(elsewhere.norm(), reference(grads, 0.0, 1.0))
        want = reference(grads, 1.0, 1.0)
        check_stats(in_place.clip(1.0), want)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("std", [1e-37, 1e-30, 1e-21, 1e-12, 1e12, 1e18, 3e19, 1e30])
def test_squares_outside_the_range_of_fp32(dtype, std):
    """Squares that leave fp32's range still count: the norm is right as long
    as it is itself an fp32 number."""
    grads, _ = make([5, 4096, 33_333], [dtype] * 3, 6, std)
    out = [torch.zeros_like(x) for x in grads]
    with og.GradClip(grads, out) as clipper:
        check_stats(clipper.norm(), reference(grads, 0.0, 1.0))
        want = reference(grads, std, 1.0)
        check_stats(clipper.clip(std), want)
        check_out(out, grads, want[1])


def test_one_large_grad_among_tiny_ones_and_zeros():
    grads, _ = make([10_000, 4, 50_000], [FP32, BF16, FP32], 7, 1e-25)
    grads[0].zero_()
    with og.GradClip(grads) as clipper:
        check_stats(clipper.norm(), reference(grads, 0.0, 1.0))
        grads[2][12_345] = 1e25
        check_stats(clipper.norm(), reference(grads, 0.0, 1.0))
        for x in grads:
            x.zero_()
        assert clipper.clip(1.0).tolist() == [0.0, 1.0, 0.0]


@pytest.mark.parametrize("mix", MIXES)
def test_halves_over_ranks_equal_the_whole(mix):
    sizes = [1000, 77, 50_001, 3, 20_000]
    types = [MIXES[mix][i % len(MIXES[mix])] for i in range(len(sizes))]
    grads, _ = make(sizes, types, 8)
    whole = [torch.zeros(n, dtype=BF16, device="cuda") for n in sizes]
    parts = [torch.zeros(n, dtype=BF16, device="cuda") for n in sizes]
    with og.GradClip(grads, whole) as every, og.GradClip(grads[:2], parts[:2]) as a, \
            og.GradClip(grads[2:], parts[2:]) as b:
        stats = every.clip(0.5, loss_scale=8.0).clone()
        ex = [torch.full((2,), 7.0, dtype=torch.float64, device="cuda") for _ in range(2)]
        total = a.partial(ex[0]) + b.partial(ex[1])
        for clipper in (a, b):
            check_stats(clipper.finish(total, 0.5, loss_scale=8.0), stats.tolist())
        check_out(parts, grads, reference(grads, 0.5, 8.0)[1])
        # One rank's inf stops the write on every rank.
        grads[4][5] = float("nan")
        kept = [x.clone() for x in parts]
        total = a.partial(ex[0]) + b.partial(ex[1])
        assert float(total[1]) == 1.0
        for clipper in (a, b):
            assert clipper.finish(total, 0.5).tolist() == [math.inf, 0.0, 1.0]
        assert all(torch.equal(x, y) for x, y in zip(parts, kept))


def test_norm_and_skip_agree_with_the_optimizer_step():
    wl = W.scaled(W.ragged(200, 16), 1 << 16)
    _, gv = W.make_grads(wl, 1, "cuda")
    st = W.make_state(wl, "cuda")
    with Lamb(st.w, st.m, st.v, st.w16, wl.wd_flags) as opt, og.GradClip(gv) as clipper:
        stats = clipper.norm().tolist()
        _, norm = opt.step(wl.lr, wl.t0, 0.0, 1.0, grads=gv)
        assert abs(stats[0] - norm) <= 2 * RTOL * norm
        ex = torch.zeros(2, dtype=torch.float64, device="cuda")
        assert abs(math.sqrt(float(clipper.partial(ex)[0])) - norm) <= 2 * RTOL * norm


def test_clip_gives_the_same_bits_every_time():
    grads, _ = make([(i * 7919) % 20_011 for i in range(400)], [BF16] * 400, 9)
    with og.GradClip(grads) as clipper:
        first = clipper.norm().clone()
        for _ in range(5):
            assert torch.equal(clipper.norm(), first)
        ex = torch.zeros(2, dtype=torch.float64, device="cuda")
        sums = [float(clipper.partial(ex)[0]) for _ in range(5)]
        assert len(set(sums)) == 1


def test_clip_runs_on_its_stream_and_in_a_graph():
    side = torch.cuda.Stream()
    source, _ = make([40_000, 3], [FP32, FP32], 10)
    grads = [torch.zeros_like(x) for x in source]
    out = [torch.zeros(x.numel(), dtype=BF16, device="cuda") for x in source]
    torch.cuda.synchronize()
    clipper = og.GradClip(grads, out, stream=side)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for a, b in zip(grads, source):
            a.copy_(b)
    stats = clipper.clip(1.0)
    side.synchronize()
    want = reference(source, 1.0, 1.0)
    check_stats(stats, want)
    check_out(out, source, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        clipper.clip(2.0)
    for x in grads:
        x.mul_(3.0)
    torch.cuda.synchronize()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    want = reference(grads, 2.0, 1.0)
    check_stats(stats, want)
    check_out(out, grads, want[1])
    clipper.close()


def test_offsets_past_32_bits():
    n = (1 << 31) + 12_345
    grads = [torch.zeros(n, dtype=BF16, device="cuda")]
    grads[0][-1], grads[0][5], grads[0][1 << 31] = 3.0, 4.0, 12.0
    with og.GradClip(grads) as clipper:
        assert clipper.norm().tolist() == [13.0, 1.0, 0.0]
        check_stats(clipper.clip(6.5), (13.0, 0.5, 0.0))
    assert [float(grads[0][k]) for k in (-1, 5, 1 << 31)] == [1.5, 2.0, 6.0]


def test_clip_refusals():
    x = torch.zeros(8, device="cuda")
    for bad in ([x.double()], ["x"], [x.to(torch.int32)]):
        with pytest.raises((TypeError, ValueError)):
            og.GradClip(bad)
    for bad in ([x.view(2, 4).t()], [x, x.cpu()]):
        with pytest.raises(ValueError):
            og.GradClip(bad)
    with pytest.raises(ValueError):
        og.GradClip([x], out=[x, x])
    with pytest.raises(ValueError):
        og.GradClip([x], out=[x[:7]])
    with pytest.raises(TypeError):
        og.GradClip([x], out=[x.double()])
    clipper = og.GradClip([x])
    for scale in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(og.LambError):
            clipper.norm(loss_scale=scale)
        with pytest.raises(og.LambError):
            clipper.clip(1.0, loss_scale=scale)
    with pytest.raises(og.LambError):
        clipper.clip(math.nan)
    for bad in (torch.zeros(2, device="cuda"), torch.zeros(3, dtype=torch.float64, device="cuda"),
                torch.zeros(2, dtype=torch.float64)):
        with pytest.raises(ValueError):
            clipper.partial(bad)
        with pytest.raises(ValueError):
            clipper.finish(bad, 1.0)
    clipper.close()
    with pytest.raises(RuntimeError):
        clipper.norm()
