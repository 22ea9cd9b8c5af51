"""Cases that measure the operators in front of the optimizer step.

Four operators: the embedding lookup with scaling (``embed``), its gradient by
sorted tokens (``embed_grad``), the global gradient norm over many tensors
(``norm``) and clipping by it (``clip``).  Each has a plain form in elementary
torch operations, 32 bits wide and rounded once at the end (``own`` false), and
the framework's own call (``own`` true).
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
ID_TYPES = {"int64": torch.int64, "int32": torch.int32}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # One new token for each of 64 sequences: a lookup where latency is all.
        {"name": "embed-64-tokens", "op": "embed", "ids": 64, "rows": 32000, "dim": 4096,
         "table": "bf16", "out": "bf16", "id_type": "int64", "first": 0, "scale": 64.0,
         "spread": "zipf"},
        # A micro-batch of 4 x 2048 tokens through the 7B table.
        {"name": "embed-8k-tokens", "op": "embed", "ids": 8192, "rows": 32000, "dim": 4096,
         "table": "bf16", "out": "bf16", "id_type": "int64", "first": 0, "scale": 64.0,
         "spread": "zipf"},
        # fp32 master weights, an odd width, and a table that holds a slice of
        # the vocabulary (ids of other slices give zero rows).
        {"name": "embed-odd-slice", "op": "embed", "ids": 50021, "rows": 15013, "dim": 1023,
         "table": "fp32", "out": "bf16", "id_type": "int32", "first": 7001, "scale": 1.0,
         "spread": "uniform"},
        # A small model's step, added on top of an fp32 grad: launches count.
        {"name": "grad-512-tokens", "op": "embed_grad", "ids": 512, "rows": 2048, "dim": 256,
         "dy": "bf16", "out": "fp32", "id_type": "int64", "first": 0, "scale": 16.0,
         "accumulate": True, "padding": -1, "spread": "zipf"},
        # The micro-batch of 8192 tokens: the dense grad of the 7B table.
        {"name": "grad-8k-tokens", "op": "embed_grad", "ids": 8192, "rows": 32000, "dim": 4096,
         "dy": "bf16", "out": "bf16", "id_type": "int64", "first": 0, "scale": 64.0,
         "accumulate": False, "padding": -1, "spread": "zipf"},
        # Odd width, padding tokens, a slice of the vocabulary, fp16 under a
        # loss scale summed into fp32.
        {"name": "grad-odd-slice", "op": "embed_grad", "ids": 50021, "rows": 15013, "dim": 1023,
         "dy": "fp16", "out": "fp32", "id_type": "int32", "first": 7001, "scale": 1.0,
         "accumulate": True, "padding": 7001, "spread": "uniform"},
        # The widest model's table: 32768 tokens of width 12288.
        {"name": "grad-32k-wide", "op": "embed_grad", "ids": 32768, "rows": 32000, "dim": 12288,
         "dy": "bf16", "out": "bf16", "id_type": "int64", "first": 0, "scale": 1.0,
         "accumulate": False, "padding": 0, "spread": "zipf"},
        # Grads of three types in tensors that follow one another without gaps.
        {"name": "norm-mixed-300", "op": "norm", "tensors": 300, "max_log2": 19, "layout": 5,
         "blocks": 0, "width": 0, "ffn": 0, "grads": "mixed", "out": "none", "gap": 1,
         "loss_scale": 1024.0, "max_norm": 0.0, "plant": "none"},
        # 24 blocks of width 2048 with fp16 grads under a loss scale.
        {"name": "norm-24-blocks", "op": "norm", "tensors": 0, "max_log2": 0, "layout": 0,
         "blocks": 24, "width": 2048, "ffn": 8192, "grads": "fp16", "out": "none", "gap": 64,
         "loss_scale": 65536.0, "max_norm": 0.0, "plant": "none"},
        # Two blocks of width 256, fp32 grads clipped into bf16: latency.
        {"name": "clip-2-blocks", "op": "clip", "tensors": 0, "max_log2": 0, "layout": 0,
         "blocks": 2, "width": 256, "ffn": 1024, "grads": "fp32", "out": "bf16", "gap": 64,
         "loss_scale": 1.0, "max_norm": 1.0, "plant": "none"},
        # 4000 tensors of 1 to 2^20 elements without gaps, bf16 to bf16.
        {"name": "clip-ragged-4000", "op": "clip", "tensors": 4000, "max_log2": 20, "layout": 3,
         "blocks": 0, "width": 0, "ffn": 0, "grads": "bf16", "out": "same", "gap": 1,
         "loss_scale": 1.0, "max_norm": 1.0, "plant": "none"},
        # One block of width 12288: fp32 grads summed over micro-batches,
        # clipped and rounded to the bf16 grads that the step reads.
        {"name": "clip-wide-block", "op": "clip", "tensors": 0, "max_log2": 0, "layout": 0,
         "blocks": 1, "width": 12288, "ffn": 49152, "grads": "fp32", "out": "bf16", "gap": 64,
         "loss_scale": 1.0, "max_norm": 1.0, "plant": "none"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _dim(rng):
    """A width: a power of two, a multiple of 64 or anything."""
    d = _log(rng, 8, 12288)
    kind = rng.random()
    if kind < 0.25:
        d = 1 << (d.bit_length() - 1)
    elif kind < 0.6:
        d = max(64, d // 64 * 64)
    return d + 1 if d == 3072 else d


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "clip"])
    if op in ("embed", "embed_grad"):
        dim = _dim(rng)
        cap = 32768 * 12288  # elements of the largest listed case's token side
        ids = _log(rng, 1, max(1, min(131072, cap // dim)))
        rows = _log(rng, 2, max(2, min(131072, 32000 * 12288 // dim)))
        first = rng.choice([0, 0, 0, rows // 2 + 1])
        case = {"op": op, "ids": ids, "rows": rows, "dim": dim,
                "id_type": rng.choice(["int64", "int64", "int32"]), "first": first,
                "scale": rng.choice([1.0, math.sqrt(dim), 0.125]),
                "spread": rng.choice(["zipf", "zipf", "uniform", "one"])}
        if op == "embed":
            case["table"] = rng.choice(["bf16", "fp16", "fp32"])
            case["out"] = rng.choice([case["table"], "bf16", "fp32"])
        else:
            case["dy"] = rng.choice(["bf16", "fp16", "fp32"])
            case["out"] = rng.choice([case["dy"], "bf16", "fp32"])
            case["accumulate"] = rng.random() < 0.4
            case["padding"] = rng.choice([-1, -1, first])
        return case
    ragged = rng.random() < 0.6
    case = {"op": op, "tensors": 0, "max_log2": 0, "layout": 0, "blocks": 0, "width": 0,
            "ffn": 0}
    if ragged:
        case.update(tensors=_log(rng, 1, 4000), max_log2=rng.randint(8, 20),
                    layout=rng.randint(0, 1 << 20))
    else:
        width = _dim(rng) // 2 + 7
        most = max(1, 1_000_000_000 // (12 * width * width))
        case.update(blocks=_log(rng, 1, min(32, most)), width=width, ffn=4 * width)
    case["grads"] = rng.choice(["bf16", "fp16", "fp32", "mixed"])
    case["out"] = "none" if op == "norm" else rng.choice(["same", "bf16"])
    case["gap"] = rng.choice([64, 64, 1])
    # 16-bit floats of few exponent bits come with a loss scale.
    case["loss_scale"] = rng.choice([1024.0, 65536.0] if case["grads"] in ("fp16", "mixed")
                                    else [1.0, 1.0, 1024.0])
    case["max_norm"] = 0.0 if op == "norm" else rng.choice([1e-2, 1.0, 1e30])
    case["plant"] = rng.choice(["none"] * 7 + ["inf"])
    return case


# -------------------------------------------------------------------- inputs
class State:
    pass


def _randn(n, dtype, std, gen):
    """n values of N(0, std^2), drawn in parts so that little room is taken."""
    out = torch.empty(n, dtype=dtype, device="cuda")
    part = 1 << 27
    for at in range(0, n, part):
        m = min(part, n - at)
        out[at:at + m] = torch.randn(m, generator=gen, device="cuda") * std
    return out


def _ids(case, gen):
    """Token ids: text-like (rank r about as frequent as 1/r), uniform, or one
    token throughout.  A table that holds a slice of the vocabulary sees the
    ids of the whole one."""
    vocab = case["rows"] + 2 * case["first"]
    u = torch.rand(case["ids"], generator=gen, device="cuda", dtype=torch.float64)
    if case["spread"] == "zipf":
        ids = torch.exp(u * math.log(vocab + 1)).floor().long() - 1
    elif case["spread"] == "uniform":
        ids = (u * vocab).floor().long()
    else:
        ids = torch.zeros(case["ids"], dtype=torch.int64, device="cuda") + (
            u[:1] * vocab).floor().long()
    return ids.clamp_(0, vocab - 1).to(ID_TYPES[case["id_type"]])


def _sizes(case):
    if case["blocks"]:
        d, f = case["width"], case["ffn"]
        return [3 * d * d, d * d, d * f, f * d, d, d] * case["blocks"]
    rng = random.Random(case["layout"])
    return [max(1, int(2.0 ** (rng.random() * case["max_log2"]))) for _ in range(case["tensors"])]


def _kinds(case, n):
    if case["grads"] == "mixed":
        return [("bf16", "fp32", "fp16")[i % 3] for i in range(n)]
    return [case["grads"]] * n


def _layout(case):
    """[(type, elements with gaps, [(offset, size)])]: one flat buffer a type."""
    sizes = _sizes(case)
    kinds = _kinds(case, len(sizes))
    gap, found = case["gap"], []
    for kind in sorted(set(kinds)):
        at, spans = 0, []
        for k, n in zip(kinds, sizes):
            if k == kind:
                spans.append((at, n))
                at += (n + gap - 1) // gap * gap
        found.append((kind, at, spans))
    return found


def _out_kind(case, kind):
    return kind if case["out"] == "same" else case["out"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = State()
    s.case = case
    if case["op"] == "embed":
        s.table = _randn(case["rows"] * case["dim"], TYPES[case["table"]], 0.02, gen).view(
            case["rows"], case["dim"])
        s.ids = _ids(case, gen)
    elif case["op"] == "embed_grad":
        s.ids = _ids(case, gen)
        s.dy = _randn(case["ids"] * case["dim"], TYPES[case["dy"]], 1e-2, gen).view(
            case["ids"], case["dim"])
        n = case["rows"] * case["dim"]
        out = TYPES[case["out"]]
        # Added to: what a tied output head left there.  Else: last step's values.
        s.grad = _randn(n, out, 1e-3, gen).view(case["rows"], case["dim"])
    else:
        s.flats, s.grads, s.outs, s.out = [], [], [], []
        for kind, total, spans in _layout(case):
            flat = _randn(total, TYPES[kind], 1e-4 * case["loss_scale"], gen)
            if case["gap"] > 1:  # what lies between the tensors is zero
                ends = torch.tensor([(o + n, o + (n + case["gap"] - 1) // case["gap"]
                                      * case["gap"]) for o, n in spans])
                for lo, hi in ends[ends[:, 0] < ends[:, 1]].tolist():
                    flat[lo:hi] = 0
            s.flats.append(flat)
            s.grads += [flat[o:o + n] for o, n in spans]
            if case["op"] == "clip":
                to = torch.zeros(total, dtype=TYPES[_out_kind(case, kind)], device="cuda")
                s.outs.append(to)
                s.out += [to[o:o + n] for o, n in spans]
        if case["plant"] != "none":
            g = s.grads[seed % len(s.grads)]
            g[seed % g.numel()] = float(case["plant"])
    if own:
        import optimizer_step_gb300 as og
        s.og = og
        if case["op"] in ("norm", "clip"):
            s.clipper = og.GradClip(s.grads, out=s.out or None)
    return s


# -------------------------------------------------------------------- passes
def _plain_embed(s):
    c = s.case
    row = s.ids.long() - c["first"]
    held = (row >= 0) & (row < c["rows"])
    x = s.table[torch.where(held, row, 0)].float() * c["scale"]
    return torch.where(held[:, None], x, 0.0).to(TYPES[c["out"]])


def _plain_embed_grad(s):
    c = s.case
    row = s.ids.long() - c["first"]
    held = (row >= 0) & (row < c["rows"]) & (s.ids != c["padding"])
    x = torch.where(held[:, None], s.dy.float(), 0.0)
    total = torch.zeros(c["rows"], c["dim"], device="cuda")
    total.index_add_(0, torch.where(held, row, 0), x)
    total = total * c["scale"]
    if c["accumulate"]:
        total = total + s.grad.float()
    return s.grad.copy_(total)


def _plain_stats(s):
    c = s.case
    sums = torch.stack([f.float().square().sum() for f in s.flats])
    norm = sums.sum().sqrt() / c["loss_scale"]
    bad = ~torch.isfinite(norm)
    factor = torch.ones_like(norm)
    if c["max_norm"] > 0:
        factor = torch.where(norm > c["max_norm"], c["max_norm"] / norm, factor)
    factor = torch.where(bad, 0.0, factor / c["loss_scale"])
    return torch.stack([torch.where(bad, math.inf, norm), factor, bad.float()])


def _plain_clip(s):
    stats = _plain_stats(s)
    return {"stats": stats,
            "out": [to.copy_(torch.where(stats[2] != 0, to.float(), f.float() * stats[1]))
                    for f, to in zip(s.flats, s.outs)]}


def run(s):
    c = s.case
    op = c["op"]
    if op == "embed":
        if not own:
            return _plain_embed(s)
        return s.og.embed(s.table, s.ids, scale=c["scale"], first_row=c["first"],
                          out_dtype=TYPES[c["out"]])
    if op == "embed_grad":
        if not own:
            return _plain_embed_grad(s)
        return s.og.embed_grad(s.dy, s.ids, out=s.grad, scale=c["scale"], first_row=c["first"],
                               padding_id=c["padding"], accumulate=c["accumulate"])
    if op == "norm":
        return s.clipper.norm(loss_scale=c["loss_scale"]) if own else _plain_stats(s)
    if not own:
        return _plain_clip(s)
    return {"stats": s.clipper.clip(c["max_norm"], loss_scale=c["loss_scale"]),
            "out": list(s.outs)}


# -------------------------------------------------------- work, exact values
def work(case):
    if case["op"] in ("embed", "embed_grad"):
        n, d, rows = case["ids"], case["dim"], case["rows"]
        vocab = rows + 2 * case["first"]
        # Distinct rows that the ids name, as expected from their spread.
        if case["spread"] == "one":
            distinct = 1.0
        elif case["spread"] == "uniform":
            distinct = rows * -math.expm1(-n / vocab)
        else:
            lo, hi = case["first"], case["first"] + rows
            width = math.log(vocab + 1)
            step = max(1, (hi - lo) // 4096)
            distinct = sum(
                -math.expm1(n * math.log1p(-min(1 - 1e-12, math.log((k + 2) / (k + 1)) / width)))
                * min(step, hi - k) for k in range(lo, hi, step))
        distinct = min(distinct, n, rows)
        size = 8 if case["id_type"] == "int64" else 4
        if case["op"] == "embed":
            return {"bytes": n * size + n * d * SIZE[case["out"]]
                    + distinct * d * SIZE[case["table"]], "flops": n * d}
        grad = 2 * distinct if case["accumulate"] else rows
        return {"bytes": n * size + n * d * SIZE[case["dy"]] + grad * d * SIZE[case["out"]],
                "flops": n * d}
    sizes = _sizes(case)
    total = 0
    for kind, n in zip(_kinds(case, len(sizes)), sizes):
        total += n * SIZE[kind]
        if case["op"] == "clip":
            total += n * SIZE[_out_kind(case, kind)]
    return {"bytes": total, "flops": 2 * sum(sizes) + (sum(sizes) if case["out"] != "none" else 0)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        out = torch.zeros(case["ids"], case["dim"], dtype=torch.float64, device="cuda")
        at = torch.nonzero((s.ids >= case["first"])
                           & (s.ids < case["first"] + case["rows"])).flatten()
        out[at] = s.table.double().index_select(0, s.ids[at].long() - case["first"])
        return out.mul_(case["scale"])
    if case["op"] == "embed_grad":
        ids = s.ids.long()
        keep = torch.nonzero((ids >= case["first"]) & (ids < case["first"] + case["rows"])
                             & (ids != case["padding"])).flatten()
        keep = keep[torch.sort(ids[keep], stable=True).indices]
        counts = torch.bincount(ids[keep] - case["first"], minlength=case["rows"])
        total = torch.empty(case["rows"], case["dim"], dtype=torch.float64, device="cuda")
        for lo in range(0, case["dim"], 1024):
            part = s.dy[:, lo:lo + 1024].double().index_select(0, keep)
            sums = torch.segment_reduce(part, "sum", lengths=counts, axis=0, initial=0.0)
            total[:, lo:lo + 1024] = sums * case["scale"]
        return total.add_(s.grad.double()) if case["accumulate"] else total
    # The sum of squares, tensor by tensor.
    square = sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in s.grads)
    bad = not math.isfinite(square)
    norm = math.inf if bad else math.sqrt(square) / case["loss_scale"]
    coefficient = 1.0
    if 0 < case["max_norm"] < norm:
        coefficient = case["max_norm"] / norm
    factor = 0.0 if bad else coefficient / case["loss_scale"]
    stats = torch.tensor([norm, factor, float(bad)], dtype=torch.float64)
    if case["op"] == "norm":
        return stats
    return {"stats": stats,
            "out": [to.double() if bad else f.double() * factor
                    for f, to in zip(s.flats, s.outs)]}
