"""Cases that measure layer norm and the distillation loss, with their gradients.

Four operators: layer norm (``ln``), its backward pass with the reduction of
the weight's and the bias's gradient (``ln_grad``), the loss against a teacher's
top logits and the true labels (``loss``), and that loss together with its
gradient for the student's logits (``loss_grad``).  Each has a plain form in
elementary torch operations, 32 bits wide and rounded once at the end (``own``
false), and the framework's own call (``own`` true).
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
ID_TYPES = {"int64": torch.int64, "int32": torch.int32}
ID_SIZE = {"int64": 8, "int32": 4}
EPS = 1e-5
IGNORE = -100


# --------------------------------------------------------------------- cases
def listed():
    return [
        # One new token for each of 64 sequences: latency is all.
        {"name": "ln-64-tokens", "op": "ln", "rows": 64, "dim": 4096, "x": "bf16", "y": "bf16",
         "params": "bf16", "pad": 0},
        # A micro-batch of 4 x 2048 tokens of the 7B width.
        {"name": "ln-8k-tokens", "op": "ln", "rows": 8192, "dim": 4096, "x": "bf16", "y": "bf16",
         "params": "bf16", "pad": 0},
        # An odd width: an fp32 residual stream, normed into bf16.
        {"name": "ln-odd-width", "op": "ln", "rows": 50021, "dim": 1023, "x": "fp32",
         "y": "bf16", "params": "fp32", "pad": 0},
        # A small model's step, weight grads added to fp32 sums: launches count.
        {"name": "ln-grad-512-tokens", "op": "ln_grad", "rows": 512, "dim": 256, "x": "bf16",
         "y": "bf16", "params": "bf16", "sums": "fp32", "accumulate": True, "pad": 0},
        # The micro-batch of 8192 tokens backwards.
        {"name": "ln-grad-8k-tokens", "op": "ln_grad", "rows": 8192, "dim": 4096, "x": "bf16",
         "y": "bf16", "params": "bf16", "sums": "bf16", "accumulate": False, "pad": 0},
        # Odd width, fp16 grads under a loss scale, added to fp32 sums.
        {"name": "ln-grad-odd-width", "op": "ln_grad", "rows": 50021, "dim": 1023, "x": "fp16",
         "y": "fp16", "params": "fp32", "sums": "fp32", "accumulate": True, "pad": 0},
        # The widest model: 32768 tokens of width 12288.
        {"name": "ln-grad-32k-wide", "op": "ln_grad", "rows": 32768, "dim": 12288, "x": "bf16",
         "y": "bf16", "params": "bf16", "sums": "fp32", "accumulate": False, "pad": 0},
        # 64 positions scored against the teacher, no gradient: latency.
        {"name": "loss-64-tokens", "op": "loss", "rows": 64, "vocab": 32000, "top": 32,
         "logits": "bf16", "teacher": "bf16", "id_type": "int64", "temperature": 1.0,
         "soft": 1.0, "hard": 0.0, "pad": 0},
        # A validation batch: 8192 positions, both terms at two temperatures.
        {"name": "loss-8k-tokens", "op": "loss", "rows": 8192, "vocab": 32000, "top": 64,
         "logits": "bf16", "teacher": "bf16", "id_type": "int32", "temperature": 2.0,
         "soft": 0.5, "hard": 0.5, "pad": 0},
        # A small model's micro-batch: fp32 logits, bf16 grads.
        {"name": "loss-grad-512-tokens", "op": "loss_grad", "rows": 512, "vocab": 2048, "top": 8,
         "logits": "fp32", "grad": "bf16", "teacher": "fp32", "id_type": "int64",
         "temperature": 1.0, "soft": 0.5, "hard": 0.5, "loss_scale": 1.0, "pad": 0},
        # The 7B head's micro-batch: 8192 x 32000 logits, 64 of the teacher's.
        {"name": "loss-grad-8k-tokens", "op": "loss_grad", "rows": 8192, "vocab": 32000,
         "top": 64, "logits": "bf16", "grad": "bf16", "teacher": "bf16", "id_type": "int32",
         "temperature": 2.0, "soft": 0.5, "hard": 0.5, "loss_scale": 1.0, "pad": 0},
        # A wide odd vocabulary, fp16 under a loss scale: no row is aligned.
        {"name": "loss-grad-wide-odd", "op": "loss_grad", "rows": 1021, "vocab": 131071,
         "top": 100, "logits": "fp16", "grad": "fp16", "teacher": "fp16", "id_type": "int32",
         "temperature": 1.0, "soft": 0.9, "hard": 0.1, "loss_scale": 1024.0, "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A power of two, a multiple of 64 or anything."""
    d = _log(rng, lo, hi)
    kind = rng.random()
    if kind < 0.25:
        d = 1 << (d.bit_length() - 1)
    elif kind < 0.6:
        d = max(64, d // 64 * 64)
    return d


def draw(rng):
    op = rng.choice(["ln", "ln_grad", "loss", "loss_grad"])
    case = {"op": op}
    if op in ("ln", "ln_grad"):
        dim = _width(rng, 8, 12288)
        case.update(rows=_log(rng, 1, min(131072, 32768 * 12288 // dim)), dim=dim)
        case["x"] = rng.choice(["bf16", "fp16", "fp32"])
        case["y"] = rng.choice([case["x"], case["x"], "bf16", "fp32"])
        case["params"] = rng.choice([case["x"], "bf16", "fp32", "none"])
        if op == "ln_grad":
            case["sums"] = "fp32" if case["params"] == "none" else rng.choice(
                [case["params"], "fp32"])
            case["accumulate"] = rng.random() < 0.4
    else:
        vocab = _width(rng, 32, 262144)
        case.update(rows=_log(rng, 1, min(16384, 8192 * 32000 // vocab)), vocab=vocab,
                    top=_log(rng, 1, min(256, vocab // 2)))
        case["logits"] = rng.choice(["bf16", "fp16", "fp32"])
        case["teacher"] = rng.choice(["bf16", "fp16", "fp32"])
        case["id_type"] = rng.choice(["int64", "int32"])
        case["temperature"] = rng.choice([1.0, 1.0, 2.0, 0.7, 4.0])
        case["soft"], case["hard"] = rng.choice([(1.0, 0.0), (0.5, 0.5), (0.9, 0.1), (0.0, 1.0)])
        if op == "loss_grad":
            case["grad"] = rng.choice([case["logits"], case["logits"], "bf16", "fp32"])
            case["loss_scale"] = 1024.0 if case["grad"] == "fp16" else 1.0
    # Rows may be parts of longer ones.
    case["pad"] = rng.choice([0, 0, 0, 8, 3])
    return case


# -------------------------------------------------------------------- inputs
class State:
    pass


def _rows(case, width, dtype):
    """Rows of `width` elements with `pad` others between them."""
    return torch.empty(case["rows"], width + case["pad"], dtype=dtype, device="cuda")[:, :width]


def _fill(to, values):
    """to[i] = values(first row, rows), a part at a time so that little room is taken."""
    part = max(1, (1 << 27) // max(1, to.shape[1]))
    for at in range(0, to.shape[0], part):
        n = min(part, to.shape[0] - at)
        to[at:at + n] = values(at, n)
    return to


def _prepare_ln(s, case, gen):
    n, d = case["rows"], case["dim"]
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    # A residual stream: channels of their own mean and spread, a few of them large.
    spread = torch.exp(0.5 * rand(d))
    spread[:: 97] *= 10.0
    centre = 0.5 * rand(d) + 0.2
    s.x = _fill(_rows(case, d, TYPES[case["x"]]), lambda at, m: rand(m, d) * spread + centre)
    s.weight = s.bias = None
    if case["params"] != "none":
        s.weight = (1.0 + 0.2 * rand(d)).to(TYPES[case["params"]])
        s.bias = (0.1 * rand(d)).to(TYPES[case["params"]])
    if case["op"] == "ln":
        return
    scale = 1024.0 if case["y"] == "fp16" else 1.0  # 16-bit grads of few exponent bits
    s.dy = _fill(_rows(case, d, TYPES[case["y"]]), lambda at, m: rand(m, d) * (1e-2 * scale))
    # What the forward pass keeps: each row's mean and 1 / sqrt(variance + eps).
    s.stats = torch.empty(2, n, device="cuda")
    for at in range(0, n, 4096):
        x = s.x[at:at + 4096].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        s.stats[0, at:at + 4096] = mean
        s.stats[1, at:at + 4096] = (var + EPS).rsqrt()
    if case["accumulate"]:  # what earlier micro-batches left there
        s.weight_sums = (scale * rand(d)).to(TYPES[case["sums"]])
        s.bias_sums = (scale * rand(d)).to(TYPES[case["sums"]])


def _prepare_loss(s, case, gen):
    n, v, k = case["rows"], case["vocab"], case["top"]
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    uniform = lambda *shape: torch.rand(*shape, generator=gen, device="cuda",
                                        dtype=torch.float64)
    # The teacher's k tokens: distinct, anywhere in the vocabulary, most likely first.
    start = (uniform(n, 1) * v).long()
    step = 1 + (uniform(n, 1) * max(1, v // k - 1)).long()
    order = torch.arange(k, device="cuda")
    ids = (start + order * step) % v
    teacher = 9.0 - 7.0 * torch.sqrt((order + 0.5) / k) + rand(n, k)
    teacher = torch.sort(teacher, dim=1, descending=True).values
    # The student: noise over the vocabulary, and what it has learned of the teacher.
    s.logits = _fill(_rows(case, v, TYPES[case["logits"]]), lambda at, m: rand(m, v) * 1.5)
    s.logits.scatter_(1, ids, (0.5 * teacher + rand(n, k)).to(s.logits.dtype))
    # The true token: mostly one of the teacher's; one in 16 rows is padding.
    pick = (uniform(n) ** 4 * k).long().clamp_(0, k - 1)
    labels = ids.gather(1, pick[:, None])[:, 0]
    labels = torch.where(uniform(n) < 0.2, (uniform(n) * v).long().clamp_(0, v - 1), labels)
    padding = uniform(n) < 1.0 / 16.0
    labels = torch.where(padding, IGNORE, labels)
    # Some rows have fewer of the teacher's tokens than there is room for.
    fewer = torch.where(uniform(n, 1) < 0.1, (uniform(n, 1) * k).long(), k)
    ids = torch.where(order < fewer, ids, -1)
    kind = ID_TYPES[case["id_type"]]
    s.ids, s.labels = ids.to(kind), labels.to(kind)
    s.teacher = teacher.to(TYPES[case["teacher"]])
    if case["op"] == "loss_grad":  # a mean over the rows that count, times the loss scale
        used = (~padding).float()
        s.row_grad = used * (case["loss_scale"] / used.sum().clamp(min=1.0))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = State()
    s.case = case
    (_prepare_ln if case["op"] in ("ln", "ln_grad") else _prepare_loss)(s, case, gen)
    return s


# -------------------------------------------------------------------- passes
def _plain_ln(s):
    x = s.x.float()
    mean = x.mean(dim=1, keepdim=True)
    centred = x - mean
    rstd = (centred.square().mean(dim=1, keepdim=True) + EPS).rsqrt()
    y = centred * rstd
    if s.weight is not None:
        y = y * s.weight.float() + s.bias.float()
    return {"y": y.to(TYPES[s.case["y"]]), "stats": torch.stack([mean[:, 0], rstd[:, 0]])}


def _plain_ln_grad(s):
    c = s.case
    mean, rstd = s.stats[0][:, None], s.stats[1][:, None]
    dy = s.dy.float()
    xhat = (s.x.float() - mean) * rstd
    g = dy if s.weight is None else dy * s.weight.float()
    dx = rstd * (g - g.mean(dim=1, keepdim=True) - xhat * (g * xhat).mean(dim=1, keepdim=True))
    weight, bias = (dy * xhat).sum(dim=0), dy.sum(dim=0)
    if c["accumulate"]:
        weight = s.weight_sums.copy_(weight + s.weight_sums.float())
        bias = s.bias_sums.copy_(bias + s.bias_sums.float())
    kind = TYPES[c["sums"]]
    return {"x": dx.to(s.x.dtype), "weight": weight.to(kind), "bias": bias.to(kind)}


def _plain_loss(s, with_grad):
    c = s.case
    v, tau = c["vocab"], c["temperature"]
    z = s.logits.float()
    z = z - z.max(dim=1, keepdim=True).values
    used = s.labels != IGNORE
    loss = torch.zeros(c["rows"], device="cuda")
    grad = 0.0
    if c["soft"]:
        e = torch.exp(z / tau)
        total = e.sum(dim=1, keepdim=True)
        held = (s.ids >= 0) & used[:, None]
        ids = torch.where(held, s.ids, 0).long()
        t = torch.where(held, s.teacher.float() / tau, -math.inf)
        some = held.any(dim=1, keepdim=True)
        t = t - torch.where(some, t.max(dim=1, keepdim=True).values, 0.0)
        size = torch.exp(t).sum(dim=1, keepdim=True)
        size = torch.where(some, size, 1.0)
        p = torch.exp(t) / size
        log_p = t - size.log()
        log_q = z.gather(1, ids) / tau - total.log()
        kl = torch.where(held, p * (log_p - log_q), 0.0).sum(dim=1)
        loss = loss + (c["soft"] * tau * tau) * kl
        if with_grad:
            grad = torch.where(some, e / total, 0.0).scatter_add_(1, ids, -p)
            grad = grad * (c["soft"] * tau)
    if c["hard"]:
        e = torch.exp(z)
        total = e.sum(dim=1, keepdim=True)
        label = torch.where(used, s.labels, 0).long()[:, None]
        log_s = (z.gather(1, label) - total.log())[:, 0]
        loss = loss - torch.where(used, c["hard"] * log_s, 0.0)
        if with_grad:
            one = torch.full_like(label, -1, dtype=torch.float32)
            grad = grad + (e / total).scatter_add_(1, label, one) * c["hard"]
    if not with_grad:
        return loss
    grad = torch.where(used[:, None], grad * s.row_grad[:, None], 0.0)
    return {"loss": loss, "grad": grad.to(TYPES[c["grad"]])}


def run(s):
    c = s.case
    op = c["op"]
    if not own:
        if op == "ln":
            return _plain_ln(s)
        return _plain_ln_grad(s) if op == "ln_grad" else _plain_loss(s, op == "loss_grad")
    import optimizer_step_gb300 as og
    if op == "ln":
        y, stats = og.layer_norm(s.x, s.weight, s.bias, eps=EPS, stats=True,
                                 out_dtype=TYPES[c["y"]])
        return {"y": y, "stats": stats}
    if op == "ln_grad":
        if c["accumulate"]:
            dx, weight, bias = og.layer_norm_grad(
                s.dy, s.x, s.weight, s.stats, weight_grad=s.weight_sums, bias_grad=s.bias_sums,
                accumulate=True)
        else:
            dx, weight, bias = og.layer_norm_grad(s.dy, s.x, s.weight, s.stats,
                                                  param_dtype=TYPES[c["sums"]])
        return {"x": dx, "weight": weight, "bias": bias}
    if op == "loss":
        return og.distill_loss(s.logits, s.ids, s.teacher, s.labels, soft_weight=c["soft"],
                               hard_weight=c["hard"], temperature=c["temperature"],
                               ignore_id=IGNORE)
    loss, grad = og.distill_loss_grad(s.logits, s.ids, s.teacher, s.labels, row_grad=s.row_grad,
                                      soft_weight=c["soft"], hard_weight=c["hard"],
                                      temperature=c["temperature"], ignore_id=IGNORE,
                                      dtype=TYPES[c["grad"]])
    return {"loss": loss, "grad": grad}


# -------------------------------------------------------- work, exact values
def work(case):
    n = case["rows"]
    if case["op"] in ("ln", "ln_grad"):
        d = case["dim"]
        params = 0 if case["params"] == "none" else d * SIZE[case["params"]]
        if case["op"] == "ln":
            return {"bytes": n * d * (SIZE[case["x"]] + SIZE[case["y"]]) + 2 * params + 8 * n,
                    "flops": 8 * n * d}
        sums = 2 * d * SIZE[case["sums"]] * (2 if case["accumulate"] else 1)
        return {"bytes": n * d * (2 * SIZE[case["x"]] + SIZE[case["y"]]) + params + sums + 8 * n,
                "flops": 14 * n * d}
    v, k = case["vocab"], case["top"]
    # One row in 16 is padding: its logits need not be read.
    read = n * v * SIZE[case["logits"]] * 15 // 16 + n * (ID_SIZE[case["id_type"]] + 4)
    if case["soft"]:
        read += n * k * (ID_SIZE[case["id_type"]] + SIZE[case["teacher"]])
    terms = (case["soft"] > 0) + (case["hard"] > 0 and (case["temperature"] != 1.0
                                                         or not case["soft"]))
    # A subtraction, a product, an exponential and a sum for each element and distribution.
    if case["op"] == "loss":
        return {"bytes": read, "flops": 4 * n * v * terms}
    return {"bytes": read + n * v * SIZE[case["grad"]] + 4 * n, "flops": 7 * n * v * terms}


def _exact_ln(s, case):
    n, d = case["rows"], case["dim"]
    y = torch.empty(n, d, dtype=torch.float64, device="cuda")
    stats = torch.empty(2, n, dtype=torch.float64, device="cuda")
    part = max(1, (1 << 26) // d)
    for at in range(0, n, part):
        x = s.x[at:at + part].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        stats[0, at:at + part], stats[1, at:at + part] = mean, 1.0 / torch.sqrt(var + EPS)
        x = (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None]
        if s.weight is not None:
            x = torch.addcmul(s.bias.double(), x, s.weight.double())
        y[at:at + part] = x
    return {"y": y, "stats": stats}


def _exact_ln_grad(s, case):
    n, d = case["rows"], case["dim"]
    dx = torch.empty(n, d, dtype=torch.float64, device="cuda")
    weight = torch.zeros(d, dtype=torch.float64, device="cuda")
    bias = torch.zeros(d, dtype=torch.float64, device="cuda")
    gamma = 1.0 if s.weight is None else s.weight.double()
    part = max(1, (1 << 26) // d)
    for at in range(0, n, part):
        mean, rstd = s.stats[:, at:at + part, None].double()
        xhat = s.x[at:at + part].double().sub_(mean).mul_(rstd)
        dy = s.dy[at:at + part].double()
        bias += dy.sum(0)
        weight += torch.einsum("nd,nd->d", dy, xhat)
        g = dy * gamma
        along = torch.einsum("nd,nd->n", g, xhat)[:, None] / d
        dx[at:at + part] = (g - g.sum(1, keepdim=True) / d - along * xhat) * rstd
    if case["accumulate"]:
        weight += s.weight_sums.double()
        bias += s.bias_sums.double()
    return {"x": dx, "weight": weight, "bias": bias}


def _exact_loss(s, case):
    n, v, tau = case["rows"], case["vocab"], case["temperature"]
    with_grad = case["op"] == "loss_grad"
    loss = torch.zeros(n, dtype=torch.float64, device="cuda")
    grad = torch.zeros(n, v, dtype=torch.float64, device="cuda") if with_grad else None
    part = max(1, (1 << 26) // v)
    for at in range(0, n, part):
        rows = slice(at, min(n, at + part))
        z = s.logits[rows].double()
        label, ids = s.labels[rows].long(), s.ids[rows].long()
        live = (label != IGNORE).double()
        # The teacher's distribution over its own tokens; none of them: no term.
        p = torch.where(ids >= 0, s.teacher[rows].double() / tau, -math.inf)
        p = torch.nan_to_num(torch.softmax(p, dim=1), nan=0.0)
        at_ids, at_label = ids.clamp(min=0), label.clamp(min=0)[:, None]
        if case["soft"]:
            lq = torch.log_softmax(z / tau, dim=1)
            terms = torch.special.xlogy(p, p) - p * lq.gather(1, at_ids)
            loss[rows] += live * case["soft"] * tau ** 2 * terms.sum(1)
            if with_grad:
                up = live * s.row_grad[rows].double() * case["soft"] * tau
                grad[rows] += lq.exp_().mul_((up * p.sum(1))[:, None])
                grad[rows].scatter_add_(1, at_ids, -up[:, None] * p)
            del lq
        if case["hard"]:
            ls = torch.log_softmax(z, dim=1)
            loss[rows] -= live * case["hard"] * ls.gather(1, at_label)[:, 0]
            if with_grad:
                up = (live * s.row_grad[rows].double() * case["hard"])[:, None]
                grad[rows] += ls.exp_().mul_(up)
                grad[rows].scatter_add_(1, at_label, -up)
    return {"loss": loss, "grad": grad} if with_grad else loss


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("ln", "ln_grad"):
        return (_exact_ln if case["op"] == "ln" else _exact_ln_grad)(s, case)
    return _exact_loss(s, case)
