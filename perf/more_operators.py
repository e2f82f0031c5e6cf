"""Timed cases of the scoring and training operators: log probabilities of given tokens with entropy, rank and top
alternatives, their gradient, and dropout from the counter-based generator with its gradient.

Each case is one call a scoring or training step makes. `run` computes it in plain torch operations
(own = False) or through the package's entry points (own = True). Sizes follow the package's workloads
(vocabularies of 8192, 131072 and 262144 columns, canvases of 16 to 256 positions) or are generic.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
IDS = {32: torch.int32, 64: torch.int64}
DEVICE = "cuda"


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # The logprob of one sampled token with its alternatives: latency.
        {"name": "logprobs one", "op": "logprobs", "rows": 1, "vocab": 262144, "pad": 0, "type": "bf16", "k": 20,
         "ids": 64, "canvas": 0, "masked": False},
        # One canvas of fp32 rows, a temperature per 64 positions.
        {"name": "logprobs canvas", "op": "logprobs", "rows": 256, "vocab": 262144, "pad": 0, "type": "fp32", "k": 20,
         "ids": 64, "canvas": 64, "masked": False},
        # Odd padded rows under a grammar's mask.
        {"name": "logprobs odd", "op": "logprobs", "rows": 1003, "vocab": 50001, "pad": 7, "type": "fp16", "k": 5,
         "ids": 32, "canvas": 0, "masked": True},
        # The prompt tokens of a scoring batch.
        {"name": "logprobs prompts", "op": "logprobs", "rows": 4096, "vocab": 262144, "pad": 0, "type": "bf16", "k": 20,
         "ids": 64, "canvas": 0, "masked": False},
        # A short training step on a small vocabulary.
        {"name": "logprobs grad small", "op": "logprobs_grad", "rows": 128, "vocab": 8192, "pad": 0, "type": "bf16",
         "out": "bf16", "ids": 64, "canvas": 0, "entropy": False},
        # Odd rows, an entropy term, temperatures, the gradient in fp32.
        {"name": "logprobs grad odd", "op": "logprobs_grad", "rows": 777, "vocab": 50001, "pad": 3, "type": "bf16",
         "out": "fp32", "ids": 32, "canvas": 16, "entropy": True},
        # A training step on the full vocabulary.
        {"name": "logprobs grad large", "op": "logprobs_grad", "rows": 4096, "vocab": 262144, "pad": 0, "type": "bf16",
         "out": "bf16", "ids": 64, "canvas": 0, "entropy": False},
        # The embeddings of one canvas: latency.
        {"name": "dropout canvas", "op": "dropout", "rows": 256, "width": 2048, "pad": 0, "type": "bf16", "out": "bf16",
         "residual": False, "p": 0.1},
        # Odd widths: rows that start off 16-byte boundaries, added to a residual.
        {"name": "dropout odd", "op": "dropout", "rows": 5003, "width": 1283, "pad": 0, "type": "fp16", "out": "fp16",
         "residual": True, "p": 0.3},
        # A training batch, added to its residual.
        {"name": "dropout large", "op": "dropout", "rows": 65536, "width": 4096, "pad": 0, "type": "bf16", "out": "bf16",
         "residual": True, "p": 0.1},
        # The gradient of a short step, from an fp32 residual stream to 16-bit activations.
        {"name": "dropout grad small", "op": "dropout_grad", "rows": 2048, "width": 1024, "pad": 0, "type": "bf16",
         "out": "fp32", "p": 0.5},
        # The gradient of a training batch.
        {"name": "dropout grad large", "op": "dropout_grad", "rows": 32768, "width": 4096, "pad": 0, "type": "bf16",
         "out": "bf16", "p": 0.1},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_grad", "dropout", "dropout_grad"])
    pick = lambda *of: rng.choice(of)  # noqa: E731
    if op in ("logprobs", "logprobs_grad"):
        vocab, rows = _log(rng, 8192, 262144), _log(rng, 1, 4096)
        vocab = vocab if rng.random() < 0.5 else -(-vocab // 64) * 64
        case = {"op": op, "rows": rows, "vocab": vocab, "pad": pick(0, 0, 64, 3), "type": pick("bf16", "fp16", "fp32")}
        case.update(ids=pick(32, 64), canvas=pick(0, 0, 1, 16, 256))
        if op == "logprobs":
            case.update(k=pick(0, 1, 5, 20, 32), masked=rng.random() < 0.3)
        else:
            case.update(out=pick(case["type"], "bf16", "fp32"), entropy=rng.random() < 0.4)
        while case["rows"] > 1 and case["rows"] * vocab * BYTES[case["type"]] > 4096 * 262144 * 2:
            case["rows"] //= 2
        while case["rows"] > 1 and op == "logprobs_grad" and \
                case["rows"] * vocab * (BYTES[case["type"]] + BYTES[case["out"]]) > 4096 * 262144 * 4:
            case["rows"] //= 2
        return case
    rows, width = _log(rng, 1, 65536), _log(rng, 64, 4096)
    width = width if rng.random() < 0.4 else -(-width // 64) * 64
    case = {"op": op, "rows": rows, "width": width, "pad": pick(0, 0, 0, 5, 64), "type": pick("bf16", "fp16", "fp32")}
    case.update(out=pick(case["type"], case["type"], "fp32"), p=pick(0.05, 0.1, 0.25, 0.5))
    if op == "dropout":
        case.update(residual=rng.random() < 0.5)
    while case["rows"] > 1 and case["rows"] * width * (BYTES[case["type"]] + 2 * BYTES[case["out"]]) > 65536 * 4096 * 6:
        case["rows"] //= 2
    return case


# ------------------------------------------------------------------ the inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _rows(rows, width, pad, dtype):
    """[rows, width] inside rows of width + pad elements."""
    return torch.zeros(rows, width + pad, dtype=dtype, device=DEVICE)[:, :width]


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] in ("logprobs", "logprobs_grad"):
        return _prepare_logprobs(case, g)
    return _prepare_dropout(case, g)


def _prepare_logprobs(case, g):
    rows, vocab = case["rows"], case["vocab"]
    logits = _rows(rows, vocab, case["pad"], DTYPES[case["type"]])
    ids = torch.randint(0, vocab, (rows,), generator=g, device=DEVICE)
    likely = torch.rand(rows, generator=g, device=DEVICE) < 0.7
    masked = torch.rand(vocab, generator=g, device=DEVICE) < 0.8 if case.get("masked") else None
    group = max(1, (1 << 28) // vocab)
    for r in range(0, rows, group):  # groups that bound the memory
        n = min(group, rows - r)
        x = 3.0 * torch.randn(n, vocab, generator=g, device=DEVICE)
        top = torch.randint(0, vocab, (n,), generator=g, device=DEVICE)
        x[torch.arange(n, device=DEVICE), top] += 8.0
        ids[r:r + n] = torch.where(likely[r:r + n], top, ids[r:r + n])  # mostly what the model expects
        if masked is not None:
            masked_now = masked.expand(n, vocab).clone()
            masked_now[torch.arange(n, device=DEVICE), ids[r:r + n]] = False
            x.masked_fill_(masked_now, -math.inf)
        logits[r:r + n] = x.to(logits.dtype)
    if rows > 64:  # the batch ends in padding
        ids[rows - rows // 64:] = -1
    ids = ids.to(IDS[case["ids"]])
    canvas = case["canvas"]
    temps = 0.5 + torch.rand(-(-rows // canvas), generator=g, device=DEVICE) if canvas else None
    f32 = dict(dtype=torch.float32, device=DEVICE)
    s = {"op": case["op"], "logits": logits, "ids": ids, "temps": temps, "canvas": max(1, canvas)}
    if case["op"] == "logprobs":
        k = s["k"] = case["k"]
        s["out"] = (torch.empty(rows, **f32), torch.empty(rows, **f32),
                    torch.empty(rows, dtype=torch.int32, device=DEVICE), torch.empty(rows, 2, **f32),
                    torch.empty(rows, k, dtype=torch.int32, device=DEVICE), torch.empty(rows, k, **f32))
        return s
    # what the forward call has left, and the gradients that arrive
    s["norm"], s["entropy"] = torch.zeros(rows, 2, **f32), torch.zeros(rows, **f32)
    for r in range(0, rows, group):
        x = logits[r:r + group].float()
        top = x.amax(1)
        t = (x - top[:, None]) / _temperature(s, r, x.shape[0])
        e = t.exp()
        total = e.sum(1, dtype=torch.float64)
        s["norm"][r:r + group] = torch.stack([top, total.log().float()], 1)
        s["entropy"][r:r + group] = (total.log() - (e * t).sum(1, dtype=torch.float64) / total).float()
    s["grad_logprob"] = -torch.rand(rows, generator=g, device=DEVICE) - 0.5
    s["grad_entropy"] = 0.01 * torch.randn(rows, generator=g, device=DEVICE) if case["entropy"] else None
    s["grad"] = _rows(rows, vocab, case["pad"], DTYPES[case["out"]])
    return s


def _prepare_dropout(case, g):
    rows, width, pad = case["rows"], case["width"], case["pad"]
    backward = case["op"] == "dropout_grad"

    def filled(name):
        t = _rows(rows, width, pad, DTYPES[name])
        t.copy_(torch.randn(rows, width, generator=g, device=DEVICE, dtype=torch.float32))
        return t

    first, last = (case["out"], case["type"]) if backward else (case["type"], case["out"])
    return {"op": case["op"], "x": filled(first), "p": case["p"], "row0": rows,
            "seed": torch.randint(0, 2**62, (1,), generator=g, device=DEVICE),
            "residual": filled(case["out"]) if case.get("residual") else None,
            "out": _rows(rows, width, pad, DTYPES[last])}


# --------------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    return {"logprobs": _plain_logprobs, "logprobs_grad": _plain_logprobs_grad, "dropout": _plain_dropout,
            "dropout_grad": _plain_dropout}[state["op"]](state)


def _run_own(s):
    import vocab_row_sampling_gb300 as drs
    if s["op"] == "logprobs":
        return drs.token_logprobs(s["logits"], s["ids"], s["k"], temps=s["temps"], canvas_len=s["canvas"], out=s["out"])
    if s["op"] == "logprobs_grad":
        return drs.token_logprobs_grad(s["logits"], s["ids"], s["norm"], s["grad_logprob"], entropy=s["entropy"],
                                       grad_entropy=s["grad_entropy"], temps=s["temps"], canvas_len=s["canvas"],
                                       out=s["grad"])
    if s["op"] == "dropout":
        return drs.dropout(s["x"], s["p"], s["seed"], residual=s["residual"], row0=s["row0"], out=s["out"])
    return drs.dropout_grad(s["x"], s["p"], s["seed"], row0=s["row0"], out=s["out"])


def _temperature(s, first, rows):
    """The rows' temperatures as a column."""
    if s["temps"] is None:
        return 1.0
    at = (first + torch.arange(rows, device=s["temps"].device)) // s["canvas"]
    return s["temps"][at].clamp_min(1e-10)[:, None]


def _plain_logprobs(s):
    ids, k = s["ids"].long(), s["k"]
    rows, vocab = s["logits"].shape
    inside = (ids >= 0) & (ids < vocab)
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    t = (x - top) / _temperature(s, 0, rows)
    e = t.exp()
    total = e.sum(1, dtype=torch.float64)
    log_sum = total.log().float()
    weighted = torch.where(e > 0, e * t, 0.0).sum(1, dtype=torch.float64)
    entropy = (total.log() - weighted / total).float()
    at = torch.where(inside, ids, 0)[:, None]
    logprob = t.gather(1, at)[:, 0] - log_sum
    rank = 1 + (x > x.gather(1, at)).sum(1)
    # the k largest, ties to the lower column: integers that grow with (value, -column)
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * 2**32 - torch.arange(vocab, device=x.device)
    best = (-torch.topk(order, k).values) & (2**32 - 1) if k else order[:, :0]
    best_lp = t.gather(1, best) - log_sum[:, None]
    one, none = inside, torch.zeros((), device=x.device)
    return (torch.where(one, logprob, none), torch.where(one, entropy, none), torch.where(one, rank, 0).int(),
            torch.where(one[:, None], torch.stack([top[:, 0], log_sum], 1), none),
            torch.where(one[:, None], best, -1).int(), torch.where(one[:, None], best_lp, -math.inf))


def _plain_logprobs_grad(s):
    ids = s["ids"].long()
    rows, vocab = s["logits"].shape
    inside = (ids >= 0) & (ids < vocab)
    te = _temperature(s, 0, rows)
    lp = (s["logits"].float() - s["norm"][:, :1]) / te - s["norm"][:, 1:]
    p = lp.exp()
    g = s["grad_logprob"][:, None]
    grad = -g * p
    if s["grad_entropy"] is not None:
        grad = grad - s["grad_entropy"][:, None] * torch.where(p > 0, p * (lp + s["entropy"][:, None]), 0.0)
    grad = grad + torch.where(torch.arange(vocab, device=ids.device) == ids[:, None], g, 0.0)
    return torch.where(inside[:, None], grad / te, 0.0).to(s["grad"].dtype)


def _philox(counter, key):
    """Philox4x32-10 on 32-bit words held in 64-bit integers: products wrap, their bits are right."""
    low = 0xFFFFFFFF
    c0, c1, c2, c3 = counter
    k0, k1 = key
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return c0, c1, c2, c3


def _plain_dropout(s):
    x, low = s["x"], 0xFFFFFFFF
    rows, width = x.shape
    group = torch.arange(-(-width // 8), device=x.device).expand(rows, -1)
    row = (s["row0"] + torch.arange(rows, device=x.device))[:, None].expand_as(group)
    # counters of their own: the sampler's noise has 0 in the second word
    words = _philox((group, torch.full_like(group, 0x64726F70), row & low, row >> 32),
                    (s["seed"] & low, (s["seed"] >> 32) & low))
    halves = torch.stack([h for w in words for h in (w & 0xFFFF, w >> 16)], 2).view(rows, -1)[:, :width]
    dropped = int(s["p"] * 65536 + 0.5)
    out = torch.where(halves >= dropped, x.float() * (65536 / (65536 - dropped)), 0.0)
    if s.get("residual") is not None:
        out = out + s["residual"].float()
    return out.to(s["out"].dtype)


# ------------------------------------------------------------- 64-bit definition

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(s)
    if case["op"] == "logprobs_grad":
        return _exact_logprobs_grad(s)
    return _exact_dropout(s)


def _distribution(s, first, last):
    """The rows' logarithms of softmax(x / T), their logsumexp relative to the largest logit, and that logit."""
    x = s["logits"][first:last].double()
    if s["temps"] is not None:
        slot = torch.arange(first, last, device=x.device).div(s["canvas"], rounding_mode="floor")
        scale = s["temps"].double()[slot].clamp(min=1e-10).unsqueeze(1)
    else:
        scale = torch.ones(1, 1, dtype=torch.float64, device=x.device)
    largest = x.max(dim=1, keepdim=True).values
    x.sub_(largest).div_(scale)
    log_sum = torch.logsumexp(x, 1, keepdim=True)
    return x.sub_(log_sum), log_sum, largest, scale


def _exact_logprobs(s):
    rows, vocab = s["logits"].shape
    parts = []
    for first in range(0, rows, 256):
        last = min(rows, first + 256)
        lp, log_sum, largest, _ = _distribution(s, first, last)
        ids = s["ids"][first:last].long()
        keep = ((ids >= 0) & (ids < vocab)).unsqueeze(1)
        entropy = torch.special.entr(lp.exp()).sum(1, keepdim=True)
        logprob = lp.gather(1, ids.clamp(0, vocab - 1).unsqueeze(1))
        # stable order: equal logits by their columns
        best = torch.sort(s["logits"][first:last], dim=1, descending=True, stable=True).indices[:, :s["k"]] \
            if s["k"] else ids.new_zeros(last - first, 0)
        value = s["logits"][first:last].gather(1, ids.clamp(0, vocab - 1).unsqueeze(1))
        rank = (s["logits"][first:last] > value).sum(1, keepdim=True) + 1
        parts.append((logprob.masked_fill(~keep, 0).squeeze(1), entropy.masked_fill(~keep, 0).squeeze(1),
                      rank.masked_fill(~keep, 0).squeeze(1).int(),
                      torch.cat([largest, log_sum], 1).masked_fill(~keep, 0),
                      best.masked_fill(~keep, -1).int(), lp.gather(1, best).masked_fill(~keep, -math.inf)))
    return tuple(torch.cat(column) for column in zip(*parts))


def _exact_logprobs_grad(s):
    rows, vocab = s["logits"].shape
    out = torch.empty(rows, vocab, dtype=torch.float64, device=DEVICE)
    for first in range(0, rows, 256):
        last = min(rows, first + 256)
        lp, _, _, scale = _distribution(s, first, last)
        ids = s["ids"][first:last].long()
        keep = (ids >= 0) & (ids < vocab)
        g = s["grad_logprob"][first:last].double().unsqueeze(1)
        p = lp.exp()
        part = -(p * g)
        if s["grad_entropy"] is not None:
            plogp = -torch.special.entr(p)
            part -= s["grad_entropy"][first:last].double().unsqueeze(1) * (plogp - p * plogp.sum(1, keepdim=True))
        part.scatter_add_(1, ids.clamp(0, vocab - 1).unsqueeze(1), g)
        out[first:last] = part.div_(scale).masked_fill_(~keep.unsqueeze(1), 0)
    return out


def _exact_dropout(s):
    rows, width = s["x"].shape
    groups = (width + 7) // 8
    half = 0xFFFF

    def times(c, m):
        """High and low words of c m from 16-bit halves: no product passes 48 bits."""
        lower, upper = (c & half) * m, (c >> 16) * m
        total = upper + (lower >> 16)
        return total >> 16, ((total & half) << 16) | (lower & half)

    out = torch.empty(rows, width, dtype=torch.float64, device=DEVICE)
    dropped = math.floor(s["p"] * 2**16 + 0.5)
    seed = int(s["seed"])
    for first in range(0, rows, 8192):
        last = min(rows, first + 8192)
        at = torch.arange(s["row0"] + first, s["row0"] + last, device=DEVICE).view(-1, 1)
        zero = torch.zeros(last - first, groups, dtype=torch.int64, device=DEVICE)
        w = [zero + torch.arange(groups, device=DEVICE), zero + 0x64726F70, zero + (at % 2**32), zero + at // 2**32]
        for i in range(10):
            ka = (seed % 2**32 + i * 0x9E3779B9) % 2**32
            kb = (seed // 2**32 + i * 0xBB67AE85) % 2**32
            (high0, low0), (high2, low2) = times(w[0], 0xD2511F53), times(w[2], 0xCD9E8D57)
            w = [high2 ^ w[1] ^ ka, low2, high0 ^ w[3] ^ kb, low0]
        kept = torch.empty(last - first, groups, 8, dtype=torch.bool, device=DEVICE)
        for i in range(8):
            kept[:, :, i] = (w[i // 2] >> (16 * (i % 2))) % 2**16 >= dropped
        part = s["x"][first:last].double() * kept.view(last - first, -1)[:, :width] / (1 - dropped / 2**16)
        out[first:last] = part if s["residual"] is None else part + s["residual"][first:last].double()
    return out


# ------------------------------------------------------------------------- work

def work(case):
    if case["op"] in ("logprobs", "logprobs_grad"):
        rows = case["rows"] - (case["rows"] // 64 if case["rows"] > 64 else 0)
        elements = rows * case["vocab"]
        if case["op"] == "logprobs":
            # the rows that have a token are read once: largest, exponential, two sums and a comparison per column
            return {"bytes": elements * BYTES[case["type"]] + case["rows"] * (case["ids"] // 8 + 20 + 8 * case["k"]),
                    "flops": 7 * elements}
        return {"bytes": elements * BYTES[case["type"]] + case["rows"] * case["vocab"] * BYTES[case["out"]]
                + case["rows"] * (case["ids"] // 8 + 16), "flops": (7 if case["entropy"] else 5) * elements}
    elements = case["rows"] * case["width"]
    arrays = BYTES[case["type"]] + BYTES[case["out"]] * (2 if case.get("residual") else 1)
    # ten rounds of two products and four bitwise operations per eight elements, a comparison and a product each
    return {"bytes": elements * arrays + 8, "flops": elements * (60 / 8 + 2)}
