"""Timed cases of the token operators: verification of drafted tokens, block tables and slot maps,
the embedding lookup and its gradient.

Each case is one call a serving or training step makes. `run` computes it in plain torch operations
(own = False) or through the package's entry points (own = True). Sizes follow the package's workloads
(vocabularies of 8192, 131072 and 262144 columns, canvases of 16 to 256 positions, 4 to 32 slots) or
are generic.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
DEVICE = "cuda"


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # One interactive request with four drafted tokens: latency.
        {"name": "verify one", "op": "verify", "requests": 1, "drafts": 4, "vocab": 131072, "pad": 0,
         "target": "bf16", "draft": "bf16"},
        # Drafts looked up in the prompt (no draft probabilities), fp32 probabilities, odd padded rows.
        {"name": "verify lookup", "op": "verify", "requests": 32, "drafts": 15, "vocab": 50001, "pad": 7,
         "target": "fp32", "draft": "none"},
        # A full serving batch, both sides' probabilities as the row statistics write them.
        {"name": "verify batch", "op": "verify", "requests": 256, "drafts": 5, "vocab": 262144, "pad": 0,
         "target": "bf16", "draft": "fp16"},
        # A decode step of 64 requests with up to 5 new tokens each, padded to a captured size.
        {"name": "slots decode", "op": "slots", "requests": 64, "new": 5, "prompts": 0, "prompt": 0,
         "context": 8192, "block": 16, "capacity": 512},
        # 32 slots that each open a canvas of 256 positions.
        {"name": "slots canvas", "op": "slots", "requests": 32, "new": 256, "prompts": 0, "prompt": 0,
         "context": 4096, "block": 64, "capacity": 8192},
        # A large mixed step: 4096 requests, most decoding, 16 with long prompts.
        {"name": "slots mixed", "op": "slots", "requests": 4096, "new": 4, "prompts": 16, "prompt": 14000,
         "context": 16384, "block": 32, "capacity": 262144},
        # One canvas of ids.
        {"name": "embed canvas", "op": "embed", "tokens": 256, "width": 2048, "vocab": 262144, "table": "bf16"},
        # Odd widths: rows that start off 16-byte boundaries.
        {"name": "embed odd", "op": "embed", "tokens": 5003, "width": 1283, "vocab": 50001, "table": "fp16"},
        # A large prompt batch.
        {"name": "embed prompts", "op": "embed", "tokens": 65536, "width": 4096, "vocab": 262144, "table": "bf16"},
        # A short training step on a small vocabulary, fp32 master gradient.
        {"name": "grad small", "op": "grad", "tokens": 2048, "width": 1024, "vocab": 8192, "out": "bf16",
         "table": "fp32"},
        # Odd sizes, the gradient in the table's 16-bit type.
        {"name": "grad odd", "op": "grad", "tokens": 10007, "width": 1283, "vocab": 131072, "out": "fp32",
         "table": "bf16"},
        # A training step on the full vocabulary.
        {"name": "grad large", "op": "grad", "tokens": 32768, "width": 2048, "vocab": 262144, "out": "bf16",
         "table": "fp32"},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["verify", "slots", "embed", "grad"])
    if op == "verify":
        vocab = _log(rng, 8192, 262144)
        vocab = vocab if rng.random() < 0.5 else -(-vocab // 64) * 64
        requests = _log(rng, 1, 256)
        drafts = _log(rng, 1, 16)
        while requests > 1 and requests * (drafts + 2) * vocab > 256 * 7 * 262144:
            requests //= 2
        return {"op": op, "requests": requests, "drafts": drafts, "vocab": vocab, "pad": rng.choice([0, 0, 64, 3]),
                "target": rng.choice(["bf16", "fp16", "fp32"]),
                "draft": rng.choice(["bf16", "fp16", "fp32", "none"])}
    if op == "slots":
        requests, new = _log(rng, 1, 4096), _log(rng, 1, 256)
        while requests * new > 200000:
            new = max(1, new // 2)
        prompts = rng.choice([0, 0, min(requests, 2), min(requests, 8)])
        prompt = _log(rng, 64, 6000) if prompts else 0
        most = requests * new + prompts * prompt
        return {"op": op, "requests": requests, "new": new, "prompts": prompts, "prompt": prompt,
                "context": _log(rng, 16, 16384), "block": rng.choice([1, 8, 16, 24, 32, 64, 128]),
                "capacity": most + rng.randrange(0, 64)}
    if op == "embed":
        tokens, width = _log(rng, 1, 65536), _log(rng, 64, 4096)
        width = width if rng.random() < 0.4 else -(-width // 64) * 64
        table = rng.choice(["bf16", "fp16", "fp32"])
        return {"op": op, "tokens": tokens if table != "fp32" else max(1, tokens // 2), "width": width,
                "vocab": _log(rng, 8192, 262144), "table": table}
    tokens, width = _log(rng, 16, 32768), _log(rng, 64, 2048)
    width = width if rng.random() < 0.4 else -(-width // 64) * 64
    return {"op": op, "tokens": tokens, "width": width, "vocab": _log(rng, 8192, 200000),
            "out": rng.choice(["bf16", "fp16", "fp32"]), "table": rng.choice(["fp32", "fp32", "bf16", "fp16"])}


# ------------------------------------------------------------------ the inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _frequent_ids(n, vocab, g):
    """Token ids whose frequency falls like 1/rank, spread over the vocabulary; the last few are padding (-1)."""
    u = torch.rand(n, generator=g, device=DEVICE, dtype=torch.float64)
    rank = torch.exp(u * math.log(vocab)).to(torch.int64).clamp(1, vocab) - 1
    ids = (rank * 1000003 + 17) % vocab
    ids[n - n // 64:] = -1
    return ids


def prepare(case, seed):
    g = _generator(seed)
    return {"verify": _prepare_verify, "slots": _prepare_slots, "embed": _prepare_embed,
            "grad": _prepare_grad}[case["op"]](case, g)


def _prepare_verify(case, g):
    requests, most, vocab = case["requests"], case["drafts"], case["vocab"]
    stride = vocab + case["pad"]
    # how many tokens each request has drafted: mostly `drafts`, some fewer, some none
    count = torch.randint(0, most + 1, (requests,), generator=g, device=DEVICE)
    count[torch.rand(requests, generator=g, device=DEVICE) < 0.5] = most
    if requests == 1:
        count[:] = most
    cu = torch.zeros(requests + 1, dtype=torch.int32, device=DEVICE)
    cu[1:] = count.cumsum(0)
    total = max(1, int(cu[-1]))
    target = torch.zeros(total + requests, stride, dtype=DTYPES[case["target"]], device=DEVICE)
    draft = None if case["draft"] == "none" else torch.zeros(total, stride, dtype=DTYPES[case["draft"]], device=DEVICE)
    tokens = torch.zeros(total, dtype=torch.int64, device=DEVICE)
    owner = torch.repeat_interleave(torch.arange(requests, device=DEVICE), count)
    if owner.numel() == 0:
        owner = torch.zeros(1, dtype=torch.int64, device=DEVICE)

    def logits(n):
        x = 3.0 * torch.randn(n, vocab, generator=g, device=DEVICE)
        x[torch.arange(n, device=DEVICE), torch.randint(0, vocab, (n,), generator=g, device=DEVICE)] += 8.0
        return x

    # rows in groups that bound the memory: the draft's distribution is a noisy copy of the target's
    group = max(1, (1 << 26) // vocab)
    for r in range(0, total, group):
        n = min(group, total - r)
        x = logits(n)
        rows = torch.arange(r, r + n, device=DEVICE)
        target[rows + owner[r:r + n], :vocab] = torch.softmax(x, 1).to(target.dtype)
        y = x + torch.randn(x.shape, generator=g, device=DEVICE)
        if draft is not None:
            draft[rows, :vocab] = torch.softmax(y, 1).to(draft.dtype)
        noise = -torch.log(-torch.log(torch.rand(x.shape, generator=g, device=DEVICE).clamp_min(1e-20)))
        # looked-up drafts are likely tokens; drafted ones are sampled
        tokens[r:r + n] = (y + noise).argmax(1) if draft is not None else (y + 0.25 * noise).argmax(1)
    last = cu[1:].long() + torch.arange(requests, device=DEVICE)
    for r in range(0, requests, group):
        target[last[r:r + group], :vocab] = torch.softmax(logits(min(group, requests - r)), 1).to(target.dtype)
    return {"op": "verify", "target": target[:, :vocab], "draft": None if draft is None else draft[:, :vocab],
            "tokens": tokens, "cu": cu, "most": most,
            "accept_u": torch.rand(total, generator=g, device=DEVICE),
            "sample_u": torch.rand(requests, generator=g, device=DEVICE),
            "out_tokens": torch.empty(requests, most + 1, dtype=torch.int64, device=DEVICE),
            "out_accepted": torch.empty(requests, dtype=torch.int32, device=DEVICE)}


def _prepare_slots(case, g):
    requests, block, capacity = case["requests"], case["block"], case["capacity"]
    lens = torch.randint(1, case["context"] + 1, (requests,), generator=g, device=DEVICE)
    new = torch.randint(1, case["new"] + 1, (requests,), generator=g, device=DEVICE)
    if case["new"] >= 64:
        new[:] = case["new"]  # canvases are opened whole
    long = case["prompts"]
    if long:  # new prompts: nothing cached yet
        lens[:long] = 0
        new[:long] = torch.randint(case["prompt"] // 2, case["prompt"] + 1, (long,), generator=g, device=DEVICE)
    kind = torch.rand(requests, generator=g, device=DEVICE)
    if requests > 8:  # some have ended and give their blocks back, some wait this step
        ended = (kind < 0.05) & (torch.arange(requests, device=DEVICE) >= long)
        had = torch.where(ended, lens, lens + (kind * 4 * block).long() * (kind > 0.8))
        lens = torch.where(ended, 0, lens)
        new = torch.where(ended | ((kind > 0.05) & (kind < 0.1)), 0, new)
    else:
        had = lens
    held = (had + block - 1) // block
    widest = (case["context"] + max(case["new"], 4 * block) + case["prompt"] + block - 1) // block + 1
    # a pool with room for every request at its longest
    total, most = int(held.sum()), max(case["new"], 4 * block)
    spare = requests * ((case["context"] + most) // block + 2) + long * (case["prompt"] // block + 1) + 64 - total
    pool = torch.randperm(total + spare, generator=g, device=DEVICE).int()
    table = torch.zeros(requests, widest, dtype=torch.int32, device=DEVICE)
    inside = torch.arange(widest, device=DEVICE) < held[:, None]
    table[inside] = pool[:total]
    # the ring of free blocks starts anywhere
    at = int(torch.randint(0, total + spare, (1,), generator=g, device=DEVICE))
    ring = torch.zeros(total + spare, dtype=torch.int32, device=DEVICE)
    ring[(at + torch.arange(spare, device=DEVICE)) % ring.numel()] = pool[total:]
    state = torch.tensor([at, at + spare], dtype=torch.int64, device=DEVICE)
    i32 = dict(dtype=torch.int32, device=DEVICE)
    return {"op": "slots", "lens": lens.int(), "new": new.int(), "held": held.int(), "table": table, "block": block,
            "ring": ring, "state": state, "capacity": capacity,
            "out": (torch.empty(requests + 1, **i32), torch.empty(capacity, **i32), torch.empty(capacity, **i32),
                    torch.empty(capacity, dtype=torch.int64, device=DEVICE), torch.empty(requests, **i32),
                    torch.empty(2, dtype=torch.int64, device=DEVICE), torch.empty(1, **i32))}


def _prepare_embed(case, g):
    dtype = DTYPES[case["table"]]
    table = torch.randn(case["vocab"], case["width"], generator=g, device=DEVICE, dtype=dtype)
    table *= 1.0 / math.sqrt(case["width"])
    return {"op": "embed", "table": table, "ids": _frequent_ids(case["tokens"], case["vocab"], g),
            "scale": math.sqrt(case["width"]),
            "out": torch.empty(case["tokens"], case["width"], dtype=dtype, device=DEVICE)}


def _prepare_grad(case, g):
    grad = torch.randn(case["tokens"], case["width"], generator=g, device=DEVICE, dtype=DTYPES[case["out"]])
    return {"op": "grad", "grad": grad, "ids": _frequent_ids(case["tokens"], case["vocab"], g),
            "scale": math.sqrt(case["width"]),
            "table": torch.empty(case["vocab"], case["width"], dtype=DTYPES[case["table"]], device=DEVICE)}


# --------------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    return {"verify": _plain_verify, "slots": _plain_slots, "embed": _plain_embed,
            "grad": _plain_grad}[state["op"]](state)


def _run_own(s):
    import vocab_row_sampling_gb300 as drs
    if s["op"] == "verify":
        return drs.verify_drafts(s["target"], s["tokens"], s["cu"], s["accept_u"], s["sample_u"], s["most"],
                                 draft_probs=s["draft"], out_tokens=s["out_tokens"], out_accepted=s["out_accepted"])
    if s["op"] == "slots":
        out = drs.map_slots(s["lens"], s["new"], s["held"], s["table"], s["block"], s["ring"], s["state"],
                            s["capacity"], out=s["out"])
        return tuple(out) + (s["table"], s["ring"])
    if s["op"] == "embed":
        return drs.embed_tokens(s["table"], s["ids"], s["scale"], out=s["out"])
    return drs.embed_tokens_grad(s["grad"], s["ids"], s["scale"], s["table"])


def _plain_verify(s):
    target, draft, tokens, cu, most = s["target"], s["draft"], s["tokens"], s["cu"].long(), s["most"]
    requests, vocab = cu.numel() - 1, target.shape[1]
    b = torch.arange(requests, device=cu.device)
    count = cu[1:] - cu[:-1]
    j = torch.arange(most, device=cu.device)
    inside = j < count[:, None]
    row = torch.where(inside, cu[:-1, None] + j, 0)
    x = tokens[row]
    # accepted where u q < p: the product of two 32-bit numbers is exact in 64
    p = target[torch.where(inside, row + b[:, None], 0), x].double()
    q = 1.0 if draft is None else draft[row, x].double()
    ok = inside & (s["accept_u"][row].double() * q < p)
    accepted = ok.long().cumprod(1).sum(1)
    whole = accepted == count
    here = torch.where(whole, 0, cu[:-1] + accepted)
    pr = target[cu[:-1] + b + accepted].float()
    if draft is None:
        at = torch.arange(vocab, device=cu.device)
        w = torch.where((at == tokens[here][:, None]) & ~whole[:, None], 0.0, pr)
    else:
        w = (pr - torch.where(whole[:, None], 0.0, draft[here].float())).clamp_min(0)
    w = torch.where((w > 0).any(1, keepdim=True), w, pr)
    # the sums that the sampled number is held against, in 64 bits
    sums = w.double().cumsum(1)
    first = (sums <= (s["sample_u"].double() * sums[:, -1])[:, None]).sum(1)
    first = torch.minimum(first, (w > 0).long().mul(torch.arange(1, vocab + 1, device=cu.device)).amax(1) - 1)
    k = torch.arange(most + 1, device=cu.device)
    drafted = torch.cat([x, x[:, :1]], 1)
    out = torch.where(k < accepted[:, None], drafted, torch.where(k == accepted[:, None], first[:, None], -1))
    return out, accepted.int()


def _plain_slots(s):
    lens, new, held, table, block = s["lens"].long(), s["new"].long(), s["held"].long(), s["table"], s["block"]
    ring, state, capacity = s["ring"], s["state"], s["capacity"]
    requests, widest = table.shape
    size = ring.numel()
    need = ((lens + new + block - 1) // block).clamp_max(widest)
    take, give = (need - held).clamp_min(0), (held - need).clamp_min(0)
    upto = take.cumsum(0)
    served = upto <= state[1] - state[0]
    now = torch.where(served, need, torch.minimum(need, held))
    col = torch.arange(widest, device=table.device)
    taken = (col >= held[:, None]) & (col < now[:, None])
    nth = (upto - take)[:, None] + col - held[:, None]
    table = torch.where(taken, ring[(state[0] + nth) % size], table)
    back = (col >= need[:, None]) & (col < held[:, None])
    nth = (give.cumsum(0) - give)[:, None] + col - need[:, None]
    ring = torch.cat([ring, ring[:1]])  # one more place for what is not given back
    ring = ring.scatter(0, torch.where(back, (state[1] + nth) % size, size).flatten(), table.flatten())[:size]
    cu = torch.cat([new[:1] * 0, new.cumsum(0)]).clamp_max(capacity)
    t = torch.arange(capacity, device=table.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    inside = b < requests
    b = b.clamp_max(requests - 1)
    position = lens[b] + t - cu[b]
    c = position // block
    place = table[b, c.clamp_max(widest - 1)].long() * block + position % block
    slot = torch.where(inside & (c < now[b]), place, -1)
    lacking = (((lens + new + block - 1) // block) - now).clamp_min(0).sum()
    state = state + torch.stack([torch.where(served, take, 0).sum(), give.sum()])
    return (cu.int(), torch.where(inside, b, -1).int(), torch.where(inside, position, 0).int(), slot, now.int(), state,
            lacking[None].int(), table, ring)


def _plain_embed(s):
    ids = s["ids"]
    inside = (ids >= 0) & (ids < s["table"].shape[0])
    rows = s["table"][torch.where(inside, ids, 0)].float() * s["scale"]
    return torch.where(inside[:, None], rows, 0.0).to(s["table"].dtype)


def _plain_grad(s):
    ids, (vocab, width) = s["ids"], s["table"].shape
    inside = (ids >= 0) & (ids < vocab)
    sums = torch.zeros(vocab + 1, width, dtype=torch.float32, device=ids.device)
    sums.index_add_(0, torch.where(inside, ids, vocab), s["grad"].float())
    return (sums[:vocab] * s["scale"]).to(s["table"].dtype)


# ------------------------------------------------------------- 64-bit definition

def exact(case, seed):
    """The embedding's values and gradients in 64 bits. The other operators return whole numbers."""
    if case["op"] not in ("embed", "grad"):
        return None
    s = prepare(case, seed)
    ids = s["ids"]
    keep = ((ids >= 0) & (ids < case["vocab"])).nonzero().flatten()
    out = torch.zeros(case["tokens"] if case["op"] == "embed" else case["vocab"], case["width"], dtype=torch.float64,
                      device=DEVICE)
    if case["op"] == "embed":
        out[keep] = torch.index_select(s["table"], 0, ids[keep]).double().mul_(s["scale"])
    else:
        out.index_put_((ids[keep],), s["grad"][keep].double().mul_(s["scale"]), accumulate=True)
    return out


# ------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "verify":
        # one target row each, and the draft's row where a draft is rejected (about 0.62 are accepted)
        requests, most, vocab = case["requests"], case["drafts"], case["vocab"]
        passed = [0.62 ** k for k in range(most + 1)]
        whole = passed[most] if requests == 1 else 0.5 * passed[most] + 0.5 * sum(passed) / (most + 1)
        q = BYTES.get(case["draft"], 0) * (1 - whole)
        elements = requests * vocab
        return {"bytes": elements * (BYTES[case["target"]] + q) + requests * (8 * (most + 1) + 20 * most + 12),
                "flops": 2 * elements}
    if case["op"] == "slots":
        mean = case["new"] if case["new"] >= 64 else (1 + case["new"]) / 2
        tokens = min(case["capacity"], case["requests"] * mean + case["prompts"] * case["prompt"] * 0.75)
        blocks = case["requests"] + tokens / case["block"]
        return {"bytes": case["requests"] * 20 + blocks * 4 + 2 * 4 * tokens / case["block"] + 16 * case["capacity"],
                "flops": 4 * tokens}
    elements = case["tokens"] * case["width"]
    if case["op"] == "embed":
        # the distinct rows among ids of frequency 1/rank: the integral of 1 - exp(-n p(rank)) over the ranks
        top, steps = math.log(case["vocab"]), 256
        ranks = [math.exp(top * (i + 0.5) / steps) for i in range(steps)]
        distinct = sum(r * (1 - math.exp(-case["tokens"] / (r * top))) for r in ranks) * top / steps
        read = min(case["tokens"], distinct) * case["width"]
        return {"bytes": (read + elements) * BYTES[case["table"]] + 8 * case["tokens"], "flops": elements}
    return {"bytes": elements * BYTES[case["out"]] + case["vocab"] * case["width"] * BYTES[case["table"]]
            + 8 * case["tokens"], "flops": elements + case["vocab"] * case["width"]}
