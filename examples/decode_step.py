"""The token operators together, as a serving loop and a training step use
them: draft tokens, verify them against the target's probabilities, extend
the paged cache's block tables, look the new tokens' embeddings up into
their slots; then a step on the embedding table.

    python examples/decode_step.py [--requests 8] [--drafts 4] [--steps 12]

The "models" are toys on one random embedding table (the target is a
softmax over the table's products with a context vector, the draft the same
over half of the columns). Everything else is the package: the
probabilities and drafted tokens come from row_stats, the random numbers
of the verification from a torch generator. A step makes no host
round trip; the loop ends with one.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import vocab_row_sampling_gb300 as drs  # noqa: E402


class PagedCache:
    """Embeddings of the requests' tokens in blocks of a shared pool."""

    def __init__(self, requests, width, block, blocks, max_blocks, capacity, dtype, device):
        i32 = dict(dtype=torch.int32, device=device)
        self.block, self.capacity = block, capacity
        self.rows = torch.zeros(blocks * block + 1, width, dtype=dtype, device=device)  # the last row takes padding
        self.lens = torch.zeros(requests, **i32)
        self.held = torch.zeros(requests, **i32)
        self.table = torch.zeros(requests, max_blocks, **i32)
        self.ring = torch.arange(blocks, **i32)
        self.state = torch.tensor([0, blocks], dtype=torch.int64, device=device)
        self.lacking = torch.zeros(1, **i32)

    def extend(self, new_lens):
        """Blocks and slots for new_lens more tokens per request; returns
        (request, offset in the request's new tokens, slot) per token."""
        out = drs.map_slots(self.lens, new_lens, self.held, self.table, self.block, self.ring, self.state, self.capacity)
        _, request, position, slot, self.held, self.state, lacking = out
        self.lacking += lacking
        b = request.long().clamp_min(0)
        offset = position - self.lens[b]
        self.lens = self.lens + new_lens
        return request, offset, slot

    def write(self, slot, rows):
        self.rows[torch.where(slot < 0, self.rows.shape[0] - 1, slot)] = rows


def distribution(context, table, temps, seed):
    """(sample, probabilities) of softmax(context table^T / T), one slot per row."""
    logits = (context.float() @ table.float().t()).contiguous()
    _, sample, _, probs = drs.row_stats(logits, temps, 1, seed, torch.bfloat16)
    return sample, probs


def decode(requests=8, drafts=4, steps=12, vocab=8192, width=256, block=16, seed=0):
    device = "cuda"
    g = torch.Generator(device=device).manual_seed(seed)
    scale = width**0.5
    table = (torch.randn(vocab, width, generator=g, device=device) * (0.4 / scale)).to(torch.bfloat16)
    half = width // 2
    temps = torch.full((requests * (drafts + 1),), 0.8, device=device)
    max_tokens = steps * (drafts + 1) + 1
    cache = PagedCache(requests, width, block, requests * (max_tokens // block + 1), max_tokens // block + 1,
                       requests * (drafts + 1), torch.bfloat16, device)
    cu = torch.arange(requests + 1, dtype=torch.int32, device=device) * drafts
    last = torch.randint(0, vocab, (requests,), generator=g, device=device)
    context = torch.zeros(requests, width, device=device)
    history, accepted_total = [], torch.zeros((), dtype=torch.int64, device=device)
    for step in range(steps):
        # draft: one token after the other from the first half of the columns
        seen, previous, drafted, q = [], last, [], []
        for j in range(drafts + 1):
            seen.append(context + drs.embed_tokens(table, previous, scale).float())
            if j < drafts:
                sample, probs = distribution(seen[j][:, :half] * 1.2, table[:, :half], temps[:requests], 1000 * step + j)
                drafted.append(sample)
                q.append(probs)
                previous = sample
        tokens = torch.stack(drafted, 1)                                    # [requests, drafts]
        q = torch.stack(q, 1).view(requests * drafts, vocab)
        # verify: the target's rows of every position, all at once
        _, p = distribution(torch.stack(seen, 1).view(-1, width), table, temps, 0)
        out, accepted = drs.verify_drafts(p, tokens.view(-1).contiguous(), cu,
                                          torch.rand(requests * drafts, generator=g, device=device),
                                          torch.rand(requests, generator=g, device=device), drafts, draft_probs=q)
        # extend the cache by the accepted drafts and the token after them
        request, offset, slot = cache.extend(accepted + 1)
        ids = torch.where(request >= 0, out[request.long().clamp_min(0), offset.long().clamp(0, drafts)], -1)
        rows = drs.embed_tokens(table, ids, scale)
        cache.write(slot, rows)
        last = out.gather(1, accepted.long()[:, None])[:, 0]
        # the context: a decaying sum of the request's new rows
        fresh = torch.zeros_like(context).index_add_(0, request.long().clamp_min(0), rows.float())
        context = 0.5 * context + 0.5 * fresh / (accepted + 1)[:, None]
        accepted_total += accepted.sum()
        history.append(out)
    return {"table": table, "scale": scale, "cache": cache, "tokens": torch.cat(history, 1),
            "accepted": accepted_total, "drafted": requests * drafts * steps, "context": context}


def train_step(run, targets, lr=0.1):
    """One step of the table on next-token prediction over the decoded
    tokens, the table tied on both sides: returns the gradient."""
    table, scale, vocab = run["table"], run["scale"], run["table"].shape[0]
    ids = torch.where(targets[:, :-1] >= 0, targets[:, :-1], -1).reshape(-1).contiguous()
    after = targets[:, 1:].reshape(-1)
    rows = drs.embed_tokens(table, ids, scale)
    logits = (rows.float() @ table.float().t()).contiguous()
    ok = (ids >= 0) & (after >= 0)
    temps = torch.ones(1, device=table.device)
    _, _, _, probs = drs.row_stats(logits, temps, logits.shape[0], 0, torch.bfloat16)
    d_logits = probs.float()
    d_logits[torch.arange(len(ids), device=ids.device), after.clamp_min(0)] -= 1.0
    d_logits *= (ok / ok.sum().clamp_min(1))[:, None]
    grad = d_logits.t() @ rows.float()                                      # the output side
    d_rows = (d_logits @ table.float()).to(torch.bfloat16)
    drs.embed_tokens_grad(d_rows, ids, scale, grad, accumulate=True)        # the input side
    table -= (lr * grad).to(table.dtype)
    return grad


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--steps", type=int, default=12)
    a = ap.parse_args(argv)
    drs.load(build_if_missing=True)
    run = decode(a.requests, a.drafts, a.steps)
    cache = run["cache"]
    print(f"{a.requests} requests, {a.steps} steps: {int(run['accepted'])} of {run['drafted']} drafted tokens accepted, "
          f"{int(cache.lens.sum())} tokens in {int(cache.held.sum())} blocks of {cache.block}, "
          f"{int(cache.state[1] - cache.state[0])} blocks free, {int(cache.lacking)} lacking")
    grad = train_step(run, run["tokens"])
    print(f"training step on the decoded tokens: gradient norm {float(grad.norm()):.4f}, "
          f"{int((grad != 0).any(1).sum())} of {grad.shape[0]} rows touched")
    return run


if __name__ == "__main__":
    main()
