"""Training steps on the package's operators together: the embedding lookup, a
layer whose output goes through dropout onto the residual, the log
probabilities of the next tokens with an entropy term, and the gradients of
all of them back into the table.

    python examples/train_step.py [--tokens 256] [--vocab 8192] [--width 256] [--steps 20]

Only the matrix products are torch's. The backward pass keeps no probabilities
and no mask: the logits' gradient is written over the logits from the norm
that the scoring call has left, and the mask is drawn again. The seed
lives on the GPU, so that the whole step replays from a CUDA graph and every
replay draws another mask.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import vocab_row_sampling_gb300 as drs  # noqa: E402


def model(vocab, width, dtype=torch.float32, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    new = lambda *shape: torch.randn(*shape, generator=g, device=device) / width**0.5  # noqa: E731
    return {"table": new(vocab, width).to(dtype), "layer": new(width, width).to(dtype), "head": new(vocab, width).to(dtype),
            "scale": width**0.5}


def gradients(m, ids, targets, seed, p=0.1, entropy_weight=0.01):
    """(loss, gradients by name) of the mean over the rows with a target of -logprob - entropy_weight entropy.
    ids and targets: int64 [tokens], -1 for padding; seed: int64 [1] on the GPU."""
    table, layer, head, scale = m["table"], m["layer"], m["head"], m["scale"]
    rows = drs.embed_tokens(table, ids, scale)
    hidden = drs.dropout(rows @ layer, p, seed, residual=rows)
    logits = hidden @ head.t()
    logprob, entropy, _, norm, _, _ = drs.token_logprobs(logits, targets)
    weight = (targets >= 0) / (targets >= 0).sum().clamp_min(1)
    loss = -(weight * (logprob + entropy_weight * entropy)).sum()
    d_logits = drs.token_logprobs_grad(logits, targets, norm, -weight, entropy=entropy,
                                       grad_entropy=-entropy_weight * weight, out=logits)
    d_hidden = d_logits @ head
    d_branch = drs.dropout_grad(d_hidden, p, seed)
    d_rows = d_hidden + d_branch @ layer.t()
    d_table = drs.embed_tokens_grad(d_rows, ids, scale, torch.empty_like(table))
    return loss, {"table": d_table, "layer": rows.t() @ d_branch, "head": d_logits.t() @ hidden}


def step(m, ids, targets, seed, lr=0.5):
    """One step of gradient descent; the seed moves on."""
    loss, grads = gradients(m, ids, targets, seed)
    for name, grad in grads.items():
        m[name] -= lr * grad
    seed += 1
    return loss


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=256)
    ap.add_argument("--vocab", type=int, default=8192)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    drs.load(build_if_missing=True)
    m = model(a.vocab, a.width)
    g = torch.Generator(device="cuda").manual_seed(1)
    text = torch.randint(0, a.vocab, (a.tokens + 1,), generator=g, device="cuda")
    ids, targets, seed = text[:-1].contiguous(), text[1:].contiguous(), torch.zeros(1, dtype=torch.int64, device="cuda")
    losses = [step(m, ids, targets, seed) for _ in range(3)]  # before the capture: everything is loaded
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step(m, ids, targets, seed)
    for _ in range(a.steps):
        graph.replay()
        losses.append(loss.clone())
    print("loss " + " ".join(f"{float(x):.3f}" for x in losses))
    return m, losses


if __name__ == "__main__":
    main()
