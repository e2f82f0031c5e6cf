"""The training step's operators together: its gradients against autograd in 64 bits on the same mask, and the step
captured into a graph against the step called."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu
U = 2.0**-24


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_step
    train_step.drs.load(build_if_missing=True)
    return train_step


def batch(tokens, vocab):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    ids, targets = (torch.randint(0, vocab, (tokens,), generator=g, device="cuda") for _ in range(2))
    ids[-1] = targets[-2:] = -1
    ids[1] = ids[0]
    return ids, targets, torch.tensor([77], device="cuda")


def reference(m, ids, targets, mask, keep, entropy_weight):
    """Loss and gradients by autograd in 64 bits, and what the magnitudes of their sums are at most."""
    w = {k: m[k].double().requires_grad_() for k in ("table", "layer", "head")}
    one = (ids >= 0)[:, None]
    rows = torch.where(one, w["table"][ids.clamp_min(0)] * m["scale"], 0.0)
    hidden = rows + mask * (rows @ w["layer"]) / keep
    lp = torch.log_softmax(hidden @ w["head"].t(), 1)
    logprob = lp.gather(1, targets.clamp_min(0)[:, None])[:, 0]
    entropy = -(lp.exp() * lp).sum(1)
    weight = (targets >= 0) / (targets >= 0).sum()
    loss = -(weight * (logprob + entropy_weight * entropy)).sum()
    loss.backward()
    with torch.no_grad():
        p = lp.exp()
        d = weight[:, None] * (torch.zeros_like(p).scatter_(1, targets.clamp_min(0)[:, None], 1.0) + p
                               + entropy_weight * p * (lp.abs() + entropy[:, None]))
        d_hidden = d @ w["head"].abs()
        d_branch = mask * d_hidden / keep
        d_rows = d_hidden + d_branch @ w["layer"].abs().t()
        table = torch.zeros_like(w["table"]).index_add_(0, ids.clamp_min(0), torch.where(one, d_rows, 0.0)) * m["scale"]
        big_hidden = rows.abs() + mask * (rows.abs() @ w["layer"].abs()) / keep
        # a logit is off by its product's roundings, and every p by a multiple of e to that
        logit = (big_hidden @ w["head"].abs().t()).amax()
    most = {"table": table, "layer": rows.abs().t() @ d_branch, "head": d.t() @ big_hidden}
    return loss.detach(), {k: w[k].grad for k in w}, most, float(logit)


@pytest.mark.parametrize("tokens,vocab,width", [(7, 97, 24), (64, 1000, 64), (33, 4099, 40)])
def test_gradients_of_a_step(example, tokens, vocab, width):
    """Tolerance: products and sums of n terms are off by n U of their magnitudes, at most four of them lie on a way
    (n: the longest, which is the vocabulary); the probabilities by the logits' errors, 2 (width + 8) U of a logit's
    magnitude, and by those of the scoring (1e-5 and less at these sizes)."""
    drs = example.drs
    m = example.model(vocab, width, seed=tokens)
    ids, targets, seed = batch(tokens, vocab)
    mask = (drs.dropout(torch.ones(tokens, width, device="cuda"), 0.1, seed) != 0).double()
    assert 0 < float(mask.mean()) < 1
    loss, grads = example.gradients(m, ids, targets, seed)
    keep = 1 - int(0.1 * 65536 + 0.5) / 65536
    want, ref, most, logit = reference(m, ids, targets, mask, keep, 0.01)
    rel = 4 * (vocab + width + tokens) * U + 2 * (width + 8) * U * logit + 1e-5
    assert abs(float(loss) - float(want)) <= rel * (1 + abs(float(want)))
    for name in ref:
        off = (grads[name].double() - ref[name]).abs()
        assert (off <= rel * most[name] + 1e-30).all(), (name, float((off / (most[name] + 1e-30)).max()), rel)


def test_captured_steps_equal_called_ones(example):
    """Every replay draws the mask of its own seed; the step's own operators give equal bits on equal calls, the products
    are the same library calls on both sides."""
    ids, targets, seed = batch(48, 1000)
    called, replayed = example.model(1000, 64), example.model(1000, 64)
    other = seed.clone()
    example.step(example.model(1000, 64), ids, targets, other.clone())  # before the capture: everything is loaded
    graph = torch.cuda.CUDAGraph()
    start = {k: replayed[k].clone() for k in ("table", "layer", "head")}
    with torch.cuda.graph(graph):
        loss = example.step(replayed, ids, targets, other)
    for k, v in start.items():
        replayed[k].copy_(v)
    for _ in range(4):
        want = example.step(called, ids, targets, seed)
        graph.replay()
        torch.cuda.synchronize()
        assert int(seed) == int(other) and torch.isfinite(loss)
        assert abs(float(loss) - float(want)) <= 1e-4 * abs(float(want))
    for k in start:
        assert torch.allclose(called[k], replayed[k], rtol=1e-4, atol=1e-5), k


def test_the_example_runs(example):
    m, losses = example.main(["--tokens", "64", "--vocab", "512", "--width", "32", "--steps", "3"])
    assert len(losses) == 6 and all(torch.isfinite(x) for x in losses)
