"""The example that runs the token operators together: the cache it leaves
holds the embeddings of the tokens it returned, block by block, and the
training step's gradient is the sum of both sides of the tied table."""
import os
import sys

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_step
    return decode_step


@pytest.mark.parametrize("requests,drafts,steps,block", [(1, 1, 3, 16), (8, 4, 12, 16), (33, 7, 5, 8)])
def test_decoding_fills_the_cache(example, requests, drafts, steps, block):
    example.drs.load(build_if_missing=True)
    run = example.decode(requests, drafts, steps, vocab=2048, width=64, block=block, seed=requests)
    cache, tokens = run["cache"], run["tokens"].cpu().numpy()
    lens, held, table = (t.cpu().numpy() for t in (cache.lens, cache.held, cache.table))
    assert int(cache.lacking) == 0
    assert np.array_equal(lens, (tokens >= 0).sum(1)) and np.array_equal(held, -(-lens // block))
    assert 0 < int(run["accepted"]) <= run["drafted"]
    used = np.concatenate([table[b, : held[b]] for b in range(requests)])
    assert len(set(used)) == len(used)
    want = (run["table"].float() * run["scale"]).to(torch.bfloat16).cpu()
    rows = cache.rows.cpu()
    for b in range(requests):
        ids = tokens[b][tokens[b] >= 0]
        at = np.arange(len(ids))
        slots = table[b, at // block].astype(np.int64) * block + at % block
        assert torch.equal(rows[torch.as_tensor(slots)], want[torch.as_tensor(ids)]), b


def test_training_step(example):
    example.drs.load(build_if_missing=True)
    run = example.decode(4, 3, 6, vocab=512, width=64, seed=3)
    before = run["table"].clone()
    grad = example.train_step(run, run["tokens"], lr=0.05)
    assert torch.isfinite(grad).all() and float(grad.norm()) > 0
    # the loss on the same tokens falls
    t = run["tokens"]
    ids, after = t[:, :-1].reshape(-1), t[:, 1:].reshape(-1)
    ok = (ids >= 0) & (after >= 0)

    def loss(table):
        rows = table.double()[ids.clamp_min(0)] * run["scale"]
        logp = torch.log_softmax(rows @ table.double().t(), 1)
        return float(-(logp[torch.arange(len(ids)), after.clamp_min(0)] * ok).sum() / ok.sum())

    assert loss(run["table"]) < loss(before)
