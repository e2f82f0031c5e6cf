"""The gradient of ids that occur very often, exactly: the gradients are small
integers, the scale a power of two, and every sum of magnitudes is below 2^24, so
fp32 additions in any order are exact and the result is rounded once. A bound that
allows n roundings of n summands lets whole tokens go missing from some
thousand occurrences on; equality shows a single one."""
import numpy as np
import pytest
import torch

from gpu_util import drs

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def case(n, vocab, width, kind, seed):
    """ids, and gradients that are non-zero integers of magnitude 1 to 8 (exact in
    every type; over 2^21 occurrences fit)."""
    rng = np.random.default_rng(seed)
    if kind == "one":
        ids = np.full(n, vocab // 3)
    elif kind == "few":
        ids = rng.choice(np.array([0, vocab // 2, vocab - 1]), n, p=[0.6, 0.3, 0.1])
    elif kind == "runs":  # an id's tokens side by side
        ids = np.sort(rng.integers(0, min(vocab, 5), n)) * (vocab // 5 or 1) % vocab
    else:  # one id in a third of the tokens, padding, and the rest anywhere
        ids = rng.integers(0, vocab, n)
        ids[::3] = vocab // 2
        ids[1::17] = -1
    grad = rng.integers(1, 9, (n, width)) * rng.choice([-1, 1], (n, width))
    return ids.astype(np.int64), grad


def sums(ids, grad, vocab):
    total = torch.zeros(vocab, grad.shape[1], dtype=torch.int64, device=grad.device)
    keep = (ids >= 0) & (ids < vocab)
    total.index_add_(0, ids[keep], grad[keep])
    return total


def test_a_missing_token_shows():
    """The oracle without one token differs in every column, however often the
    id occurs; the magnitudes' sum stays exact in fp32."""
    n, vocab = 100003, 50
    ids, grad = (torch.as_tensor(a) for a in case(n, vocab, 4, "most", 1))
    assert int(sums(ids, grad.abs(), vocab).max()) < 1 << 24
    whole = sums(ids, grad, vocab)
    for t in (0, 3, 99999):
        assert int(ids[t]) == vocab // 2
        without = sums(torch.cat([ids[:t], ids[t + 1:]]), torch.cat([grad[:t], grad[t + 1:]]), vocab)
        assert bool((whole[vocab // 2] != without[vocab // 2]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["one", "few", "runs", "most"])
@pytest.mark.parametrize("n,vocab,width", [
    (4096, 4097, 72), (4097, 1, 16), (9001, 3001, 264), (5000, 600, 4100), (70001, 262144, 33), (131072, 1, 16),
    (131073, 1, 16), (131073, 262144, 8), (300007, 262144, 24), (300007, 1500, 9), (1500011, 3, 8)])
def test_frequent_ids(n, vocab, width, kind):
    """The rank sort, the cluster sort and the tiled one; pieces of both
    lengths; parts of an id over up to twelve thousand pieces."""
    ids, grad = (torch.as_tensor(a).cuda() for a in case(n, vocab, width, kind, n))
    assert int(sums(ids, grad.abs(), vocab).max()) < 1 << 24
    want = sums(ids, grad, vocab).double() * 0.5
    for up, out in (("fp32", "fp32"), ("bf16", "fp32"), ("fp16", "bf16")):
        table = torch.full((vocab, width), float("nan"), dtype=TYPES[out], device="cuda")
        drs().embed_tokens_grad(grad.to(TYPES[up]), ids, 0.5, table)
        assert torch.equal(table, want.to(TYPES[out])), (up, out)
    base = torch.randint(-4, 5, (vocab, width), device="cuda", generator=torch.Generator("cuda").manual_seed(n))
    table = base.float()
    drs().embed_tokens_grad(grad.to(torch.bfloat16), ids.int(), 0.5, table, accumulate=True)
    assert torch.equal(table.double(), want + base)
