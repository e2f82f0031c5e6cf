"""drs_verify_drafts at the ends of its ranges: the largest number of drafts that
the call takes (a request's places are counted in 64 bits), and rows whose whole
mass lies at the bottom of the type's range (against the plain implementation
in 64 bits, which such weights, their sums and products fit exactly)."""
import numpy as np
import pytest
import torch

from gpu_util import drs
from test_verify_gpu import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [2**31 - 1, 2**31 - 257])
def test_most_drafts(most):
    """One request of two drafts whose row of 2^31 output places (17 GB) is
    written to its end; then one outside the arrays, whose places are all -1."""
    lib = drs()
    target = torch.tensor([[0.5, 0.5, 0.0], [0.0, 1.0, 0.0], [0.0, 0.0, 1.0]], device="cuda")
    tokens = torch.tensor([1, 1], device="cuda")
    u = torch.tensor([0.25, 0.5], device="cuda")
    out = torch.full((1, most + 1), 7, dtype=torch.int64, device="cuda")
    for cu, first, accepted in (([0, 2], [1, 1, 2], 2), ([1, 5], [-1, -1, -1], -1)):
        out.fill_(7)
        _, acc = lib.verify_drafts(target, tokens, torch.tensor(cu, dtype=torch.int32, device="cuda"), u, u[:1].clone(), most,
                                   out_tokens=out)
        assert out[0, :3].tolist() == first and int(acc) == accepted
        for part in out[0, 3:].split(1 << 28):
            assert bool((part == -1).all())


def tiny_rows(rng, rows, vocab, step, pad):
    """Up to 40 weights of 1 to 63 steps per row, zeros between them."""
    w = np.zeros((rows, vocab), np.float32)
    for r in range(rows):
        at = rng.choice(vocab, min(vocab, int(rng.integers(1, 41))), replace=False)
        w[r, at] = (rng.integers(1, 64, len(at)) * np.float64(step)).astype(np.float32)
    buffer = torch.zeros(rows, vocab + pad)
    buffer[:, :vocab] = torch.as_tensor(w)
    return buffer


@pytest.mark.parametrize("vocab,pad", [(3, 0), (50, 1), (1000, 0), (9001, 2), (140000, 0)])
@pytest.mark.parametrize("dtype,step", [("float32", 2.0**-149), ("float32", 2.0**-130), ("float32", 2.0**-100),
                                        ("float32", 2.0**-27), ("bfloat16", 2.0**-133), ("float16", 2.0**-24)])
def test_weights_of_a_few_smallest_steps(vocab, pad, dtype, step):
    """u times the total is compared exactly however small the weights are:
    rows after the last draft, and residuals of a refused one."""
    rng = np.random.default_rng(vocab)
    t, n = getattr(torch, dtype), 120
    su = rng.integers(0, 64, n).astype(np.float32) / 64
    su[::3] = rng.random(len(su[::3]), dtype=np.float32)
    none = np.zeros(0, np.float32)
    p = tiny_rows(rng, n, vocab, step, pad).to(t).cuda()[:, :vocab]
    check(p, None, none.astype(np.int64), np.zeros(n + 1), none, su, 0, where="whole rows")
    n //= 2
    p = tiny_rows(rng, 2 * n, vocab, step, pad).to(t).cuda()[:, :vocab]
    q = tiny_rows(rng, n, vocab, step, pad).to(t).cuda()[:, :vocab]
    refused = np.full(n, 0.999, np.float32)
    q[torch.arange(n), 0] = 1.0
    for draft in (q, None):
        check(p, draft, np.zeros(n, np.int64), np.arange(n + 1), refused, su[:n], 1, where=draft is None)


def test_three_smallest_weights():
    """u = 1/2 of three weights of the smallest step: the second column's sum is the first above it."""
    p = torch.zeros(1, 8)
    p[0, [1, 4, 6]] = 2.0**-149
    out, _ = drs().verify_drafts(p.cuda(), torch.zeros(0, dtype=torch.int64, device="cuda"),
                                 torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(0, device="cuda"),
                                 torch.full((1,), 0.5, device="cuda"), 0)
    assert out.tolist() == [[4]]
