"""drs_verify_drafts against a plain implementation in 64 bits.

The weights are the fp32 differences that the call defines; everything
after them (products, sums, comparisons) is fp64 on the CPU. Accepted
counts and tokens are exact: sums on both sides are good to about 1e-13,
and a sampled number that close to a border has a probability of about
1e-13 times the number of columns. Inputs with sums that are exact in
fp32 (multiples of 1/64) put the sampled numbers on the borders themselves."""
import numpy as np
import pytest
import torch

from gpu_util import drs

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def reference(target, draft, tokens, cu, au, su, most):
    """CPU tensors of any type; (tokens, accepted) as numpy."""
    p32 = target.float().numpy()
    q32 = None if draft is None else draft.float().numpy()
    requests, vocab = len(su), p32.shape[1]
    out = np.full((requests, most + 1), -1, np.int64)
    accepted = np.full(requests, -1, np.int32)
    for b in range(requests):
        first, count = int(cu[b]), min(max(int(cu[b + 1]) - int(cu[b]), 0), most)
        if first < 0 or first + count > len(tokens) or first + b + count >= len(p32):
            continue
        n = 0
        while n < count:
            r, x = first + n, int(tokens[first + n])
            if not 0 <= x < vocab:
                break
            q = 1.0 if q32 is None else float(q32[r, x])
            if not float(au[r]) * q < float(p32[r + b, x]):
                break
            n += 1
        accepted[b] = n
        out[b, :n] = tokens[first:first + n]
        p = p32[first + b + n]
        with np.errstate(invalid="ignore"):
            w = p.copy()
            if n < count:
                if q32 is not None:
                    w = p - q32[first + n]
                elif 0 <= int(tokens[first + n]) < vocab:
                    w[int(tokens[first + n])] = 0.0
            w = np.where(w > 0, w, np.float32(0))
            if not w.any():
                w = np.where(p > 0, p, np.float32(0))
        run = np.cumsum(w.astype(np.float64))
        if run[-1] > 0:
            over = np.flatnonzero((run > float(su[b]) * run[-1]) & (w > 0))
            out[b, n] = over[0] if len(over) else np.flatnonzero(w > 0)[-1]
    return out, accepted


def check(target, draft, tokens, cu, au, su, most, where):
    """target and draft: CUDA tensors (views of any stride); the rest numpy."""
    dev = lambda a, t: torch.as_tensor(a, dtype=t).cuda()
    got, acc = drs().verify_drafts(target, dev(tokens, torch.int64), dev(cu, torch.int32), dev(au, torch.float32),
                                   dev(su, torch.float32), most, draft_probs=draft)
    ref, ref_acc = reference(target.cpu(), None if draft is None else draft.cpu(), tokens, cu, au, su, most)
    assert np.array_equal(acc.cpu().numpy(), ref_acc), where
    assert np.array_equal(got.cpu().numpy(), ref), where
    return ref, ref_acc


def batch(seed, requests, most, vocab, target, draft, pad=0, offset=0, spread=3.0):
    """Rows of softmax probabilities inside a buffer whose other places hold
    NaN: `offset` elements before the first row, `pad` after each."""
    rng = np.random.default_rng(seed)
    count = rng.integers(0, most + 1, requests)
    count[rng.random(requests) < 0.5] = most
    cu = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    total = int(cu[-1])
    g = torch.Generator().manual_seed(seed)

    def rows(x, dtype):
        buffer = torch.full((offset + x.shape[0] * (vocab + pad),), float("nan"), dtype=dtype)
        view = buffer[offset:].view(x.shape[0], vocab + pad)[:, :vocab]
        view.copy_(x.to(dtype))
        return buffer.cuda()[offset:].view(x.shape[0], vocab + pad)[:, :vocab]

    y = spread * torch.randn(total, vocab, generator=g)
    q = torch.softmax(y, 1)
    p = torch.softmax(spread * torch.randn(total + requests, vocab, generator=g), 1)
    owner = np.repeat(np.arange(requests), count)
    at = torch.as_tensor(np.arange(total) + owner)
    p[at] = torch.softmax(y + torch.randn(total, vocab, generator=g), 1)
    tokens = torch.multinomial(q, 1, generator=g)[:, 0].numpy() if total else np.zeros(0, np.int64)
    return (rows(p, TYPES[target]), None if draft is None else rows(q, TYPES[draft]), tokens, cu,
            rng.random(total, dtype=np.float32), rng.random(requests, dtype=np.float32), most)


@pytest.mark.parametrize("target", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("draft", ["fp32", "bf16", "fp16", None])
def test_every_pair_of_types(target, draft):
    for seed, (vocab, pad) in enumerate([(1000, 0), (8192, 0), (20011, 5)]):
        check(*batch(seed, 9, 6, vocab, target, draft, pad), where=(vocab, pad))


@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 31, 255, 256, 257, 4095, 4097, 8191, 8193, 16385, 65537, 131072, 262144])
def test_every_row_length(vocab):
    check(*batch(vocab, 5, 3, vocab, "bf16", "fp16"), where=vocab)
    check(*batch(vocab + 1, 3, 2, vocab, "fp32", None), where=vocab)


@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 2), (8, 8), (64, 4)])
def test_strides_and_alignment(pad, offset):
    for draft in ("bf16", None):
        check(*batch(pad, 6, 4, 5000, "bf16", draft, pad, offset), where=(pad, offset, draft))
    check(*batch(pad, 3, 2, 12001, "fp32", "fp32", pad, offset), where=(pad, offset))


def test_longest_row():
    check(*batch(3, 2, 2, 1 << 21, "bf16", "bf16", spread=2.0), where="2^21")


@pytest.mark.parametrize("requests,most", [(1, 0), (1, 1), (1, 33), (4, 64), (40, 100), (300, 5), (700, 2)])
def test_counts_of_requests_and_drafts(requests, most):
    """More than 32 drafts, requests without any, and drafts that are all
    accepted (identical distributions)."""
    a = list(batch(requests, requests, most, 600, "fp32", "fp32"))
    check(*a, where="random")
    owner = np.repeat(np.arange(requests), np.diff(a[3]))
    if len(owner):
        a[0][torch.as_tensor(np.arange(len(owner)) + owner).cuda()] = a[1]
        _, acc = check(*a, where="identical")
        assert np.array_equal(acc, np.diff(a[3]))


@pytest.mark.parametrize("requests,vocab,target,draft,pad", [
    (200, 40000, "bf16", "fp16", 0), (200, 40001, "bf16", "fp16", 0), (48, 140000, "fp16", None, 0),
    (40, 66003, "fp32", "fp32", 2), (100, 131072, "bf16", "bf16", 0), (24, 262144, "bf16", None, 8)])
def test_batches_of_every_cluster_size(requests, vocab, target, draft, pad):
    """Batches that fill the GPU once or several times, with 1 to 16 CTAs per request."""
    check(*batch(requests + vocab, requests, 2, vocab, target, draft, pad), where=(requests, vocab))


def test_sampled_numbers_on_the_borders():
    """Weights that are multiples of 1/64: every sum is exact, so numbers at,
    just below and just above each border have one right column. Zero
    weights before, between and after the others are never drawn."""
    for vocab in (64, 1000, 70000):
        rng = np.random.default_rng(vocab)
        at = np.sort(rng.choice(np.arange(1, vocab - 1), 16, replace=False))
        p = np.zeros(vocab, np.float32)
        p[at] = rng.multinomial(48, np.ones(16) / 16) / 64 + 1 / 64
        assert p.sum() == 1.0
        borders = np.concatenate([[0], np.cumsum(p[p > 0])]).astype(np.float32)
        su = np.concatenate([borders, np.nextafter(borders, np.float32(2)), np.nextafter(borders, np.float32(-1))])
        n = len(su)
        target = torch.as_tensor(p).expand(n, vocab).contiguous().cuda()
        for t in (torch.float32, torch.bfloat16):
            check(target.to(t), None, np.zeros(0, np.int64), np.zeros(n + 1), np.zeros(0, np.float32), su, 0, where=vocab)


def test_acceptance_is_exact():
    """u q < p at equality (refused) and one step to either side."""
    vocab, u = 16, np.float32(0.7)
    q = np.float32(0.3)
    p0 = float(u) * float(q)
    ps = [np.float32(p0), np.nextafter(np.float32(p0), np.float32(1)), np.nextafter(np.float32(p0), np.float32(0)),
          np.float32(0), np.float32(0.35)]
    us = [u, u, u, np.float32(0), np.float32(1) - np.float32(2**-24)]
    target = np.full((2 * len(ps), vocab), 0.01, np.float32)
    target[0::2, 5] = ps
    draft = np.full((len(ps), vocab), 0.02, np.float32)
    draft[:, 5] = q
    cu = np.arange(len(ps) + 1)
    _, acc = check(torch.as_tensor(target).cuda(), torch.as_tensor(draft).cuda(), np.full(len(ps), 5), cu,
                   np.array(us, np.float32), np.full(len(ps), 0.5, np.float32), 1, where="equality")
    assert acc[3] == 0 and acc[4] == 1


@pytest.mark.parametrize("vocab", [40, 9000, 140000])
def test_rows_without_weight_and_odd_values(vocab):
    """No residual (the draft's probabilities are nowhere below the target's):
    from the target's row. No weight at all: -1. NaN and negative entries
    weigh nothing. Draft tokens outside the vocabulary are refused."""
    rng = np.random.default_rng(vocab)
    requests = 7
    target = np.zeros((2 * requests, vocab), np.float32)
    draft = np.zeros((requests, vocab), np.float32)
    target[:, : vocab // 2] = rng.random((2 * requests, vocab // 2)).astype(np.float32) / vocab
    draft[:] = 1.0
    target[2] = 0.0                      # request 1: nothing at all
    target[4] = np.nan                   # request 2: nothing but NaN
    target[6, ::3] = np.nan              # request 3: NaN between weights
    target[6, 1::3] = -1.0
    draft[3] = np.nan                    # request 3: p - q is NaN everywhere
    target[8] = 0.0                      # request 4: one column only
    target[8, vocab - 1] = 1.0
    draft[5, : vocab // 3] = 0.0         # request 5: a residual in part of the row
    tokens = np.array([0, 1, 2, 0, 0, -1, vocab], np.int64)
    cu = np.arange(requests + 1)
    au = np.full(requests, 0.999, np.float32)
    for u in (0.0, 0.3, 1.0 - 2.0**-24, 1.0):
        su = np.full(requests, u, np.float32)
        for d in (draft, None):
            out, acc = check(torch.as_tensor(target).cuda(), None if d is None else torch.as_tensor(d).cuda(), tokens,
                             cu, au, su, 1, where=(u, d is None))
            assert out[1, 0] == -1 and out[2, 0] == -1


def test_offsets_past_32_bits():
    """Rows 2^31 + 8 elements apart: the last ones lie past 2^32 elements."""
    a = list(batch(12, 2, 1, 3000, "bf16", "bf16"))
    a[3], a[2] = np.array([0, 1, 2], np.int32), np.array([7, 2999])
    g = torch.Generator().manual_seed(1)
    far = []
    for n in (4, 2):
        buffer = torch.empty(n * (2**31 + 8), dtype=torch.bfloat16, device="cuda")
        rows_far = buffer.view(n, 2**31 + 8)[:, :3000]
        rows_far.copy_(torch.softmax(3 * torch.randn(n, 3000, generator=g), 1))
        far.append(rows_far)
    for u in (0.0, 0.99):
        check(far[0], far[1], a[2], a[3], np.full(2, u, np.float32), np.array([0.2, 0.9], np.float32), 1, where=u)
        check(far[0], None, a[2], a[3], np.full(2, u, np.float32), np.array([0.2, 0.9], np.float32), 1, where=u)


def test_requests_outside_the_arrays_are_marked():
    """Offsets that are negative, past the drafts or past the target's rows:
    -1, nothing read; the others are as ever. Falling offsets are no drafts."""
    a = list(batch(8, 6, 3, 500, "bf16", "bf16"))
    total = len(a[2])
    cu = a[3].copy()
    for bad in (np.array([-1, 2, 3, 3, 2, total, total + 1]), np.array([0, 1, total + 5, 0, 1, 2, 1 << 30]),
                np.array([-(1 << 31), (1 << 31) - 1, 0, 2, 2, 1, total])):
        a[3] = bad.astype(np.int32)
        check(*a, where=bad)
    a[3] = cu
    a[0] = a[0][:-2]  # the last requests' rows are missing
    check(*a, where="short target")


def test_outputs_streams_and_graphs():
    """Given outputs, another stream, a captured graph whose inputs change."""
    lib = drs()
    a = batch(11, 8, 5, 30000, "bf16", "fp16")
    target, draft = a[0], a[1]
    dev = lambda x, t: torch.as_tensor(x, dtype=t).cuda()
    tokens, cu, au, su = dev(a[2], torch.int64), dev(a[3], torch.int32), dev(a[4], torch.float32), dev(a[5], torch.float32)
    ref = reference(target.cpu(), draft.cpu(), *a[2:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = lib.verify_drafts(target, tokens, cu, au, su, 5, draft_probs=draft, stream=side)
    side.synchronize()
    assert np.array_equal(out[0].cpu().numpy(), ref[0]) and np.array_equal(out[1].cpu().numpy(), ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib.verify_drafts(target, tokens, cu, au, su, 5, draft_probs=draft)
    for _ in range(3):
        su.copy_(torch.rand(8))
        graph.replay()
        ref = reference(target.cpu(), draft.cpu(), *a[2:5], su.cpu().numpy(), 5)
        assert np.array_equal(out[0].cpu().numpy(), ref[0]) and np.array_equal(out[1].cpu().numpy(), ref[1])


def test_drawn_tokens_follow_the_target():
    """The law of speculative sampling: whatever the draft's distribution, the
    first token out is distributed as the target's. 40000 requests against
    the exact probabilities, within five standard deviations."""
    g = torch.Generator().manual_seed(5)
    vocab, n = 24, 40000
    p, q = torch.softmax(2 * torch.randn(vocab, generator=g), 0), torch.softmax(2 * torch.randn(vocab, generator=g), 0)
    tokens = torch.multinomial(q, n, replacement=True, generator=g)
    target = p.expand(2 * n, vocab).contiguous().cuda()
    out, _ = drs().verify_drafts(target, tokens.cuda(), torch.arange(n + 1, dtype=torch.int32).cuda(),
                                 torch.rand(n, generator=g).cuda(), torch.rand(n, generator=g).cuda(), 1,
                                 draft_probs=q.expand(n, vocab).contiguous().cuda())
    freq = torch.bincount(out[:, 0].cpu(), minlength=vocab).double() / n
    sigma = (p.double() * (1 - p.double()) / n).sqrt()
    assert ((freq - p.double()).abs() <= 5 * sigma + 1e-6).all()
