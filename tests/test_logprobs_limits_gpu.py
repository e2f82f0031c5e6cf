"""drs_token_logprobs at the edges of what its sums are held in: floors that leave the type's range, and values that
have a bound of their own (tolerances: score_util)."""
import pytest
import torch

from gpu_util import drs
from score_util import TYPES, check_logprobs, close, grad_reference, ids_of, logits_of

pytestmark = pytest.mark.gpu
INF = float("inf")


def behind_a_mask(rows, vocab, dtype, centre, spread, seed):
    """Logits around `centre` behind a prefix of -inf: whole blocks of it come before a warp's first finite logit."""
    logits = logits_of("plain", rows, vocab, torch.float32, seed)
    logits = (logits * (spread / 3) + centre).to(dtype)
    logits[:, : vocab * 5 // 8] = -INF
    logits[1] = -INF
    return logits, ids_of(rows, vocab, seed)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("temp,centre,spread", [(472.6, 50.0, 3.0), (480.0, 1100.0, 10.0), (500.0, 5000.0, 300.0),
                                                (700.0, 40000.0, 1000.0)])
@pytest.mark.parametrize("rows,vocab,k", [(6, 30000, 8), (2, 131072, 0), (400, 9000, 20), (700, 20000, 0)])
def test_masked_prefixes_before_the_first_reference(dtype, temp, centre, spread, rows, vocab, k):
    """Without a reference the logits whose exponents (base 2) are -200 lie at -138.63 T, below fp16's range from T = 472.6
    on; with one, a largest logit of at least 138.63 T - 65504 (12 for 472.6, 3811 for 500), they are within it again, and
    the sums go on without care. Clusters and teams."""
    temps = torch.tensor([temp], device="cuda")
    logits, ids = behind_a_mask(rows, vocab, TYPES[dtype], centre, spread, rows)
    out = drs().token_logprobs(logits, ids, k, temps, rows)
    ref = check_logprobs(out, logits, ids, k, temps, rows)
    assert out[1].isfinite().all()
    # and the entropy's gradient, from what the call has left
    one = torch.ones(rows, device="cuda")
    alive = ref["inside"] & (ref["max"] > -INF)
    grad = drs().token_logprobs_grad(logits, ids, out[3], one, out[1], one, temps, rows, out=torch.empty_like(logits))
    value, tol = grad_reference(logits, ids, out[3], one, out[1], one, temps, rows, TYPES[dtype])
    close(grad[alive], value[alive], tol[alive], "gradient")
    assert (grad[~alive] == 0).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", ["alone", "peaks", "ties", "far"])
@pytest.mark.parametrize("rows,vocab", [(40, 20011), (300, 8192), (3000, 1000)])
@pytest.mark.parametrize("temp", [None, 0.013, 0.7, 31.0])
def test_no_log_probability_above_zero_and_no_entropy_below(dtype, kind, rows, vocab, temp):
    """S holds the largest logit's term, 1, so that ln S >= 0, every log probability <= 0 and the entropy >= 0, by exactly
    that much: no tolerance. Rows whose largest logit is all there is (alone: of any value, all others -inf) are
    those where the sum's own roundings decide."""
    logits, ids = logits_of("plain" if kind == "alone" else kind, rows, vocab, TYPES[dtype], rows), ids_of(rows, vocab, rows)
    if kind == "alone":
        at = torch.arange(rows, device="cuda")
        peak = (100 * logits[:, 0].float()).to(TYPES[dtype])
        logits.fill_(-INF)
        logits[at, at % vocab] = peak
        ids[::2] = (at % vocab)[::2]
    temps = None if temp is None else torch.tensor([temp], device="cuda")
    out = drs().token_logprobs(logits, ids, 6, temps, rows)
    check_logprobs(out, logits, ids, 6, temps, rows)
    logprob, entropy, _, norm, _, top = out
    assert (logprob <= 0).all() and (entropy >= 0).all() and (norm[:, 1] >= 0).all() and (top <= 0).all()
