"""The checks of the scoring operators' tests notice small mistakes (no GPU needed): outputs are made by the plain 64-bit form
and rounded to fp32, then one of them is changed."""
import pytest
import torch

from score_util import check_logprobs, grad_reference, close, reference

ROWS, VOCAB, K = 5, 4000, 6


def inputs():
    g = torch.Generator().manual_seed(3)
    logits = 3 * torch.randn(ROWS, VOCAB, generator=g)
    logits[:, 17] = logits.amax(1)  # equal ones at the top
    ids = torch.tensor([5, 17, -1, VOCAB - 1, 99])
    return logits, ids


def outputs(logits, ids, drop=None):
    """The outputs by the definition; drop: a column that the sums leave out."""
    rows = torch.arange(ROWS)
    kept = logits.clone()
    if drop is not None:
        kept[rows, drop] = -float("inf")
    ref, short = reference(logits, ids, K), reference(kept, ids, K)
    off = ref["log_sum"][0] - short["log_sum"][0]
    gone = ~ref["inside"]
    log_sum = short["log_sum"][0]
    out = [ref["logprob"][0] + off, short["entropy"][0], ref["rank"].clone(), torch.stack([ref["max"], log_sum], 1),
           ref["top_ids"].clone(), ref["top_logprobs"][0] + off[:, None]]
    for t, nothing in zip(out, (0, 0, 0, 0, -1, -float("inf"))):
        t[gone] = nothing
    return [t.float() if t.is_floating_point() else t.int() for t in out]


def test_the_definition_passes():
    logits, ids = inputs()
    check_logprobs(outputs(logits, ids), logits, ids, K)


def test_a_column_of_weight_one_thousandth_that_is_left_out():
    logits, ids = inputs()
    p = reference(logits, ids, K)["p"]
    at = (p - 1e-3).abs().argmin(1)
    weight = p[torch.arange(ROWS), at]
    assert ((weight > 5e-4) & (weight < 2e-3)).all() and not (at == ids).any()
    out = outputs(logits, ids, at)
    with pytest.raises(AssertionError):
        check_logprobs(out, logits, ids, K)
    right = outputs(logits, ids)
    for changed in (0, 1, 3, 5):  # by each output alone
        mixed = list(right)
        mixed[changed] = out[changed]
        with pytest.raises(AssertionError):
            check_logprobs(mixed, logits, ids, K)


@pytest.mark.parametrize("change", ["rank", "order", "tie", "id", "logprob", "entropy", "passed over"])
def test_one_wrong_value(change):
    logits, ids = inputs()
    out = outputs(logits, ids)
    if change == "rank":
        out[2][4] += 1
    elif change == "order":
        out[4][0, 2:4] = out[4][0, 2:4].flip(0)
    elif change == "tie":  # the equal ones at the top, the higher column first
        assert logits[1, out[4][1, 0]] == logits[1, out[4][1, 1]]
        out[4][1, :2] = out[4][1, :2].flip(0)
    elif change == "id":
        out[4][3, K - 1] += 1
    elif change == "logprob":
        out[0][0] += 1e-4
    elif change == "entropy":
        out[1][1] *= 1 + 1e-4
    else:
        out[0][2] = -1.0
    with pytest.raises(AssertionError):
        check_logprobs(out, logits, ids, K)


@pytest.mark.parametrize("dtype,by", [(torch.float32, 1e-4), (torch.bfloat16, 0.02), (torch.float16, 2e-3)])
def test_a_gradient_that_is_off(dtype, by):
    logits, ids = inputs()
    ref = reference(logits, ids, K)
    norm = torch.stack([ref["max"], ref["log_sum"][0]], 1).float()
    one = torch.ones(ROWS)
    value, tol = grad_reference(logits, ids, norm, one, ref["entropy"][0].float(), one, None, 1, dtype)
    close(value.to(dtype), value, tol, "gradient")
    for at in ((0, 5), (1, 17), (4, int(ref["p"][4].argmax()))):
        wrong = value.clone()
        wrong[at] *= 1 + by
        with pytest.raises(AssertionError):
            close(wrong.to(dtype), value, tol, "gradient")
