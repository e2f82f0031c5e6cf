"""drs_token_logprobs and drs_token_logprobs_grad against plain forms in 64 bits (score_util has them and the
tolerances), and the gradient against differences."""
import pytest
import torch

from gpu_util import drs
from score_util import (EX2, TYPES, U, additions, check_logprobs, close, grad_reference, ids_of, logits_of, reference,
                        rows_in_buffer)

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 31, 255, 256, 257, 1000, 2048, 4097, 8192, 20011, 50001, 131072])
def test_sizes(dtype, vocab):
    for rows, k, id_type in ((1, 1, torch.int64), (3, 20, torch.int32), (40, 64, torch.int64), (330, 0, torch.int32)):
        k = min(k, vocab)
        logits, ids = logits_of("plain", rows, vocab, TYPES[dtype], rows + vocab), ids_of(rows, vocab, vocab, id_type)
        check_logprobs(drs().token_logprobs(logits, ids, k), logits, ids, k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab,k", [(1, 262144, 20), (2, 262144, 64), (5, 300007, 33), (1, 2097152, 20),
                                          (40, 262144, 5), (700, 16384, 8), (5000, 256, 4), (160, 100000, 64)])
def test_large(dtype, rows, vocab, k):
    logits, ids = logits_of("plain", rows, vocab, TYPES[dtype], vocab), ids_of(rows, vocab, 5)
    check_logprobs(drs().token_logprobs(logits, ids, k), logits, ids, k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", ["ties", "equal", "rising", "falling", "peaks", "masked", "lowest", "zeros", "far"])
@pytest.mark.parametrize("rows,vocab,k", [(9, 777, 64), (6, 50001, 20), (320, 8192, 20), (3, 262144, 64)])
def test_kinds_of_rows(dtype, kind, rows, vocab, k):
    logits, ids = logits_of(kind, rows, vocab, TYPES[dtype], 7), ids_of(rows, vocab, 3)
    check_logprobs(drs().token_logprobs(logits, ids, k), logits, ids, k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "masked", "rising"])
@pytest.mark.parametrize("rows", [5, 40, 300, 470, 700, 1000, 2300, 3700])
def test_numbers_of_rows(dtype, kind, rows):
    """Rows by clusters and by teams of 8, 4, 2 and 1 warps, several in turn, rows that are passed over among them."""
    for vocab, k, pad in ((1500, 20, 1), (13000, 64, 0)) if rows < 1500 else ((1500, 64, 0), (5003, 20, 1)):
        logits, ids = logits_of(kind, rows, vocab, TYPES[dtype], rows, pad), ids_of(rows, vocab, rows)
        if rows == 700:
            ids[:650] = -1
        check_logprobs(drs().token_logprobs(logits, ids, k), logits, ids, k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab,k", [(500, 140001, 5), (600, 262144, 64), (1100, 70001, 20), (3300, 4099, 7), (4300, 4099, 7),
                                          (2500, 15700, 61), (2500, 16000, 62), (1000, 16100, 63), (3000, 15900, 63)])
def test_where_the_teams_change(dtype, rows, vocab, k):
    """Numbers of rows at which other sizes of teams take them, and a few segments fewer than alternatives."""
    logits = logits_of("ties" if k > 60 else "plain", rows, vocab, TYPES[dtype], vocab)
    ids = ids_of(rows, vocab, 3)
    check_logprobs(drs().token_logprobs(logits, ids, k), logits, ids, k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab", [(3, 100000), (60, 30011), (700, 20000), (2500, 3000)])
def test_temperatures_of_all_sizes_in_a_batch(dtype, rows, vocab):
    """Rows that need care from the start, on the way (huge logits) and not at all, in turn for one team."""
    temps = torch.tensor([0.0, 1.0, 1e-4, 0.02, 3.0, 1e-7, 0.7], device="cuda").repeat(-(-rows // 7))[:rows]
    for kind in ("ties", "far", "masked"):
        logits, ids = logits_of(kind, rows, vocab, TYPES[dtype], rows, 1), ids_of(rows, vocab, 1)
        check_logprobs(drs().token_logprobs(logits, ids, 9, temps), logits, ids, 9, temps)


@pytest.mark.parametrize("temp", [400.0, 1e4, 1e30, 3e38])
def test_large_temperatures_under_masks(temp):
    """The floor of the exponents leaves the type's range; whole parts of the rows are -inf."""
    temps = torch.tensor([temp], device="cuda")
    for dtype in TYPES.values():
        for rows, vocab in ((6, 30000), (400, 9000)):
            logits, ids = logits_of("plain", rows, vocab, dtype, 1), ids_of(rows, vocab, 1)
            logits[:, : vocab * 3 // 4] = -INF
            logits[1] = -INF
            out = drs().token_logprobs(logits, ids, 8, temps, rows)
            check_logprobs(out, logits, ids, 8, temps, rows)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [520, 4100, 50001])
@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (8, 8), (3, 5), (24, 0), (7, 3)])
def test_strides_and_offsets(dtype, vocab, pad, offset):
    logits, ids = logits_of("ties", 11, vocab, TYPES[dtype], pad, pad, offset), ids_of(11, vocab, 2)
    check_logprobs(drs().token_logprobs(logits, ids, 20), logits, ids, 20)


@pytest.mark.parametrize("canvas_len", [1, 4, 1000])
def test_temperatures(canvas_len):
    rows, vocab = 37, 5000
    temps = torch.linspace(0.3, 2.5, -(-rows // canvas_len), device="cuda")
    for dtype in TYPES.values():
        logits, ids = logits_of("plain", rows, vocab, dtype, 1), ids_of(rows, vocab, 1)
        check_logprobs(drs().token_logprobs(logits, ids, 8, temps, canvas_len), logits, ids, 8, temps, canvas_len)


def test_temperatures_at_and_below_zero():
    """Clamped at 1e-10: the distribution of the largest logit alone, exactly. At 1e-3 the exponents are x c - (m c
    rounded), 2^-24 of their size off at x = m; e^d is 2^t to 2^-22, so that ln S is within the tolerances but not
    exactly 0."""
    temps = torch.tensor([0.0, -1.0, 1e-12, 1e-10, 1e-3], device="cuda")
    logits, ids = logits_of("peaks", 5, 3001, torch.float32, 1), torch.tensor([0, 1, 2, 3, 4], device="cuda")
    out = drs().token_logprobs(logits, ids, 4, temps)
    check_logprobs(out, logits, ids, 4, temps)
    assert (out[1][:4] == 0).all() and (out[5][:4, 0] == 0).all()


def test_nan_and_infinite_logits():
    """NaN where the sum enters, nothing else: columns are ordered with NaN at the end, the rank counts what exceeds
    the token's logit."""
    for dtype in TYPES.values():
        for vocab in (40, 5000, 70001):
            logits, ids = logits_of("plain", 6, vocab, dtype, 4), torch.tensor([3, 3, 3, 3, 3, 3], device="cuda")
            logits[0, 7] = INF
            logits[1, 9] = float("nan")
            logits[2, 3] = float("nan")
            logits[3] = float("nan")
            logits[4] = -INF
            logits[4, vocab // 2] = float("nan")
            out = drs().token_logprobs(logits, ids, 20)
            assert out[0][:5].isnan().all() and out[1][:4].isnan().all() and out[5][:5].isnan().all()
            assert out[0][5:].isfinite().all() and out[1][5:].isfinite().all()
            ref = reference(logits, ids, 20)
            assert torch.equal(out[4].long(), ref["top_ids"])
            assert torch.equal(out[2].long(), ref["rank"])


def test_outputs_that_are_not_wanted_and_rows_behind_the_last():
    lib = drs()
    logits, ids = logits_of("plain", 9, 3000, torch.bfloat16, 4), ids_of(9, 3000, 4)
    whole = lib.token_logprobs(logits, ids, 5)
    alone = torch.empty(9, device="cuda")
    assert lib.token_logprobs(logits, ids, 0, out=(alone, None, None, None, None, None))[0] is alone
    assert torch.equal(alone, whole[0])
    parts = [torch.full((12, *t.shape[1:]), 77, dtype=t.dtype, device="cuda") for t in whole]
    lib.token_logprobs(logits, ids, 5, out=tuple(t[:9] for t in parts))
    for part, t in zip(parts, whole):
        assert torch.equal(part[:9], t) and (part[9:] == 77).all()
    assert all(t.shape[0] == 0 for t in lib.token_logprobs(logits[:0], ids[:0], 5))


def test_equal_calls_give_equal_bits_and_streams():
    lib = drs()
    logits, ids = logits_of("plain", 50, 30000, torch.bfloat16, 4), ids_of(50, 30000, 4)
    first = lib.token_logprobs(logits, ids, 20)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [lib.token_logprobs(logits, ids, 20, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_offsets_past_32_bits():
    rows, vocab = 16500, 131072
    logits = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    logits[-2:] = logits_of("plain", 2, vocab, torch.bfloat16, 1)
    ids = torch.full((rows,), -1, device="cuda")
    ids[-2:] = torch.tensor([5, vocab - 1], device="cuda")
    out = drs().token_logprobs(logits, ids, 7)
    check_logprobs([t[-2:] for t in out], logits[-2:], ids[-2:], 7)
    grad = drs().token_logprobs_grad(logits, ids, out[3], torch.ones(rows, device="cuda"), out=logits)
    assert (grad[:-2] == 0).all() and (grad[-2:] != 0).any()


# ------------------------------------------------------------- the gradient

def forward_state(logits, ids, temps, canvas_len):
    ref = reference(logits, ids, 0, temps, canvas_len)
    norm = torch.stack([ref["max"], ref["log_sum"][0]], 1).float()
    return norm, ref["entropy"][0].float()


def arriving(rows, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, generator=g, device="cuda"), torch.randn(rows, generator=g, device="cuda")


def check_grad(logits, ids, out_type, temps=None, canvas_len=1, which="both", out=None):
    norm, entropy = forward_state(logits, ids, temps, canvas_len)
    g, h = arriving(logits.shape[0], 3)
    g, h = (g if which != "entropy" else None), (h if which != "logprob" else None)
    if out is None:
        out = torch.empty(logits.shape, dtype=out_type, device="cuda")
    value, tol = grad_reference(logits, ids, norm, g, entropy, h, temps, canvas_len, out_type)  # before logits change
    got = drs().token_logprobs_grad(logits, ids, norm, g, entropy=entropy if h is not None else None, grad_entropy=h,
                                    temps=temps, canvas_len=canvas_len, out=out)
    close(got, value, tol, "gradient")
    return got


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 7), (3, 8), (5, 257), (33, 1000), (7, 4097), (3, 50001), (2, 262144),
                                        (400, 2048)])
def test_grad_sizes(dtype, out, rows, vocab):
    logits, ids = logits_of("plain", rows, vocab, TYPES[dtype], vocab), ids_of(rows, vocab, 1, torch.int32)
    for which in ("both", "logprob", "entropy"):
        check_grad(logits, ids, TYPES[out], which=which)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", ["ties", "equal", "peaks", "masked", "lowest", "far"])
def test_grad_kinds_of_rows(dtype, kind):
    logits, ids = logits_of(kind, 9, 3001, TYPES[dtype], 7), ids_of(9, 3001, 3)
    check_grad(logits, ids, TYPES[dtype])
    check_grad(logits, ids, torch.float32, which="logprob")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("pads,offsets", [((1, 0), (0, 0)), ((0, 1), (1, 0)), ((8, 8), (8, 8)), ((3, 3), (5, 5)),
                                          ((24, 5), (0, 3)), ((0, 0), (3, 7))])
def test_grad_strides(dtype, out, pads, offsets):
    for vocab in (520, 523):
        logits = logits_of("plain", 11, vocab, TYPES[dtype], 1, pads[0], offsets[0])
        grad, whole = rows_in_buffer(11, vocab, TYPES[out], pads[1], offsets[1])
        check_grad(logits, ids_of(11, vocab, 2), TYPES[out], out=grad)
        assert torch.isnan(whole[:, vocab:]).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 0), (0, 1)])
def test_grad_in_place(dtype, pad, offset):
    for vocab in (520, 523, 9001):
        logits = logits_of("plain", 11, vocab, TYPES[dtype], 1, pad, offset)
        check_grad(logits, ids_of(11, vocab, 2), TYPES[dtype], out=logits)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_grad_of_rows_with_nan_or_infinity(dtype):
    """Rows whose sum is NaN have NaN everywhere, the others keep theirs; a row of -inf with one NaN among them."""
    for pad in (0, 3):
        logits, ids = logits_of("plain", 6, 600, TYPES[dtype], 4, pad), torch.tensor([3, 3, 3, 3, 3, -1], device="cuda")
        logits[0, 7] = INF
        logits[1, 9] = float("nan")
        logits[2] = -INF
        logits[2, 300] = float("nan")
        logits[3] = -INF
        out = drs().token_logprobs(logits, ids)
        one = torch.ones(6, device="cuda")
        grad = drs().token_logprobs_grad(logits, ids, out[3], one, out[1], one)
        assert grad[:3].isnan().all() and (grad[3] == 0).all() and grad[4].isfinite().all() and (grad[5] == 0).all()


def test_the_longest_rows_by_teams():
    """2^21 columns, more rows than clusters take: teams whose segments need most of the shared memory."""
    vocab = 2097152
    for dtype in (torch.float32, torch.bfloat16):
        logits = torch.zeros(320, vocab, dtype=dtype, device="cuda")
        at = torch.tensor([0, 151, 304, 319], device="cuda")
        logits[at] = logits_of("plain", 4, vocab, dtype, 1)
        ids = torch.full((320,), -1, device="cuda")
        ids[at] = torch.tensor([0, 77, vocab - 1, 1234567], device="cuda")
        ids[5] = 9  # a row of zeros: all equal
        out = drs().token_logprobs(logits, ids, 64)
        check_logprobs([t[at] for t in out], logits[at], ids[at], 64)
        assert torch.equal(out[4][5].long(), torch.arange(64, device="cuda")) and int(out[2][5]) == 1
        del logits


def test_many_short_rows():
    logits, ids = logits_of("ties", 100003, 40, torch.float16, 1), ids_of(100003, 40, 1)
    check_logprobs(drs().token_logprobs(logits, ids, 7), logits, ids, 7)


def test_grad_temperatures():
    temps = torch.tensor([0.4, 0.9, 1.7], device="cuda")
    logits, ids = logits_of("plain", 11, 1500, torch.bfloat16, 1), ids_of(11, 1500, 2)
    check_grad(logits, ids, torch.float32, temps, 4)


@pytest.mark.parametrize("temp", [None, 0.7])
def test_grad_against_differences(temp):
    """Central differences in 64 bits of the plain logprob and entropy, step 2^-10. The third derivatives of both along a
    direction v are at most 100 / T^3 max |v|^3 for these rows (|ln p| stays below 20, the derivatives are cumulants
    of v times at most it), so the quotient is off by 2^-20 / 6 of that: below 2e-5 / T^3. The directions have entries of
    +-1, hence the gradient's tolerances add up over the columns."""
    rows, vocab = 8, 60
    temps = None if temp is None else torch.tensor([temp], device="cuda")
    logits, ids = logits_of("plain", rows, vocab, torch.float32, 1), torch.arange(rows, device="cuda") * 7
    norm, entropy = forward_state(logits, ids, temps, rows)
    for which in ("logprob", "entropy"):
        one = torch.ones(rows, device="cuda")
        g, h = (one, None) if which == "logprob" else (None, one)
        grad = drs().token_logprobs_grad(logits, ids, norm, g, entropy, h, temps, rows)
        _, tol = grad_reference(logits, ids, norm, g, entropy, h, temps, rows, torch.float32)
        step = 2.0**-10
        for seed in range(4):
            v = torch.randint(0, 2, (rows, vocab), generator=torch.Generator("cuda").manual_seed(seed), device="cuda",
                              dtype=torch.float64) * 2 - 1
            up = reference(logits.double() + step * v, ids, 0, temps, rows)[which][0]
            down = reference(logits.double() - step * v, ids, 0, temps, rows)[which][0]
            bound = tol.sum(1) + 2e-5 / (temp or 1.0) ** 3
            close((grad.double() * v).sum(1), (up - down) / (2 * step), bound, which)


def test_grad_of_the_forward_calls_own_state():
    """norm and entropy as the forward call writes them: off by their own tolerances, which move ln p by as much."""
    logits, ids = logits_of("peaks", 33, 9000, torch.bfloat16, 1), ids_of(33, 9000, 2)
    lib = drs()
    _, entropy, _, norm, _, _ = lib.token_logprobs(logits, ids)
    exact_norm, exact_entropy = forward_state(logits, ids, None, 1)
    g, h = arriving(33, 3)
    got = lib.token_logprobs_grad(logits, ids, norm, g, entropy, h, out=torch.empty(33, 9000, device="cuda"))
    value, tol = grad_reference(logits, ids, exact_norm, g, exact_entropy, h, None, 1, torch.float32)
    ref = reference(logits, ids, 0)
    off = (ref["log_sum"][1] + ref["entropy"][1] + 2 * U * exact_norm[:, 1].abs())[:, None]
    parts = g.abs()[:, None] + h.abs()[:, None] * (2 + exact_entropy[:, None] + ref["d"].abs().clamp_max(200))
    close(got, value, tol + 2 * off * ref["p"] * parts.double() + (ids.long()[:, None] == torch.arange(9000, device="cuda"))
          * 2 * off * ref["p"] * g.abs()[:, None], "gradient")


def test_graphs_share_nothing():
    """A step captured twice, replayed in turn with other inputs: no workspace is shared."""
    lib = drs()
    logits, ids = logits_of("plain", 12, 9001, torch.bfloat16, 1), ids_of(12, 9001, 2)
    one = torch.ones(12, device="cuda")
    graphs = []
    for _ in range(2):
        out = lib.token_logprobs(logits, ids, 5)
        grad = torch.empty_like(logits)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.token_logprobs(logits, ids, 5, out=out)
            lib.token_logprobs_grad(logits, ids, out[3], one, out=grad)
        graphs.append((graph, out, grad))
    for seed in (4, 5):
        logits.copy_(logits_of("plain", 12, 9001, torch.bfloat16, seed))
        for graph, out, grad in graphs:
            for t in (*out, grad):
                t.fill_(3)
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = lib.token_logprobs(logits, ids, 5)
        want_grad = lib.token_logprobs_grad(logits, ids, want[3], one)
        for _, out, grad in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(grad, want_grad)


def test_tolerances_are_not_vacuous():
    """The logprob's tolerance stays far below what a lost column of weight 1/1000 would change."""
    assert 6 * U * 20 + EX2 + additions(262144) * U < 1e-4
