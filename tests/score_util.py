"""Plain 64-bit forms of the scoring operators with the tolerances of fp32 computation, shared by their tests.

Roundings counted (U = 2^-24, half a step of fp32, relative):
  d = (x - m) / T: the difference, 1 / T, its product with log2 e, that constant and the product with the
      difference: at most 6 U |d|.
  e^d: 2^t to 2^-22 (the bound of ex2.approx), and the error of d.
  S = sum e^d: every term's relative error, and one rounding per addition on the way of a term into the sum. A warp
      takes 256 columns or more at once, whose terms (8 or 16 per lane) are added up first, then the lane's sum of
      them to its sum of the row, at most vocab / 256 times; the lanes' and warps' sums meet in fewer than 20 steps:
      additions() of them in all.
  With D = the mean of |d| under the softmax (= entropy - ln S): S is off by rel = 6 U D + 2^-22 + additions U.
  ln S: rel, and one step of its own value; the logprob d - ln S: the errors of both and a rounding.
  entropy = ln S + D: rel (1 + D), the errors of the weights e^d |d| (with D2, the mean of d^2: 6 U D2 + D (2^-22 +
      6 U + additions U)), and four roundings of its parts."""
import torch

U = 2.0**-24
EX2 = 2.0**-22
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def additions(vocab):
    return vocab // 256 + 32


def half_step(dtype, ref):
    info = torch.finfo(dtype)
    return info.eps / 2 * ref.abs() * (1 + 2.0**-7) + info.tiny * info.eps / 2


def rows_in_buffer(n, width, dtype, pad=0, offset=0):
    """[n, width] inside a buffer whose other places hold NaN (whole: with the places between the rows)."""
    buffer = torch.full((offset + n * (width + pad),), float("nan"), dtype=dtype, device="cuda")
    whole = buffer[offset:].view(n, width + pad)
    return whole[:, :width], whole


def temperature(temps, canvas_len, rows, device):
    if temps is None:
        return torch.ones(rows, 1, dtype=torch.float64, device=device)
    at = torch.arange(rows, device=device) // canvas_len
    return temps.clamp_min(torch.tensor(1e-10, dtype=torch.float32, device=device))[at].double()[:, None]


def reference(logits, ids, k, temps=None, canvas_len=1):
    """Values and tolerances in 64 bits: a dict with value, tol pairs, and the whole numbers."""
    rows, vocab = logits.shape
    x = logits.double()
    te = temperature(temps, canvas_len, rows, x.device)
    m = x.amax(1, keepdim=True)
    d = (x - m) / te
    e = d.exp()
    s = e.sum(1, keepdim=True)
    p = e / s
    drop = p == 0
    dead = (m[:, 0] == -float("inf"))
    dd = torch.where(drop, 0.0, d)
    mean, square = (p * -dd).sum(1, keepdim=True), (p * dd * dd).sum(1, keepdim=True)
    n = additions(vocab)
    rel = 6 * U * mean + EX2 + n * U
    log_s = torch.where(dead[:, None], -float("inf"), s.log())
    tol_log = rel + 4 * U * log_s.abs()
    entropy = log_s + mean
    tol_entropy = rel * (1 + mean) + 6 * U * square + mean * (EX2 + 6 * U + n * U) + 4 * U * (entropy + log_s + mean)
    entropy = torch.where(dead[:, None], 0.0, entropy)
    inside = (ids >= 0) & (ids < vocab)
    at = torch.where(inside, ids, 0).long()[:, None]
    own = d.gather(1, at)

    def lp(dist):
        v = dist - log_s
        return v, 6 * U * dist.abs() + tol_log + 2 * U * v.abs()

    value = x.gather(1, at)
    order = torch.nan_to_num(x, nan=-float("inf"), posinf=float("inf"), neginf=-float("inf")) + 0.0
    best = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
    return {"inside": inside, "logprob": [v[:, 0] for v in lp(own)], "entropy": (entropy[:, 0], tol_entropy[:, 0]),
            "rank": 1 + (x > value).sum(1), "max": m[:, 0], "log_sum": (log_s[:, 0], tol_log[:, 0]), "top_ids": best,
            "top_logprobs": lp(d.gather(1, best)), "p": p, "d": d}


def close(got, ref, tol, what):
    got = got.double()
    same = (got == ref) | (got.isnan() & ref.isnan())
    bad = ~(same | ((got - ref).abs() <= tol))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first {got[bad][:3].tolist()} for " \
                          f"{ref[bad][:3].tolist()}, tolerance {tol[bad][:3].tolist()}"


def check_logprobs(out, logits, ids, k, temps=None, canvas_len=1):
    logprob, entropy, rank, norm, top_ids, top_lps = out
    ref = reference(logits, ids, k, temps, canvas_len)
    one = ref["inside"]
    gone = ~one
    assert torch.equal(rank[one].long(), ref["rank"][one])
    assert torch.equal(top_ids[one].long(), ref["top_ids"][one])
    assert torch.equal(norm[one][:, 0].double().nan_to_num(1.25), ref["max"][one].nan_to_num(1.25))
    for got, name in ((logprob, "logprob"), (entropy, "entropy"), (norm[:, 1], "log_sum"), (top_lps, "top_logprobs")):
        close(got[one], ref[name][0][one], ref[name][1][one], name)
    for got in (logprob, entropy, rank, norm):
        assert (got[gone] == 0).all()
    assert (top_ids[gone] == -1).all() and (top_lps[gone] == -float("inf")).all()
    return ref


def grad_reference(logits, ids, norm, grad_logprob, entropy, grad_entropy, temps, canvas_len, dtype):
    """(value, tolerance) of the gradient from the given norm, in 64 bits. With l = (x - m) / T - L: l is off by
    6 U |d| + 4 U |L| + 2 U |l|, p = e^l by that and 2^-22, the bracket g + h (l + H) by 8 roundings of its parts and
    |h| times l's error; the token's own g (1 - p) by p times l's error and 8 roundings."""
    rows, vocab = logits.shape
    x = logits.double()
    te = temperature(temps, canvas_len, rows, x.device)
    m, log_s = norm[:, :1].double(), norm[:, 1:].double()
    d = (x - m) / te
    l = d - log_s
    p = l.exp()
    zero = torch.zeros(rows, 1, dtype=torch.float64, device=x.device)
    g = zero if grad_logprob is None else grad_logprob.double()[:, None]
    h = zero if grad_entropy is None else grad_entropy.double()[:, None]
    big = zero if grad_entropy is None else entropy.double()[:, None]
    drop = p == 0
    l0, d0 = torch.where(drop, 0.0, l), torch.where(drop, 0.0, d)
    inside = ((ids >= 0) & (ids < vocab) & (m[:, 0] > -float("inf")))[:, None]
    own = torch.arange(vocab, device=x.device) == ids.long()[:, None]
    value = (torch.where(own, g, 0.0) - g * p - h * p * torch.where(drop, 0.0, l + big)) / te
    off = 6 * U * d0.abs() + 4 * U * log_s.abs() + 2 * U * l0.abs()
    parts = g.abs() + h.abs() * (big.abs() + l0.abs())
    tol = (p * (parts * (off + EX2 + 10 * U) + h.abs() * off) + torch.where(own, g.abs() * (p * off + 10 * U), 0.0)) / te
    tol = tol + 2.0**-125 * (parts / te)  # p below the normal range
    value, tol = torch.where(inside, value, 0.0), torch.where(inside, tol, 0.0)
    return value, tol + half_step(dtype, value.abs() + tol)


def logits_of(kind, rows, vocab, dtype, seed, pad=0, offset=0):
    """Rows of the kinds where selection and sums can go wrong."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = 3 * torch.randn(rows, vocab, generator=g, device="cuda")
    inf = float("inf")
    if kind == "ties":
        x = x.round()
    elif kind == "equal":
        x = torch.full_like(x, -1.5)
    elif kind == "rising":
        x = x.sort(1).values
    elif kind == "falling":
        x = x.sort(1, descending=True).values
    elif kind == "peaks":
        x[torch.arange(rows, device="cuda"), torch.randint(0, vocab, (rows,), generator=g, device="cuda")] += 30
    elif kind == "masked":
        x[torch.rand(rows, vocab, generator=g, device="cuda") < 0.9] = -inf
        x[::3] = -inf  # nothing left
        x[1::3, : vocab - 1] = -inf  # one column left
    elif kind == "lowest":
        x[torch.rand(rows, vocab, generator=g, device="cuda") < 0.5] = torch.finfo(dtype).min
        x[::3] = torch.finfo(dtype).min
        x[1::3, : vocab // 2] = -inf
    elif kind == "zeros":
        x = torch.where(torch.rand(rows, vocab, generator=g, device="cuda") < 0.5, 0.0, -0.0)
    elif kind == "far":
        x = x * 100 + 5000
    view, _ = rows_in_buffer(rows, vocab, dtype, pad, offset)
    view.copy_(x)
    return view


def ids_of(rows, vocab, seed, dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000)
    ids = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    ids[1::5] = vocab - 1
    ids[3::7] = -1
    ids[6::7] = vocab
    return ids.to(dtype)
