"""drs_embed_tokens and drs_embed_tokens_grad against plain implementations in
64 bits, and the gradient against differences of the lookup.

Tolerances, from the roundings. Lookup: the fp32 product (2^-24 relative)
and the rounding to the type (half a step: eps / 2 relative, or half the
smallest subnormal). Gradient: n fp32 additions in any order are off by at
most n 2^-24 times the sum of magnitudes, then the product by the scale
(2^-24), the addition to the old value when accumulating (2^-24) and the
rounding to the type."""
import numpy as np
import pytest
import torch

from gpu_util import drs

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0**-24


def half_step(dtype, ref):
    info = torch.finfo(dtype)
    return info.eps / 2 * ref.abs() * (1 + 2.0**-7) + info.tiny * info.eps / 2


def rows(n, width, dtype, seed, pad=0, offset=0, scale=1.0):
    """[n, width] inside a buffer whose other places hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buffer = torch.full((offset + n * (width + pad),), float("nan"), dtype=dtype, device="cuda")
    view = buffer[offset:].view(n, width + pad)[:, :width]
    view.copy_(scale * torch.randn(n, width, generator=g, device="cuda"))
    return view


def some_ids(n, vocab, seed, kind="zipf"):
    rng = np.random.default_rng(seed)
    if kind == "zipf":
        ids = np.minimum(np.exp(rng.random(n) * np.log(vocab + 1)).astype(np.int64), vocab) - 1
        ids = ids * 7919 % vocab
    elif kind == "one":
        ids = np.full(n, vocab // 2)
    elif kind == "distinct":
        ids = rng.permutation(max(n, vocab))[:n] % vocab
    elif kind == "two":
        ids = np.where(rng.random(n) < 0.5, 0, vocab - 1)
    elif kind == "none":
        ids = np.full(n, -1)
    else:  # padding and garbage among the others
        ids = rng.integers(0, vocab, n)
        ids[rng.random(n) < 0.3] = -1
        ids[rng.random(n) < 0.1] = vocab
        ids[rng.random(n) < 0.05] = -(2**31)
        ids[rng.random(n) < 0.05] = 2**31 - 1
    return ids.astype(np.int64)


def check_lookup(table, ids, scale, id_type=torch.int64, out=None):
    vocab, width = table.shape
    ids_gpu = torch.as_tensor(ids).to(id_type).cuda()
    got = drs().embed_tokens(table, ids_gpu, scale, out=out)
    inside = torch.as_tensor((ids >= 0) & (ids < vocab)).cuda()
    ref = table.double()[torch.as_tensor(np.where(inside.cpu().numpy(), ids, 0)).cuda()] * float(np.float32(scale))
    ref = torch.where(inside[:, None], ref, 0.0)
    err = (got.double() - ref).abs()
    assert got.shape == (len(ids), width) and got.dtype == table.dtype
    tol = half_step(table.dtype, ref) + (U * ref.abs() if table.dtype != torch.float32 else 0)
    assert (err <= tol).all(), float((err - tol).max())
    assert (got[~inside] == 0).all()
    return got


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("width", [1, 2, 7, 8, 64, 100, 1000, 1283, 2048, 4104])
def test_lookup_widths(dtype, width):
    table = rows(517, width, TYPES[dtype], width)
    for n, id_type in ((1, torch.int64), (3, torch.int32), (130, torch.int64), (1025, torch.int32)):
        check_lookup(table, some_ids(n, 517, n, "mixed"), width**0.5, id_type)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (8, 8), (3, 5), (24, 0)])
def test_lookup_strides(dtype, pad, offset):
    table = rows(300, 520, TYPES[dtype], pad, pad, offset)
    out = rows(77, 520, TYPES[dtype], 1, pad, offset)
    whole = out.as_strided((77, 520 + pad), (520 + pad, 1), out.storage_offset())
    check_lookup(table, some_ids(77, 300, 3, "mixed"), 1.0, out=out)
    # the places between the rows keep what they held (the last row's lie past the buffer's end)
    assert torch.isnan(whole[:-1, 520:]).all()


def test_lookup_special_values_and_empty_calls():
    """scale 1 copies every finite value and infinity bit for bit; NaN stays NaN."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(256, 256)
    for dtype in (torch.bfloat16, torch.float16):
        table = bits.view(dtype).cuda()
        got = drs().embed_tokens(table, torch.arange(256).cuda(), 1.0)
        nan = torch.isnan(table)
        assert torch.equal(got.view(torch.int16)[~nan], table.view(torch.int16)[~nan])
        assert torch.isnan(got[nan]).all()
    assert drs().embed_tokens(table, torch.zeros(0, dtype=torch.int64).cuda(), 1.0).shape == (0, 256)


def test_lookup_offsets_past_32_bits():
    """A table of over 2^32 elements: the last rows are reached."""
    vocab, width = 1 << 21, 2064
    table = torch.zeros(vocab, width, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    table[-3:] = torch.randn(3, width, generator=g, device="cuda").bfloat16()
    ids = torch.tensor([vocab - 1, 0, vocab - 3, vocab - 2]).cuda()
    assert torch.equal(drs().embed_tokens(table, ids, 1.0), table[ids])


def grad_reference(grad, ids, scale, vocab, old=None):
    """(values, tolerance without the final rounding) in 64 bits."""
    ids = torch.as_tensor(ids).cuda()
    keep = ((ids >= 0) & (ids < vocab)).nonzero().flatten()
    width = grad.shape[1]
    g = grad[keep].double()
    total = torch.zeros(vocab, width, dtype=torch.float64, device="cuda").index_add_(0, ids[keep], g)
    size = torch.zeros(vocab, width, dtype=torch.float64, device="cuda").index_add_(0, ids[keep], g.abs())
    count = torch.bincount(ids[keep], minlength=vocab).double()[:, None]
    s = float(np.float32(scale))
    ref = total * s
    tol = s * size * count * U + ref.abs() * U
    if old is not None:
        ref = ref + old.double()
        tol = tol + ref.abs() * U
    return ref, tol * 1.01


def check_grad(grad, ids, scale, table, accumulate=False, id_type=torch.int64):
    vocab, width = table.shape
    old = table.clone() if accumulate else None
    if not accumulate:
        table.fill_(float("nan"))
    ids_gpu = torch.as_tensor(ids).to(id_type).cuda()
    drs().embed_tokens_grad(grad, ids_gpu, scale, table, accumulate)
    ref, tol = grad_reference(grad, ids, scale, vocab, old)
    tol = tol + half_step(table.dtype, ref)
    err = (table.double() - ref).abs()
    assert (err <= tol).all(), float((err - tol).max())
    hit = torch.zeros(vocab, dtype=torch.bool)
    hit[torch.as_tensor(ids[(ids >= 0) & (ids < vocab)])] = True
    hit = hit.cuda()
    if accumulate:
        assert torch.equal(table[~hit], old[~hit])  # not touched
    else:
        assert (table[~hit] == 0).all()


@pytest.mark.parametrize("grad", list(TYPES))
@pytest.mark.parametrize("table", list(TYPES))
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_types(grad, table, accumulate):
    for n, width in ((300, 256), (77, 129)):
        g = rows(n, width, TYPES[grad], n)
        t = rows(1000, width, TYPES[table], 5)
        check_grad(g, some_ids(n, 1000, n, "mixed"), 1.7, t, accumulate, torch.int32 if accumulate else torch.int64)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 1000, 1024, 1025, 4096, 4097, 9001])
@pytest.mark.parametrize("kind", ["zipf", "one", "distinct", "two", "mixed", "none"])
def test_grad_lengths_and_repetition(n, kind):
    """From one id for every token to none repeated."""
    g = rows(n, 72, torch.bfloat16, n)
    t = rows(3001, 72, torch.float32, 6)
    check_grad(g, some_ids(n, 3001, n, kind), 0.5, t)
    check_grad(g, some_ids(n, 3001, n + 1, kind), 0.5, t, accumulate=True)


@pytest.mark.parametrize("vocab", [1, 2, 5, 1023, 1024, 2047, 2048, 65536, 262144, 1 << 21])
def test_grad_vocabularies(vocab):
    """One and two digits of the sort, and their borders; the sort by one
    cluster and, above 131072 tokens, by tiles."""
    for n in (500, 20000, 131072, 131073):
        g = rows(n, 16, torch.float32, n)
        t = torch.empty(vocab, 16, device="cuda")
        check_grad(g, some_ids(n, vocab, n, "mixed"), 1.0, t)


@pytest.mark.parametrize("width", [1, 3, 8, 40, 264, 1283, 2048, 5000])
def test_grad_widths(width):
    g = rows(700, width, torch.float16, width, scale=0.1)
    t = torch.empty(400, width, dtype=torch.bfloat16, device="cuda")
    check_grad(g, some_ids(700, 400, width), 2.0, t)


@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (8, 8), (3, 5)])
def test_grad_strides(pad, offset):
    g = rows(500, 264, torch.bfloat16, 1, pad, offset)
    t = rows(300, 264, torch.float16, 2, pad, offset)
    whole = t.as_strided((299, 264 + pad), (264 + pad, 1), t.storage_offset())
    for accumulate in (True, False):
        check_grad(g, some_ids(500, 300, 3), 0.3, t, accumulate)
        assert torch.isnan(whole[:, 264:]).all()


def test_grad_many_tokens_and_equal_bits():
    """More tokens than the sort's tiles hold at once, a token in a third of
    them; two calls give equal bits, whatever the workspace held."""
    lib = drs()
    n, vocab, width = 300007, 262144, 24
    ids = some_ids(n, vocab, 1)
    ids[::3] = 77
    g = rows(n, width, torch.float32, 1)
    t = torch.empty(vocab, width, device="cuda")
    check_grad(g, ids, 1.0, t)
    ws = torch.empty(lib.drs_embed_tokens_grad_workspace_bytes(n, vocab, width), dtype=torch.uint8, device="cuda")
    first = t.clone()
    for fill in (0, 255, 127):
        ws.fill_(fill)
        t.fill_(float("nan"))
        lib.drs_embed_tokens_grad(g, torch.as_tensor(ids).cuda(), 1.0, False, t, ws)
        assert torch.equal(t.view(torch.int32), first.view(torch.int32))


@pytest.mark.parametrize("width", [64, 4096, 4100])
def test_grad_equal_bits_over_many_calls(width):
    """Ids that cross many pieces, whose parts different CTAs may add up: the
    order of the sums does not change with who does."""
    lib = drs()
    ids = some_ids(5000, 600, 2)
    ids[::4] = 5
    ids[1::4] = 599
    g = rows(5000, width, torch.bfloat16, 4)
    t = torch.zeros(600, width, device="cuda")
    check_grad(g, ids, 1.0, t)
    ids = torch.as_tensor(ids).cuda()
    first = t.clone()
    for _ in range(30):
        lib.embed_tokens_grad(g, ids, 1.0, t)
        assert torch.equal(t, first)


def test_grad_of_no_tokens():
    t = torch.ones(100, 33, device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    drs().embed_tokens_grad(torch.zeros(0, 33, device="cuda"), none, 1.0, t, accumulate=True)
    assert (t == 1).all()
    drs().embed_tokens_grad(torch.zeros(0, 33, device="cuda"), none, 1.0, t)
    assert (t == 0).all()


@pytest.mark.parametrize("width", [2064, 2051])
def test_grad_offsets_past_32_bits(width):
    """A table of over 2^32 elements: its last rows receive sums, its others zeros."""
    vocab = 1 << 21
    t = torch.full((vocab, width), 7.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([vocab - 1, 0, vocab - 3, vocab - 1]).cuda()
    g = rows(4, width, torch.float32, 1)
    drs().embed_tokens_grad(g, ids, 1.0, t)
    want = torch.stack([g[2], torch.zeros_like(g[0]), g[0] + g[3]]).bfloat16()
    assert torch.equal(t[-3:], want) and torch.equal(t[0], g[1].bfloat16())
    assert int(t.count_nonzero()) == int(t[-3:].count_nonzero()) + int(t[0].count_nonzero())
    drs().embed_tokens_grad(g, ids, 1.0, t, accumulate=True)
    assert torch.equal(t[-1], (want[2].float() + (g[0] + g[3])).bfloat16())


def test_grad_against_differences():
    """The lookup is linear in its table, so a difference of the loss
    sum(c * embed(table)) along a direction d is the product of the gradient
    with d. Powers of two for the scale and the step and small integers for
    the rest make every operation exact."""
    lib = drs()
    g = torch.Generator().manual_seed(3)
    vocab, width, n = 50, 24, 200
    ids = torch.randint(-1, vocab, (n,), generator=g).cuda()
    c = torch.randint(-3, 4, (n, width), generator=g).float().cuda()
    table = torch.randint(-8, 9, (vocab, width), generator=g).float().cuda()
    grad = lib.embed_tokens_grad(c, ids, 4.0, torch.empty(vocab, width, device="cuda"))
    for _ in range(5):
        d = torch.randint(-2, 3, (vocab, width), generator=g).float().cuda()
        up, down = (float((c.double() * lib.embed_tokens(table + h * d, ids, 4.0).double()).sum()) for h in (0.5, -0.5))
        assert up - down == float((grad.double() * d.double()).sum())


def test_workspaces_of_streams():
    """Calls of growing and shrinking sizes, in turn on three streams that run
    at the same time, and inside a graph whose workspace is its own."""
    lib = drs()
    streams = [torch.cuda.Stream() for _ in range(3)]
    sizes = [(40, 64), (3000, 512), (200, 1024), (9000, 256), (10, 8)]
    cases = []
    for k, (n, width) in enumerate(sizes):
        g, ids = rows(n, width, torch.bfloat16, k), torch.as_tensor(some_ids(n, 700, k)).cuda()
        cases.append((g, ids, lib.embed_tokens_grad(g, ids, 1.0, torch.empty(700, width, device="cuda"))))
    outs = [[torch.empty_like(want) for _, _, want in cases] for _ in streams]
    graph = torch.cuda.CUDAGraph()
    captured = torch.empty_like(cases[1][2])
    with torch.cuda.graph(graph):
        lib.embed_tokens_grad(cases[1][0], cases[1][1], 1.0, captured)
    torch.cuda.synchronize()
    for repeat in range(4):
        graph.replay()
        for k, (g, ids, _) in enumerate(cases):
            for st, out in zip(streams, outs):
                lib.embed_tokens_grad(g, ids, 1.0, out[k], stream=st)
    torch.cuda.synchronize()
    assert torch.equal(captured, cases[1][2])
    for out in outs:
        for got, (_, _, want) in zip(out, cases):
            assert torch.equal(got, want)


def test_streams_and_graphs():
    """Both calls on another stream than the tensors' own, and a training step
    of both captured into a graph and replayed on new ids."""
    lib = drs()
    table = rows(4000, 512, torch.bfloat16, 1)
    ids = torch.as_tensor(some_ids(900, 4000, 2)).cuda()
    up = rows(900, 512, torch.bfloat16, 3)
    want = lib.embed_tokens_grad(up, ids, 2.0, torch.empty(4000, 512, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grad = torch.empty(4000, 512, device="cuda")
    got = lib.embed_tokens(table, ids, 2.0, stream=side)
    lib.embed_tokens_grad(up, ids, 2.0, grad, stream=side)
    side.synchronize()
    assert torch.equal(got, lib.embed_tokens(table, ids, 2.0)) and torch.equal(grad, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lib.embed_tokens(table, ids, 2.0)
        lib.embed_tokens_grad(got, ids, 2.0, grad)
    for seed in (5, 6):
        ids.copy_(torch.as_tensor(some_ids(900, 4000, seed, "mixed")))
        graph.replay()
        rows_now = lib.embed_tokens(table, ids, 2.0)
        assert torch.equal(got, rows_now)
        assert torch.equal(grad, lib.embed_tokens_grad(rows_now, ids, 2.0, torch.empty(4000, 512, device="cuda")))
