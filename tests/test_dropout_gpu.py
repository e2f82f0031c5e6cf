"""drs_dropout and drs_dropout_grad against a plain form with its own Philox4x32-10 (whole numbers in numpy), values in
64 bits. Tolerance: the scale and the product are rounded (2 U of the product), the sum with the residual (U of it), then
the result to its type (half a step)."""
import numpy as np
import pytest
import torch

from gpu_util import drs
from score_util import TYPES, U, close, half_step, rows_in_buffer

pytestmark = pytest.mark.gpu
SEED = 0x9E3779B97F4A7C15


def philox(counter, seed):
    c = [np.asarray(w, dtype=np.uint64) for w in np.broadcast_arrays(*counter)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    low, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> half) ^ c[1] ^ np.uint64(k0), b & low, (a >> half) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def kept(rows, width, p, seed, row0=0):
    """The mask as a numpy array, and 1 - q."""
    group = np.arange((width + 7) // 8, dtype=np.uint64)[None, :]
    row = np.array([row0 + r for r in range(rows)], dtype=np.uint64)[:, None]
    words = philox((group, np.uint64(0x64726F70), row & np.uint64(0xFFFFFFFF), row >> np.uint64(32)), seed)
    halves = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 2).reshape(rows, -1)
    dropped = int(np.floor(float(np.float32(p)) * 65536 + 0.5))
    return halves[:, :width] >= dropped, 1 - dropped / 65536


def filled(rows, width, dtype, seed, pad=0, offset=0):
    view, whole = rows_in_buffer(rows, width, dtype, pad, offset)
    view.copy_(torch.randn(rows, width, generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
    return view, whole


def check(got, x, p, seed, residual=None, row0=0):
    mask, keep = kept(*x.shape, p, seed, row0)
    mask = torch.as_tensor(mask).cuda()
    ref = torch.where(mask, x.double() / keep if keep else 0.0, 0.0)  # what is dropped has no part in it
    tol = 2 * U * ref.abs()
    if residual is not None:
        ref = ref + residual.double()
        tol = tol + U * (ref.abs() + tol)
    close(got, ref, tol + half_step(got.dtype, ref.abs() + tol), "dropout")
    if residual is None:
        assert (got[~mask] == 0).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("width", [1, 2, 7, 8, 9, 64, 100, 1000, 1283, 2048, 4104])
def test_sizes(dtype, out, width):
    for rows in (1, 3, 130):
        x, _ = filled(rows, width, TYPES[dtype], width)
        residual, _ = filled(rows, width, TYPES[out], width + 1)
        target = torch.empty(rows, width, dtype=TYPES[out], device="cuda")
        check(drs().dropout(x, 0.3, SEED, out=target), x, 0.3, SEED)
        check(drs().dropout(x, 0.3, 12345, residual=residual, row0=7), x, 0.3, 12345, residual, 7)
        check(drs().dropout_grad(x, 0.3, SEED, row0=2**33 + 5, out=target), x, 0.3, SEED, None, 2**33 + 5)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("pads,offsets", [((1, 0, 0), (0, 0, 0)), ((0, 1, 2), (1, 0, 0)), ((8, 8, 8), (8, 8, 8)),
                                          ((3, 3, 3), (5, 5, 5)), ((24, 0, 5), (0, 3, 1))])
def test_strides(dtype, out, pads, offsets):
    for width in (520, 523):
        x, _ = filled(21, width, TYPES[dtype], 1, pads[0], offsets[0])
        residual, _ = filled(21, width, TYPES[out], 2, pads[1], offsets[1])
        target, whole = rows_in_buffer(21, width, TYPES[out], pads[2], offsets[2])
        check(drs().dropout(x, 0.1, SEED, residual=residual, out=target), x, 0.1, SEED, residual)
        assert torch.isnan(whole[:, width:]).all()
        check(drs().dropout_grad(x, 0.1, SEED, out=target), x, 0.1, SEED)


@pytest.mark.parametrize("p", [0.0, 2.0**-17, 2.0**-16, 1e-7, 0.5, 0.999, 1 - 2.0**-16, 1 - 2.0**-18, 1.0])
def test_probabilities(p):
    x, _ = filled(17, 1000, torch.float32, 1)
    residual, _ = filled(17, 1000, torch.float32, 2)
    check(drs().dropout(x, p, SEED), x, p, SEED)
    check(drs().dropout(x, p, SEED, residual=residual), x, p, SEED, residual)


@pytest.mark.parametrize("p", [1.0, 1 - 2.0**-18, 0.0])
@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 5)])
def test_all_and_nothing_dropped_in_strided_rows(p, pad, offset):
    for dtype in TYPES.values():
        x, _ = filled(9, 203, torch.float32, 1, pad, offset)
        x[0, 0] = float("nan") if p else 1.0
        residual, _ = filled(9, 203, dtype, 2, pad, offset)
        out, whole = rows_in_buffer(9, 203, dtype, pad, offset)
        check(drs().dropout(x, p, SEED, residual=residual, out=out), x, p, SEED, residual)
        assert torch.isnan(whole[:, 203:]).all()
        check(drs().dropout_grad(x, p, SEED, out=out), x, p, SEED)
        assert torch.isnan(whole[:, 203:]).all()


@pytest.mark.parametrize("p", [1.0, 0.25])
def test_rows_that_lie_2_gib_apart(p):
    stride = 2**30 + 8
    whole = torch.empty(2 * stride + 203, dtype=torch.bfloat16, device="cuda")
    out = whole.as_strided((3, 203), (stride, 1))
    out.fill_(float("nan"))
    beyond = whole.as_strided((2, 16), (stride, 1), 203)
    beyond.fill_(5.0)
    x, _ = filled(3, 203, torch.float32, 1)
    check(drs().dropout(x, p, SEED, out=out), x, p, SEED)
    out.fill_(float("nan"))
    check(drs().dropout_grad(x, p, SEED, out=out), x, p, SEED)
    assert (beyond == 5.0).all()


def test_all_dropped_in_a_graph():
    x, _ = filled(9, 203, torch.bfloat16, 1, 3, 5)
    out, whole = rows_in_buffer(9, 203, torch.bfloat16, 3, 5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        drs().dropout(x, 1.0, SEED, out=out)
    for _ in range(2):
        out.fill_(3.0)
        graph.replay()
        assert (out == 0).all() and torch.isnan(whole[:, 203:]).all()


def test_the_share_dropped():
    """Of n = 2^22 draws the dropped are within 6 standard deviations (n q (1 - q))^(1/2) of n q; the numbers are fixed by
    the seed, so the test cannot fail by chance after its first run."""
    x = torch.ones(1024, 4096, device="cuda")
    for p in (0.1, 0.5):
        q = int(p * 65536 + 0.5) / 65536
        dropped = int((drs().dropout(x, p, 1) == 0).sum())
        assert abs(dropped - 2**22 * q) < 6 * (2**22 * q * (1 - q)) ** 0.5


def test_nothing_of_the_dropped_remains():
    for special in (float("nan"), float("inf"), -float("inf")):
        x = torch.full((9, 333), special, device="cuda")
        mask = torch.as_tensor(kept(9, 333, 0.4, SEED)[0]).cuda()
        out = drs().dropout(x, 0.4, SEED)
        assert (out[~mask] == 0).all() and not out[mask].isfinite().any()
        residual = torch.ones(9, 333, device="cuda")
        assert (drs().dropout(x, 0.4, SEED, residual=residual)[~mask] == 1).all()


@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 0), (0, 1)])
def test_in_place(pad, offset):
    for dtype in TYPES.values():
        for width in (64, 523, 4099):
            x, _ = filled(33, width, dtype, 1, pad, offset)
            residual, _ = filled(33, width, dtype, 2, pad, offset)
            want = drs().dropout(x, 0.2, 5, residual=residual)
            drs().dropout(x, 0.2, 5, residual=residual, out=residual)
            assert torch.equal(residual, want)
            want = drs().dropout(x, 0.2, 5)
            drs().dropout(x, 0.2, 5, out=x)
            assert torch.equal(x, want)


def test_one_batch_in_several_calls():
    x, _ = filled(50, 777, torch.bfloat16, 1)
    whole = drs().dropout(x, 0.25, 3, row0=10)
    parts = torch.cat([drs().dropout(x[:13], 0.25, 3, row0=10), drs().dropout(x[13:], 0.25, 3, row0=23)])
    assert torch.equal(whole, parts)


def test_gradient_against_differences():
    """The call is linear in x, so that a difference over any step is the derivative: with integers of up to 8 bits and
    q = 1/2 (a scale of 2) all of it is exact."""
    g = torch.Generator("cuda").manual_seed(1)
    x, v, up = (torch.randint(-99, 100, (31, 259), generator=g, device="cuda").float() for _ in range(3))
    residual = torch.ones(31, 259, device="cuda")
    moved = drs().dropout(x + v, 0.5, SEED, residual=residual) - drs().dropout(x, 0.5, SEED, residual=residual)
    grad = drs().dropout_grad(up, 0.5, SEED)
    assert (moved.double() * up).sum() == (grad.double() * v).sum()


def test_seeds_on_the_gpu_and_graphs():
    """A captured call draws from the seed that stands in the tensor at each replay; the host's integers and both integer
    types give the same masks."""
    lib = drs()
    x, _ = filled(40, 1003, torch.bfloat16, 1)
    seed = torch.tensor([SEED - 2**64], device="cuda")
    assert torch.equal(lib.dropout(x, 0.3, seed), lib.dropout(x, 0.3, SEED))
    assert torch.equal(lib.dropout(x, 0.3, seed), lib.dropout(x, 0.3, SEED - 2**64))
    assert torch.equal(lib.dropout(x, 0.3, seed.view(torch.uint64)), lib.dropout(x, 0.3, SEED))
    out, grad = torch.empty_like(x), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.dropout(x, 0.3, seed, out=out)
        lib.dropout_grad(x, 0.3, seed, out=grad)
        seed += 1
    for step in range(3):
        at = int(seed)
        graph.replay()
        torch.cuda.synchronize()
        check(out, x, 0.3, at % 2**64)
        assert torch.equal(out, grad) and int(seed) == at + 1


def test_streams():
    """Calls on other streams, at the same time, and the two outputs allocated on theirs."""
    lib = drs()
    x, _ = filled(500, 1003, torch.bfloat16, 1)
    want = lib.dropout(x, 0.3, SEED)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [(lib.dropout(x, 0.3, SEED, stream=s), lib.dropout_grad(x, 0.3, SEED, stream=s)) for s in streams]
    torch.cuda.synchronize()
    for out, grad in outs:
        assert torch.equal(out, want) and torch.equal(grad, want)


def test_x_residual_and_out_are_one():
    for width in (64, 333):
        x, _ = filled(21, width, torch.float32, 1)
        want = drs().dropout(x, 0.4, 9, residual=x)
        assert torch.equal(drs().dropout(x, 0.4, 9, residual=x, out=x), want)


@pytest.mark.parametrize("width", [1048576, 1048575])
def test_the_widest_rows(width):
    x, _ = filled(3, width, torch.bfloat16, 1)
    check(drs().dropout(x, 0.3, SEED), x, 0.3, SEED)


def test_empty_calls_and_rows_behind_the_last():
    assert drs().dropout(torch.zeros(0, 5, device="cuda"), 0.5, 1).shape == (0, 5)
    x = torch.ones(4, 100, device="cuda")
    out = torch.full((6, 100), 77.0, device="cuda")
    drs().dropout(x, 0.5, 1, out=out[:4])
    assert (out[4:] == 77).all()


def test_offsets_past_32_bits():
    rows, width = 34000, 131080
    x = torch.ones(rows, width, dtype=torch.bfloat16, device="cuda")
    out = drs().dropout(x, 0.5, SEED, out=x)
    check(out[-3:], torch.ones(3, width, dtype=torch.bfloat16, device="cuda"), 0.5, SEED, None, rows - 3)


def test_apart_from_the_samplers_noise():
    """The same seed, row and columns as the Gumbel noise give other bits."""
    bits, _ = drs().philox_gumbel(SEED, 0, 1, 4096)
    drawn = kept(1, 4096, 0.5, SEED)[0]
    noise = ((bits.cpu().numpy().astype(np.int64) & 0xFFFF) >= 32768)[0]
    assert 0.45 < (noise == drawn[0]).mean() < 0.55
