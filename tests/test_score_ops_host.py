"""The refusals of the scoring operators and of dropout (no GPU needed): the C ABI's argument checks (addresses are made
up and never dereferenced), the binding's checks of types, devices, lengths and autograd, with stand-in tensors."""
import pytest
import torch

import vocab_row_sampling_gb300 as drs
from fake_tensors import FakeStream, FakeTensor
from test_current_device_host import stub  # noqa: F401
from vocab_row_sampling_gb300 import _build

FAKE = 0x7F0000000000
INV, UNS, OK = drs.DRS_ERR_INVALID_ARG, drs.DRS_ERR_UNSUPPORTED, drs.DRS_OK
HUGE = drs.DRS_MAX_VOCAB + 1


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return drs.load()


def _logprobs(lib, logits=FAKE, t=1, rows=4, vocab=16, stride=16, ids=FAKE, bits=64, temps=FAKE, canvas=1, k=4, lp=FAKE,
              entropy=FAKE, rank=FAKE, norm=FAKE, top=FAKE, tops=FAKE):
    return lib.drs_token_logprobs(logits, t, rows, vocab, stride, ids, bits, temps, canvas, k, lp, entropy, rank, norm,
                                  top, tops, None)


@pytest.mark.parametrize("kw,expect", [
    ({"rows": 0}, OK), ({"rows": 0, "logits": None, "lp": None}, OK), ({"rows": -1}, INV), ({"vocab": 0}, INV),
    ({"t": 3}, INV), ({"t": -1}, INV), ({"stride": 15}, INV), ({"bits": 16}, INV), ({"canvas": 0}, INV), ({"k": -1}, INV),
    ({"k": 17}, INV), ({"logits": None}, INV), ({"ids": None}, INV), ({"lp": None}, INV), ({"top": None}, INV),
    ({"tops": None}, INV), ({"logits": FAKE + 1}, INV), ({"t": 0, "logits": FAKE + 2}, INV), ({"ids": FAKE + 4}, INV),
    ({"temps": FAKE + 2}, INV), ({"lp": FAKE + 2}, INV), ({"entropy": FAKE + 1}, INV), ({"rank": FAKE + 2}, INV),
    ({"norm": FAKE + 2}, INV), ({"top": FAKE + 2}, INV), ({"tops": FAKE + 2}, INV), ({"vocab": HUGE, "stride": HUGE}, UNS),
    ({"k": 65, "vocab": 100, "stride": 100}, UNS), ({"rows": drs.DRS_MAX_SCORE_ROWS + 1}, UNS),
])
def test_logprobs_argument_checks(lib, kw, expect):
    assert _logprobs(lib, **kw) == expect


def _grad(lib, logits=FAKE, t=1, rows=4, vocab=16, stride=16, ids=FAKE, bits=64, temps=FAKE, canvas=1, norm=FAKE,
          entropy=FAKE, g=FAKE, h=FAKE, grad=FAKE + 4096, gt=0, gstride=16):
    return lib.drs_token_logprobs_grad(logits, t, rows, vocab, stride, ids, bits, temps, canvas, norm, entropy, g, h, grad,
                                       gt, gstride, None)


@pytest.mark.parametrize("kw,expect", [
    ({"rows": 0}, OK), ({"rows": -1}, INV), ({"vocab": 0}, INV), ({"t": 3}, INV), ({"gt": 3}, INV), ({"stride": 15}, INV),
    ({"gstride": 15}, INV), ({"bits": 8}, INV), ({"canvas": 0}, INV), ({"logits": None}, INV), ({"ids": None}, INV),
    ({"norm": None}, INV), ({"grad": None}, INV), ({"g": None, "h": None}, INV), ({"entropy": None}, INV),
    ({"logits": FAKE + 1}, INV), ({"grad": FAKE + 2}, INV), ({"ids": FAKE + 4}, INV), ({"norm": FAKE + 2}, INV),
    ({"entropy": FAKE + 2}, INV), ({"g": FAKE + 2}, INV), ({"h": FAKE + 1}, INV), ({"temps": FAKE + 2}, INV),
    ({"grad": FAKE}, INV), ({"grad": FAKE, "gt": 1, "gstride": 24}, INV),
    ({"vocab": HUGE, "stride": HUGE, "gstride": HUGE}, UNS), ({"rows": drs.DRS_MAX_SCORE_ROWS + 1}, UNS),
])
def test_logprobs_grad_argument_checks(lib, kw, expect):
    assert _grad(lib, **kw) == expect


def _dropout(lib, x=FAKE, t=1, rows=4, width=16, xstride=16, residual=FAKE + 8192, rstride=16, p=0.1, seed=None, row0=0,
             out=FAKE + 4096, ot=0, ostride=16):
    return lib.drs_dropout(x, t, rows, width, xstride, residual, rstride, p, 1, seed, row0, out, ot, ostride, None)


def _dropout_grad(lib, x=FAKE, t=1, rows=4, width=16, xstride=16, p=0.1, seed=None, row0=0, out=FAKE + 4096, ot=0,
                  ostride=16):
    return lib.drs_dropout_grad(x, t, rows, width, xstride, p, 1, seed, row0, out, ot, ostride, None)


@pytest.mark.parametrize("call", [_dropout, _dropout_grad])
@pytest.mark.parametrize("kw,expect", [
    ({"rows": 0}, OK), ({"rows": -1}, INV), ({"width": 0}, INV), ({"t": 3}, INV), ({"ot": 3}, INV), ({"xstride": 15}, INV),
    ({"ostride": 15}, INV), ({"p": -0.1}, INV), ({"p": 1.5}, INV), ({"p": float("nan")}, INV), ({"row0": -1}, INV),
    ({"row0": 2**63 - 2}, INV), ({"x": None}, INV), ({"out": None}, INV), ({"x": FAKE + 1}, INV), ({"out": FAKE + 2}, INV),
    ({"seed": FAKE + 4}, INV), ({"out": FAKE}, INV), ({"out": FAKE, "ot": 1, "ostride": 24}, INV),
    ({"width": drs.DRS_MAX_WIDTH + 1, "xstride": 1 << 21, "ostride": 1 << 21, "residual": None}, UNS),
    ({"rows": 1 << 60}, UNS),
])
def test_dropout_argument_checks(lib, call, kw, expect):
    if call is _dropout_grad:
        kw = {name: value for name, value in kw.items() if name != "residual"}
    assert call(lib, **kw) == expect


@pytest.mark.parametrize("kw", [{"rstride": 15}, {"residual": FAKE + 8194}, {"out": FAKE + 8192, "ostride": 24}])
def test_dropout_residual_checks(lib, kw):
    assert _dropout(lib, **kw) == INV


# ------------------------------------------------------------- the binding

f32, i32, i64 = torch.float32, torch.int32, torch.int64


def logprobs(gpu=0, stream=None, **kw):
    t = lambda *shape, dtype=f32, name=None: FakeTensor(shape, dtype, gpu, requires_grad=kw.get("grad") == name)  # noqa
    return drs.drs_token_logprobs(t(8, 16, name="x"), t(8, dtype=i64), t(4), 2, t(8, name="out"), t(8), t(8, dtype=i32),
                                  t(8, 2), t(8, 3, dtype=i32), t(8, 3), stream)


def logprobs_grad(gpu=0, stream=None, **kw):
    t = lambda *shape, dtype=f32, name=None: FakeTensor(shape, dtype, gpu, requires_grad=kw.get("grad") == name)  # noqa
    return drs.drs_token_logprobs_grad(t(8, 16, name="x"), t(8, dtype=i32), None, 1, t(8, 2), t(8), t(8), t(8),
                                       t(8, 16, name="out"), stream)


def dropout(gpu=0, stream=None, **kw):
    t = lambda *shape, dtype=f32, name=None: FakeTensor(shape, dtype, gpu, requires_grad=kw.get("grad") == name)  # noqa
    return drs.drs_dropout(t(8, 16, name="x"), t(8, 16, name="residual"), 0.1, t(1, dtype=i64), 0, t(8, 16, name="out"),
                           stream)


def dropout_grad(gpu=0, stream=None, **kw):
    t = lambda *shape, dtype=f32, name=None: FakeTensor(shape, dtype, gpu, requires_grad=kw.get("grad") == name)  # noqa
    return drs.drs_dropout_grad(t(8, 16, name="x"), 0.1, 5, 0, t(8, 16, name="out"), stream)


CALLS = [logprobs, logprobs_grad, dropout, dropout_grad]


@pytest.mark.parametrize("call", CALLS)
def test_devices_and_streams(stub, call):  # noqa: F811
    call()
    assert len(stub.calls) == 1 and stub.calls[0][1][-1] == 1000
    call(0, FakeStream(0, 77))
    assert len(stub.calls) == 2 and stub.calls[1][1][-1] == 77
    with pytest.raises(ValueError, match="current device"):
        call(1)
    with pytest.raises(ValueError, match="stream"):
        call(0, FakeStream(1, 78))
    assert len(stub.calls) == 2


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in ("x", "out")] + [(dropout, "residual")])
def test_tensors_that_require_a_gradient(stub, call, name):  # noqa: F811
    with pytest.raises(ValueError, match="requires a gradient"):
        call(grad=name)
    assert not stub.calls
    with torch.no_grad():
        call(grad=name)
    assert len(stub.calls) == 1


def test_binding_refuses_other_types_shapes_and_lengths(stub):  # noqa: F811
    t = lambda *shape, dtype=f32, gpu=0: FakeTensor(shape, dtype, gpu)  # noqa: E731
    x, ids = t(8, 16), t(8, dtype=i64)
    out = lambda k=3: (t(8), t(8), t(8, dtype=i32), t(8, 2), t(8, k, dtype=i32), t(8, k))  # noqa: E731
    drs.token_logprobs(x, ids, 3, out=out())
    assert len(stub.calls) == 1
    for bad in (dict(logits=t(8, 16, dtype=torch.float64)), dict(logits=t(8)), dict(ids=t(7, dtype=i64)), dict(ids=t(8)),
                dict(ids=t(8, dtype=i64, gpu=1)), dict(temps=t(7)), dict(temps=t(8, dtype=i32)), dict(canvas_len=0),
                dict(k=4), dict(out=out()[:4] + (None, None)), dict(out=out()[:5] + (None,)),
                dict(out=out()[:4] + (t(24, dtype=i32), t(24)), k=24), dict(out=(t(9),) + out()[1:]),
                dict(out=out()[:2] + (t(8),) + out()[3:]), dict(out=out()[:4] + (t(8, 3, dtype=i64), t(8, 3))),
                dict(out=out()[:3] + (t(8),) + out()[4:])):
        with pytest.raises((ValueError, IndexError)):
            drs.token_logprobs(**{**dict(logits=x, ids=ids, k=3, out=out()), **bad})
    drs.token_logprobs_grad(x, ids, t(8, 2), t(8), out=t(8, 16))
    assert len(stub.calls) == 2
    for bad in (dict(out=t(8, 15)), dict(out=t(8, 16, dtype=i32)), dict(norm=t(8)), dict(grad_logprob=t(7)),
                dict(grad_entropy=t(9)), dict(entropy=t(9)), dict(ids=t(9, dtype=i32)), dict(out=t(8, 16, gpu=1))):
        with pytest.raises(ValueError):
            drs.token_logprobs_grad(**{**dict(logits=x, ids=ids, norm=t(8, 2), grad_logprob=t(8), out=t(8, 16)), **bad})
    drs.dropout(x, 0.5, 1, out=t(8, 16))
    assert len(stub.calls) == 3
    for bad in (dict(out=t(8, 15)), dict(out=t(8, 16, dtype=i32)), dict(residual=t(8, 16, dtype=torch.bfloat16)),
                dict(residual=t(7, 16)), dict(seed=t(1)), dict(seed=t(2, dtype=i64)), dict(seed=t(1, dtype=i64, gpu=1)),
                dict(x=t(8)), dict(x=t(8, 16, gpu=1))):
        with pytest.raises(ValueError):
            drs.dropout(**{**dict(x=x, p=0.5, seed=1, out=t(8, 16)), **bad})
    with pytest.raises(ValueError):
        drs.dropout_grad(x, 0.5, 1, out=t(7, 16))
    assert len(stub.calls) == 3


def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 16)
    for call in (lambda: drs.token_logprobs(x, torch.zeros(4, dtype=i64), 2), lambda: drs.dropout(x, 0.5, 1),
                 lambda: drs.token_logprobs_grad(x, torch.zeros(4, dtype=i64), torch.zeros(4, 2), torch.zeros(4)),
                 lambda: drs.dropout_grad(x, 0.5, 1)):
        with pytest.raises(ValueError):
            call()
