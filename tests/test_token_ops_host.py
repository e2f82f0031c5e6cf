"""The token operators' refusals (no GPU needed): the C ABI's argument checks,
which return before anything is launched (the device addresses are made up
and never dereferenced), and the binding's checks of types, devices and
lengths."""
import pytest
import torch

import vocab_row_sampling_gb300 as drs
from vocab_row_sampling_gb300 import _build

FAKE = 0x7F0000000000  # a 256-byte aligned address; never dereferenced
INV, UNS, OK = drs.DRS_ERR_INVALID_ARG, drs.DRS_ERR_UNSUPPORTED, drs.DRS_OK


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return drs.load()


def _verify(lib, target=FAKE, tt=1, trows=8, tstride=16, draft=FAKE, dt=2, drows=4, dstride=16, vocab=16, tokens=FAKE,
            cu=FAKE, requests=4, most=3, au=FAKE, su=FAKE, out=FAKE, acc=FAKE):
    return lib.drs_verify_drafts(target, tt, trows, tstride, draft, dt, drows, dstride, vocab, tokens, cu, requests,
                                 most, au, su, out, acc, None)


@pytest.mark.parametrize("kw,expect", [
    ({"requests": 0}, OK), ({"requests": 0, "target": None}, OK),
    ({"requests": -1}, INV), ({"most": -1}, INV), ({"trows": -1}, INV), ({"drows": -1}, INV),
    ({"tt": 3}, INV), ({"tt": -1}, INV), ({"dt": 3}, INV), ({"vocab": 0}, INV), ({"tstride": 15}, INV),
    ({"dstride": 15}, INV), ({"target": None}, INV), ({"tokens": None}, INV), ({"cu": None}, INV), ({"au": None}, INV),
    ({"su": None}, INV), ({"out": None}, INV), ({"acc": None}, INV), ({"target": FAKE + 1}, INV),
    ({"tt": 0, "target": FAKE + 2}, INV), ({"draft": FAKE + 1}, INV), ({"tokens": FAKE + 4}, INV),
    ({"out": FAKE + 4}, INV), ({"cu": FAKE + 2}, INV), ({"su": FAKE + 1}, INV),
    ({"vocab": drs.DRS_MAX_VOCAB + 1, "tstride": drs.DRS_MAX_VOCAB + 1, "dstride": drs.DRS_MAX_VOCAB + 1}, UNS),
    ({"requests": 1 << 27}, UNS),
])
def test_verify_argument_checks(lib, kw, expect):
    assert _verify(lib, **kw) == expect


def _slots(lib, lens=FAKE, new=FAKE, held=FAKE, requests=4, block=16, table=FAKE, stride=8, most=8, ring=FAKE, size=32,
           state=FAKE, capacity=64, cu=FAKE, request=FAKE, position=FAKE, slot=FAKE, out_held=FAKE, out_state=FAKE,
           lacking=FAKE):
    return lib.drs_map_slots(lens, new, held, requests, block, table, stride, most, ring, size, state, capacity, cu,
                             request, position, slot, out_held, out_state, lacking, None)


@pytest.mark.parametrize("kw,expect", [
    ({"requests": -1}, INV), ({"block": 0}, INV), ({"most": 0}, INV), ({"stride": 7}, INV), ({"size": 0}, INV),
    ({"capacity": -1}, INV), ({"lens": None}, INV), ({"new": None}, INV), ({"held": None}, INV), ({"table": None}, INV),
    ({"ring": None}, INV), ({"state": None}, INV), ({"cu": None}, INV), ({"request": None}, INV),
    ({"position": None}, INV), ({"slot": None}, INV), ({"out_held": None}, INV), ({"out_state": None}, INV),
    ({"lacking": None}, INV), ({"lens": FAKE + 2}, INV), ({"slot": FAKE + 4}, INV), ({"state": FAKE + 4}, INV),
    ({"out_state": FAKE + 4}, INV), ({"requests": drs.DRS_MAX_REQUESTS + 1}, UNS), ({"capacity": 1 << 31}, UNS),
])
def test_slots_argument_checks(lib, kw, expect):
    assert _slots(lib, **kw) == expect


def _embed(lib, table=FAKE, t=1, vocab=16, width=8, tstride=8, ids=FAKE, bits=64, tokens=4, out=FAKE, ostride=8):
    return lib.drs_embed_tokens(table, t, vocab, width, tstride, ids, bits, tokens, 1.0, out, ostride, None)


@pytest.mark.parametrize("kw,expect", [
    ({"tokens": 0}, OK), ({"tokens": -1}, INV), ({"vocab": 0}, INV), ({"width": 0}, INV), ({"t": 3}, INV),
    ({"bits": 16}, INV), ({"tstride": 7}, INV), ({"ostride": 7}, INV), ({"table": None}, INV), ({"ids": None}, INV),
    ({"out": None}, INV), ({"table": FAKE + 1}, INV), ({"out": FAKE + 1}, INV), ({"ids": FAKE + 4}, INV),
    ({"vocab": drs.DRS_MAX_VOCAB + 1}, UNS),
    ({"width": drs.DRS_MAX_WIDTH + 1, "tstride": 1 << 21, "ostride": 1 << 21}, UNS),
])
def test_embed_argument_checks(lib, kw, expect):
    assert _embed(lib, **kw) == expect


def _grad(lib, grad=FAKE, g=1, tokens=4, width=8, gstride=8, ids=FAKE, bits=64, acc=0, table=FAKE, t=0, vocab=16,
          tstride=8, ws=FAKE, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = lib.drs_embed_tokens_grad_workspace_bytes(tokens, vocab, width)
    return lib.drs_embed_tokens_grad(grad, g, tokens, width, gstride, ids, bits, 1.0, acc, table, t, vocab, tstride, ws,
                                     ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    ({"tokens": 0, "acc": 1}, OK), ({"tokens": -1}, INV), ({"vocab": 0}, INV), ({"width": 0}, INV), ({"g": 3}, INV),
    ({"t": 3}, INV), ({"bits": 8}, INV), ({"gstride": 7}, INV), ({"tstride": 7}, INV), ({"grad": None}, INV),
    ({"ids": None}, INV), ({"table": None}, INV), ({"ws": None}, INV), ({"ws_bytes": 64}, INV), ({"ws": FAKE + 8}, INV),
    ({"grad": FAKE + 1}, INV), ({"table": FAKE + 2}, INV), ({"ids": FAKE + 4}, INV),
    ({"vocab": drs.DRS_MAX_VOCAB + 1}, UNS), ({"tokens": drs.DRS_MAX_TOKENS + 1}, UNS),
    ({"width": drs.DRS_MAX_WIDTH + 1, "tstride": 1 << 21, "gstride": 1 << 21}, UNS),
    # more CTAs than a launch has: refused before the sort is launched
    ({"tokens": drs.DRS_MAX_TOKENS, "width": drs.DRS_MAX_WIDTH - 1, "tstride": 1 << 20, "gstride": 1 << 20}, UNS),
])
def test_grad_argument_checks(lib, kw, expect):
    assert _grad(lib, **kw) == expect


def test_grad_workspace_sizes(lib):
    size = drs.drs_embed_tokens_grad_workspace_bytes
    assert size(0, 16, 8) == size(-1, 16, 8) == size(4, 0, 8) == size(4, 16, 0) == 0
    assert size(4, drs.DRS_MAX_VOCAB + 1, 8) == size(drs.DRS_MAX_TOKENS + 1, 16, 8) == 0
    assert size(32768, 262144, 2048) >= 32768 * 8


def test_binding_refuses_other_types_devices_and_lengths():
    """What the library cannot see: CPU tensors, other element types."""
    f, i = torch.zeros(4, 16), torch.zeros(4, dtype=torch.int64)
    cu, u = torch.zeros(5, dtype=torch.int32), torch.zeros(4)
    with pytest.raises(ValueError):
        drs.verify_drafts(f, i, cu, u, u, 3, draft_probs=f)
    with pytest.raises(ValueError):
        drs.verify_drafts(f, i, cu, u, u, -1)
    with pytest.raises(ValueError):
        drs.embed_tokens(f, i)
    with pytest.raises(ValueError):
        drs.embed_tokens_grad(f, i, 1.0, torch.zeros(8, 16))
    n = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        drs.map_slots(n, n, n, torch.zeros(4, 8, dtype=torch.int32), 16, n, torch.zeros(2, dtype=torch.int64), 8)
