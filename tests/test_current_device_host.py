"""The token operators on tensors or streams of another GPU than the current one
(no GPU needed: stand-in tensors and a stub library). The library launches on the
current device, so such calls are refused before they reach it."""
import pytest
import torch

import vocab_row_sampling_gb300 as drs
from fake_tensors import FakeStream, FakeTensor, fake_empty


class StubLibrary:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *a: 4096

        def call(*a):
            self.calls.append((name, a))
            return drs.DRS_OK
        return call


@pytest.fixture
def stub(monkeypatch):
    library = StubLibrary()
    monkeypatch.setattr(drs, "load", lambda *a, **k: library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda gpu: 1000 + gpu, raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch, "empty", fake_empty)
    monkeypatch.setattr(drs, "_stream_workspaces", {})
    drs.drs_embed_tokens_grad_workspace_bytes.cache_clear()
    yield library
    drs.drs_embed_tokens_grad_workspace_bytes.cache_clear()


def verify(gpu, stream=None):
    t = lambda shape, dtype=torch.float32: FakeTensor(shape, dtype, gpu)
    return drs.drs_verify_drafts(t((8, 16)), t((4, 16)), t((4,), torch.int64), t((5,), torch.int32), t((4,)), t((4,)),
                                 t((4, 3), torch.int64), t((4,), torch.int32), stream)


def slots(gpu, stream=None):
    i32 = lambda *shape: FakeTensor(shape, torch.int32, gpu)
    i64 = lambda *shape: FakeTensor(shape, torch.int64, gpu)
    return drs.drs_map_slots(i32(4), i32(4), i32(4), i32(4, 8), 16, i32(32), i64(2), i32(5), i32(64), i32(64), i64(64),
                             i32(4), i64(2), i32(1), stream)


def embed(gpu, stream=None):
    return drs.drs_embed_tokens(FakeTensor((16, 8), gpu=gpu), FakeTensor((4,), torch.int64, gpu), 1.0,
                                FakeTensor((4, 8), gpu=gpu), stream)


def grad(gpu, stream=None):
    return drs.drs_embed_tokens_grad(FakeTensor((4, 8), gpu=gpu), FakeTensor((4,), torch.int64, gpu), 1.0, False,
                                     FakeTensor((16, 8), gpu=gpu), FakeTensor((4096,), torch.uint8, gpu), stream)


def grad_wrapper(gpu, stream=None):
    return drs.embed_tokens_grad(FakeTensor((4, 8), gpu=gpu), FakeTensor((4,), torch.int64, gpu), 1.0,
                                 FakeTensor((16, 8), gpu=gpu), stream=stream)


CALLS = [verify, slots, embed, grad, grad_wrapper]


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_the_current_device(stub, call):
    call(0)
    assert len(stub.calls) == 1 and stub.calls[0][1][-1] == 1000


@pytest.mark.parametrize("call", CALLS)
def test_tensors_of_another_device_are_refused(stub, call):
    with pytest.raises(ValueError, match="current device"):
        call(1)
    assert not stub.calls


@pytest.mark.parametrize("call", CALLS[:-1])
def test_streams(stub, call):
    call(0, FakeStream(0, 77))
    assert len(stub.calls) == 1 and stub.calls[0][1][-1] == 77
    with pytest.raises(ValueError, match="stream"):
        call(0, FakeStream(1, 78))
    assert len(stub.calls) == 1
