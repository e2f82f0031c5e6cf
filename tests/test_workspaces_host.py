"""The gradient's workspaces under host threads (no GPU needed): the library is
a stub that sees which workspace each call got. A call makes several launches
and the interpreter runs other threads meanwhile, so a workspace belongs to one
call until that call's launches are all on the stream."""
import threading

import pytest
import torch

import vocab_row_sampling_gb300 as drs
from fake_tensors import FakeTensor, fake_empty


class StubLibrary:
    """Holds every call for a moment and notes the workspaces in use at once."""

    def __init__(self, wait=0.3):
        self.wait = wait
        self.lock, self.held, self.shared, self.calls = threading.Lock(), [], [], []

    def drs_embed_tokens_grad_workspace_bytes(self, tokens, vocab, width):
        return tokens * 4096

    def drs_embed_tokens_grad(self, *args):
        workspace, size = args[-3], args[-2]
        with self.lock:
            self.shared += [workspace] if workspace in self.held else []
            self.held.append(workspace)
            self.calls.append((workspace, size))
        threading.Event().wait(self.wait)
        with self.lock:
            self.held.remove(workspace)
        return drs.DRS_OK


@pytest.fixture
def stub(monkeypatch):
    library = StubLibrary()
    monkeypatch.setattr(drs, "load", lambda *a, **k: library)
    monkeypatch.setattr(drs, "_raw_stream", lambda stream, gpu: 0 if stream is None else stream.cuda_stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch, "empty", fake_empty)
    drs.drs_embed_tokens_grad_workspace_bytes.cache_clear()
    monkeypatch.setattr(drs, "_stream_workspaces", {})
    yield library
    drs.drs_embed_tokens_grad_workspace_bytes.cache_clear()


def grad_call(tokens, width=8, vocab=16):
    table = FakeTensor((vocab, width))
    assert drs.embed_tokens_grad(FakeTensor((tokens, width)), FakeTensor((tokens,), torch.int64), 1.0, table) is table


@pytest.mark.parametrize("tokens", [(4, 4), (4, 64), (64, 4), (4, 4, 4, 4), (4, 100000, 100000)])
def test_calls_of_several_threads_never_hold_one_workspace(stub, tokens):
    failed = []

    def call(n):
        try:
            grad_call(n)
        except BaseException as e:
            failed.append(e)

    for _ in range(2):  # on first use, and with a workspace kept from before
        threads = [threading.Thread(target=call, args=(n,)) for n in tokens]
        for t in threads:
            t.start()
        for t in threads:
            t.join(timeout=30)
    assert not failed and len(stub.calls) == 2 * len(tokens)
    assert not stub.shared
    assert sorted(size for _, size in stub.calls)[0] >= 4 * 4096 and all(workspace for workspace, _ in stub.calls)


def test_a_call_from_within_a_call(stub, monkeypatch):
    """A finaliser that runs while a call allocates may call again on the same thread."""
    stub.wait, allocate, depth = 0.0, torch.empty, []

    def empty(*a, **k):
        if not depth:
            depth.append(1)
            grad_call(8)
        return allocate(*a, **k)

    monkeypatch.setattr(torch, "empty", empty)
    done = threading.Thread(target=grad_call, args=(4,), daemon=True)
    done.start()
    done.join(timeout=10)
    assert not done.is_alive() and len(stub.calls) == 2 and not stub.shared


def test_what_is_kept_is_bounded(stub, monkeypatch):
    """A large call's workspace goes back to the allocator with the call, and
    a stream that is not used again does not keep one for good."""
    stub.wait = 0.0
    live = set()

    class Counted(FakeTensor):
        def __init__(self, *a, **k):
            super().__init__(*a, **k)
            self.token = object()
            live.add((id(self.token), self.numel()))

        def __del__(self):
            live.discard((id(self.token), self.numel()))

    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: Counted((n,), dtype))
    grad_call(1000000)
    assert sum(size for _, size in live) <= 4 << 20
    handle = [0]
    monkeypatch.setattr(drs, "_raw_stream", lambda stream, gpu: handle[0])
    for handle[0] in range(1, 200):
        grad_call(500)
    assert sum(size for _, size in live) <= 64 << 20
