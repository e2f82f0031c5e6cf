"""Gradients that several host threads ask for at the same time on one stream:
each gets the bits of a call by itself."""
import threading

import pytest
import torch

from gpu_util import drs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("threads,n,width,vocab", [(2, 3000, 64, 5000), (4, 500, 264, 700), (3, 9000, 16, 40000)])
def test_threads_on_one_stream(threads, n, width, vocab):
    """Equal sizes, ids and gradients of each thread's own."""
    lib = drs()
    stream = torch.cuda.Stream()
    cases = []
    for k in range(threads):
        g = torch.Generator(device="cuda").manual_seed(k)
        ids = torch.randint(0, vocab, (n,), generator=g, device="cuda")
        ids[:: k + 2] = 7 * k
        up = torch.randn(n, width, generator=g, device="cuda")
        cases.append((up, ids, lib.embed_tokens_grad(up, ids, 2.0, torch.empty(vocab, width, device="cuda"))))
    torch.cuda.synchronize()
    outs = [[torch.empty(vocab, width, device="cuda") for _ in range(8)] for _ in cases]
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(threads)

    def work(k):
        try:
            up, ids, _ = cases[k]
            start.wait(timeout=30)
            for repeat in range(40):
                lib.embed_tokens_grad(up, ids, 2.0, outs[k][repeat % 8], stream=stream)
        except BaseException as e:
            failed.append(e)

    hosts = [threading.Thread(target=work, args=(k,)) for k in range(threads)]
    for t in hosts:
        t.start()
    for t in hosts:
        t.join()
    stream.synchronize()
    assert not failed
    for (_, _, want), got in zip(cases, outs):
        for o in got:
            assert torch.equal(o, want)
