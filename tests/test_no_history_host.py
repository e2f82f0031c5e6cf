"""The lookup and its gradient leave no autograd history, so tensors that require
a gradient are refused while autograd records (no GPU needed: stand-in tensors
and a stub library); under torch.no_grad() they are taken."""
import pytest
import torch

import vocab_row_sampling_gb300 as drs
from fake_tensors import FakeTensor
from test_current_device_host import stub  # noqa: F401


def lookup(table=False, out=False):
    return drs.drs_embed_tokens(FakeTensor((16, 8), requires_grad=table), FakeTensor((4,), torch.int64), 1.0,
                                FakeTensor((4, 8), requires_grad=out))


def lookup_wrapper(table=False):
    return drs.embed_tokens(FakeTensor((16, 8), requires_grad=table), FakeTensor((4,), torch.int64))


def grad(up=False, table=False):
    return drs.drs_embed_tokens_grad(FakeTensor((4, 8), requires_grad=up), FakeTensor((4,), torch.int64), 1.0, True,
                                     FakeTensor((16, 8), requires_grad=table), FakeTensor((4096,), torch.uint8))


def grad_wrapper(up=False, table=False):
    return drs.embed_tokens_grad(FakeTensor((4, 8), requires_grad=up), FakeTensor((4,), torch.int64), 1.0,
                                 FakeTensor((16, 8), requires_grad=table))


@pytest.mark.parametrize("call,arguments", [
    (lookup, {"table": True}), (lookup, {"out": True}), (lookup_wrapper, {"table": True}), (grad, {"up": True}),
    (grad, {"table": True}), (grad_wrapper, {"up": True}), (grad_wrapper, {"table": True})])
def test_tensors_that_require_a_gradient(stub, call, arguments):  # noqa: F811
    call()
    assert len(stub.calls) == 1
    with pytest.raises(ValueError, match="requires a gradient"):
        call(**arguments)
    assert len(stub.calls) == 1
    with torch.no_grad():
        call(**arguments)
    assert len(stub.calls) == 2
