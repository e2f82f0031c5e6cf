"""drs_verify_drafts at the largest number of drafts that the call takes: a
request's places are counted in 64 bits."""
import pytest
import torch

from gpu_util import drs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most", [2**31 - 1, 2**31 - 257])
def test_most_drafts(most):
    """One request of two drafts whose row of 2^31 output places (17 GB) is
    written to its end; then one outside the arrays, whose places are all -1."""
    lib = drs()
    target = torch.tensor([[0.5, 0.5, 0.0], [0.0, 1.0, 0.0], [0.0, 0.0, 1.0]], device="cuda")
    tokens = torch.tensor([1, 1], device="cuda")
    u = torch.tensor([0.25, 0.5], device="cuda")
    out = torch.full((1, most + 1), 7, dtype=torch.int64, device="cuda")
    for cu, first, accepted in (([0, 2], [1, 1, 2], 2), ([1, 5], [-1, -1, -1], -1)):
        out.fill_(7)
        _, acc = lib.verify_drafts(target, tokens, torch.tensor(cu, dtype=torch.int32, device="cuda"), u, u[:1].clone(), most,
                                   out_tokens=out)
        assert out[0, :3].tolist() == first and int(acc) == accepted
        for part in out[0, 3:].split(1 << 28):
            assert bool((part == -1).all())
