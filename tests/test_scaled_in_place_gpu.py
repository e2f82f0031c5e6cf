"""drs_scaled_logits into its input's own memory gives what it gives into another array."""
import pytest
import torch

from gpu_util import drs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 255, 257, 152 * 32 * 256 + 3, 5_000_001])
def test_in_place(n):
    x = 8 * torch.randn(n, generator=torch.Generator("cuda").manual_seed(n), device="cuda")
    want = torch.empty_like(x)
    drs().drs_scaled_logits(x, 0.37, want)
    drs().drs_scaled_logits(x, 0.37, x)
    assert torch.equal(x, want)
