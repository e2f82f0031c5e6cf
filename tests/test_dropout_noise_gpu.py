"""Dropout's mask against the sampler's noise of the same seed, row and columns."""
import numpy as np
import pytest
import torch

from gpu_util import drs
from test_dropout_gpu import philox

pytestmark = pytest.mark.gpu
GROUPS = 512  # counters of a row: eight columns each for dropout, four words for the noise


def mask_of(words):
    """Which of the row's 8 GROUPS columns dropout with q = 1/2 would keep if these were its words: two halves to a
    word, the lower first."""
    halves = torch.stack([words & 0xFFFF, words >> 16 & 0xFFFF], 1).reshape(-1)
    return halves >= 32768


def words_of(tag, row, seed):
    """The words of a row's counters with this second word."""
    w = philox((np.arange(GROUPS, dtype=np.uint64), np.uint64(tag), np.uint64(row % 2**32), np.uint64(row // 2**32)), seed)
    return torch.as_tensor(np.stack(w, 1).reshape(-1).astype(np.int64)).cuda()


def agreement(a, b):
    return float((a == b).double().mean())


@pytest.mark.parametrize("seed", [1, 0x9E3779B97F4A7C15, 2**64 - 1])
@pytest.mark.parametrize("row0", [0, 2**32 + 7])
def test_the_calls_draw_other_numbers(seed, row0):
    """The noise's words have the counters (column / 4, 0, row), dropout's (column / 8, its tag, row): without the tag the
    mask would be that of the noise's words, as they stand. With it the two agree by chance: in half of n = 4096
    places, off by less than 6 standard deviations n^-1/2 / 2 (fixed by the seeds)."""
    lib = drs()
    words = lib.philox_gumbel(seed, row0, 1, 4 * GROUPS)[0][0].long()
    x = torch.ones(1, 8 * GROUPS, device="cuda")
    kept = lib.dropout(x, 0.5, seed, row0=row0)[0] != 0
    assert torch.equal(words & 0xFFFFFFFF, words_of(0, row0, seed))
    assert torch.equal(kept, mask_of(words_of(0x64726F70, row0, seed)))
    without_tag = mask_of(words)
    spread = 6 * 0.5 / kept.numel() ** 0.5
    assert abs(float(without_tag.double().mean()) - 0.5) < spread and abs(float(kept.double().mean()) - 0.5) < spread
    assert abs(agreement(kept, without_tag) - 0.5) < spread
    # another row's words, and the words of the columns themselves, are as far away
    other = lib.philox_gumbel(seed, row0 + 1, 1, 4 * GROUPS)[0][0].long()
    assert abs(agreement(kept, mask_of(other)) - 0.5) < spread
    assert abs(agreement(kept[: 4 * GROUPS], words >> 31 & 1 == 1) - 0.5) < 1.5 * spread
