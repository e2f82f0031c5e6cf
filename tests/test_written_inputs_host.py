"""Kernels whose calls allow an output in an input's place read their inputs by
the coherent path: the read-only one (ld.global.nc, __ldg) is defined only for
memory that nothing writes while the kernel runs (no GPU needed: the loads in
the sources)."""
import re

import pytest

from test_cluster_start_host import without_comments
from vocab_row_sampling_gb300 import _build

# out may be x or residual; grad may be logits; out may be logits; out_held may be held
IN_PLACE = ("dropout.cu", "logprobs_grad.cu", "scale.cu", "slots.cu")
READ_ONLY = re.compile(r"\.nc\b|__ldg\s*\(|(?:\.\s*(?:template\s+)?load|\bload16_stream)\s*(?:<\s*false\s*>)?\s*\(|__restrict__")


def read_only_loads(text):
    return READ_ONLY.findall(without_comments(text))


def test_the_rule_itself():
    for bad in ("raw.load(p)", "raw[u].load (p)", "w = load16_stream(p)", "__ldg(p)", 'asm("ld.global.nc.v4.u32")',
                "x.template load<false>(p)", "const float* __restrict__ x"):
        assert read_only_loads(bad), bad
    for good in ("raw.template load<true>(p)", "w = load16_stream<true>(p)", "x[i]", "// raw.load(p)", "reload(p)"):
        assert not read_only_loads(good), good


@pytest.mark.parametrize("name", IN_PLACE)
def test_inputs_that_may_be_outputs(name):
    assert name in _build.SOURCES
    with open(f"{_build.CSRC}/{name}") as f:
        assert read_only_loads(f.read()) == []


def test_the_shared_loads_hand_it_on():
    """The loads of the shared header are all made by load16_stream with the caller's choice, and plain ones."""
    with open(f"{_build.CSRC}/token_common.cuh") as f:
        text = without_comments(f.read())
    rest = re.sub(r"template <bool kWritten = false> __device__ __forceinline__ uint4 load16_stream\(.*?\n}\n", "", text,
                  count=1, flags=re.S)
    assert rest != text
    assert not re.search(r"\.nc\b|__ldg\s*\(|__restrict__", rest)
    calls = re.findall(r"(?:load16_stream|\.(?:template )?load)\b[^(\n]*\(", rest)
    assert len(calls) >= 4 and all("<kWritten>" in call for call in calls), calls
