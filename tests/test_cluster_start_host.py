"""Kernels of thread-block clusters reach into another CTA's shared memory only
once all CTAs of the cluster have started, which a cluster barrier alone tells
(no GPU needed: the order of the calls in the sources). A function that maps
addresses of other CTAs, or calls one that does, without waiting on a barrier
before it leaves that wait to its callers; a kernel has none."""
import os
import re

import pytest

from vocab_row_sampling_gb300 import _build

WAIT = re.compile(r"\bcluster_sync_all\s*\(|\bcluster_wait\s*\(|barrier\.cluster\.wait")


def without_comments(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", lambda m: re.sub(r"[^\n]", " ", m.group()), text, flags=re.S)


def functions(text):
    """(name, whether it is a kernel, body) of the device functions of a source."""
    text = without_comments(text)
    for m in re.finditer(r"__(global|device)__", text):
        bounds = re.compile(r"__launch_bounds__\s*\(").search(text, m.end())
        at = m.end()
        semicolon = re.compile(r"[;{]").search(text, at).start()
        if bounds and bounds.start() < semicolon:
            at = bounds.end()
            depth = 1
            while depth:
                depth += {"(": 1, ")": -1}.get(text[at], 0)
                at += 1
        call = re.compile(r"(operator\s*\S+|\w+)\s*\(").search(text, at)
        end = call.end()
        depth = 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[end], 0)
            end += 1
        brace = re.compile(r"[;{]").search(text, end)
        if text[brace.start()] == ";":
            continue  # a declaration
        at = brace.end()
        depth = 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield call.group(1), m.group(1) == "global", text[brace.end():at]


def early_reach(text):
    """Kernels of a source that reach into other CTAs before any wait."""
    found = list(functions(text))
    remote = set()
    while True:
        reach = re.compile("|".join([r"mapa\.shared"] + [rf"\b{n}\s*(?:<[^;()]*>)?\s*\(" for n in sorted(remote)]))
        early = []
        for name, kernel, body in found:
            first, wait = reach.search(body), WAIT.search(body)
            if first and not (wait and wait.start() < first.start()):
                early.append((name, kernel))
        more = {name for name, _ in early} - remote
        if not more:
            return sorted({name for name, kernel in early if kernel})
        remote |= more


def source(name):
    text = ""
    for header in ("drs_device.cuh", "token_common.cuh", "row_common.cuh", name):
        with open(os.path.join(_build.CSRC, header)) as f:
            text += f.read() + "\n"
    return text


def test_the_rule_itself():
    helper = "__device__ void put(int r) { asm(\"mapa.shared::cluster.u32\"); }\n"
    wrap = "template <int k> __device__ void send(int r) { put(r); }\n"
    head = "__global__ void __launch_bounds__(f(2), g<3>(4)) "
    assert early_reach(helper + head + "k(int r) { put(r); cluster_sync_all(); }") == ["k"]
    assert early_reach(helper + head + "k(int r) { cluster_sync_all(); put(r); }") == []
    assert early_reach(helper + wrap + head + "k(int r) { send<2>(r); cluster_wait(); }") == ["k"]
    assert early_reach(helper + wrap + head + "k(int r) { cluster_wait(); send<2>(r); }") == []
    assert early_reach(helper + wrap + head + "k(int r) { /* cluster_wait(); */ send<2>(r); }") == ["k"]


@pytest.mark.parametrize("name", [s for s in _build.SOURCES if s.endswith(".cu")])
def test_every_kernel_waits_first(name):
    assert early_reach(source(name)) == []


def test_the_cluster_kernels_are_seen():
    """The rule looks at the kernels that it is for."""
    for name, kernel in (("verify.cu", "verify_kernel"), ("slots.cu", "slots_kernel"),
                         ("embed_grad.cu", "sort_cluster_kernel"), ("row_cluster.cu", "split_cluster")):
        bodies = [body for n, k, body in functions(source(name)) if k and n == kernel]
        assert len(bodies) == 1 and WAIT.search(bodies[0]), (name, kernel)
