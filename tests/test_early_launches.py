"""The rules of kernels that are launched before the kernel ahead of them in the stream has ended, read from
the sources: they load plainly (the read-only path is for memory that nothing writes while a kernel lives),
and every way out of them is behind a wait for what is ahead."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "prefill_only_cascade_gb300", "csrc")
EARLY = ["paged_rows.cu", "fp4_decode.cu", "paged_decode.cuh", "evict.cu", "paged.cu"]


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    if name == "paged.cu":   # rows into bf16 and e4m3 pages: launched when the kernel ahead has ended
        text = re.sub(r"template <bool FP8>\s+__global__[^{]*?paged_append_kernel\(.*?\n}\n", "", text, flags=re.S)
        assert "paged_append_kernel(" not in text.split("cudaError_t")[0]
    return text


@pytest.mark.parametrize("name", EARLY + ["join_cluster.inc"])
def test_loads_are_plain(name):
    assert not re.search(r"__ldg|ld\.global\.nc|__restrict__", code(name))


@pytest.mark.parametrize("name", EARLY)
def test_returns_are_behind_the_wait(name):
    """In a kernel the first return follows a wait; the weights' blocks have it in a function of theirs."""
    text = code(name)
    kernels = [m.group(0) for m in re.finditer(r"__global__.*?\n}\n", text, flags=re.S)]
    weights = [m.group(0) for m in re.finditer(r"void add_weights\(.*?\n}\n", text, flags=re.S)]
    assert kernels
    for body in kernels + weights:
        first = re.search(r"\breturn\b", body)
        before = body[:first.start()] if first else body
        assert "after_stream();" in before or (body in kernels and "add_weights(" in before), body[:80]
