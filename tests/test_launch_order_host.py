"""Kernels that are launched as programmatic dependents may begin before the kernel ahead of them on the
stream has ended: each of them has to wait before it touches global memory, which its source shows. No GPU."""

from __future__ import annotations

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_116_b200", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(name, kernel):
    """The text of a __global__ function, without comments."""
    text = source(name)
    start = text.index("{", re.search(r"\b" + kernel + r"\(", text).end())
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise AssertionError(kernel)


GLOBAL = r"__ld\w+\(|p\.(cu|seqlens|block_table|split|o_part|lse_part|o|lse|rows|cache|k_new|v_new)\b"
READERS = r"report_bad_batch|cache_place|chunk_plan|dec_prologue"  # functions that read global memory


@pytest.mark.parametrize("name,kernel", [("fa_cache.cuh", "fa_cache_write_kernel"), ("fa_cache.cuh", "fa_cache_read_kernel"),
                                         ("fa_chunk.cuh", "fa_chunk_kernel"), ("fa_chunk.cuh", "fa_chunk_merge_kernel"),
                                         ("fa_chunk_few.cuh", "fa_chunk_few_kernel"), ("fa_decode.cuh", "fa_decode_kernel")])
def test_the_wait_comes_first(name, kernel):
    text = body(name, kernel)
    first = re.search("griddep_wait\\(\\)", text)
    access = re.search(GLOBAL + "|" + READERS, text)
    assert first and access and first.start() < access.start()


def test_every_dependent_launch_is_one_of_these():
    api = source("fa_api.cu")
    assert len(re.findall("cudaLaunchAttributeProgrammaticStreamSerialization", api)) == 3
    launched = set(re.findall(r"launch_dependent\(fa::(\w+)", api)) | set(re.findall(r"cudaLaunchKernelEx\(&cfg, fa::(\w+)", api))
    # (the forward follows its own counter reset, a launch in full)
    assert launched == {"fa_chunk_kernel", "fa_chunk_merge_kernel", "fa_chunk_few_kernel", "fa_decode_kernel", "fa_fwd_kernel"}


def test_the_decode_kernel_waits_in_every_thread_and_for_its_prep_kernel():
    text = body("fa_decode.cuh", "fa_decode_kernel")
    prologue = text.index("dec_prologue<D>(")
    assert re.search(r";\s*if \(p\.pieces == 1\) griddep_wait\(\);", text[:prologue])
    end = text.rindex("__syncthreads()")
    assert re.search(r"if \(tid == 0\) griddep_wait\(\);\s*$", text[:end])  # outside every role's branch


@pytest.mark.parametrize("name", ["fa_cache.cuh", "fa_chunk.cuh", "fa_chunk_few.cuh"])
def test_nothing_is_read_as_constant(name):
    """These kernels live while the one before them still writes: no load may be one of memory that stays as it
    is for the kernel's life (which may also be moved ahead of the wait)."""
    text = source(name)
    assert not re.findall(r"__ld(?:g|cs|cg|ca|lu|cv)\(|__restrict__", text)
    seg_of = source("sm100_ptx.cuh")
    assert "__ldg" not in seg_of[seg_of.index("int seg_of("):seg_of.index("void seg_bounds(")]
