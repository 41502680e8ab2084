"""Kernels that take tensor memory, in the order in which they take it (CPU: the sources are
read; a kernel that got this wrong would wait for ever).

A kernel launched early, while the one before it on the stream still runs, must not hold
tensor memory while it waits for that one: a CTA of the latter on the same SM may not have
taken its own yet, and would wait for the former's in turn."""

import os
import re

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "paged_kv_cache_51_gb300", "csrc")


def _text(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


KERNELS = [n for n in sorted(os.listdir(CSRC)) if n.endswith(".cu") and "tcgen05.alloc" in _text(n)]


def test_the_kernels_are_found():
    assert {"latent_attn.cu", "latent_pair.cu", "expanded_tc.cu", "prefill_tc.cu"} <= set(KERNELS)


@pytest.mark.parametrize("name", KERNELS)
def test_tensor_memory_is_taken_behind_the_wait(name):
    text = _text(name)
    assert text.count("tcgen05.alloc") == 1 == text.count("pdl_wait_prerequisites()")
    assert text.index("pdl_wait_prerequisites()") < text.index("tcgen05.alloc")


@pytest.mark.parametrize("name", ["latent_attn.cu", "latent_pair.cu", "expanded_tc.cu"])
def test_the_next_kernel_is_let_in_behind_the_barrier_that_follows(name):
    """Not before every CTA has its tensor memory: the next kernel may be another library's,
    which takes its own before it waits."""
    text = _text(name)
    assert text.count("pdl_launch_dependents()") == 1
    between = text[text.index("tcgen05.alloc"):text.index("pdl_launch_dependents()")]
    # latent_plan ends with a barrier of its own
    assert "__syncthreads()" in between or "latent_plan<" in between
