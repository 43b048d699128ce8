"""Kernels that start while the one before them still writes: their sources promise the compiler
nothing about memory that it could use to load before the wait."""

import glob
import os
import re

import pytest

from pass_attention_gb300 import build_lib

CSRC = os.path.join(os.path.dirname(build_lib.__file__), "csrc")


def source(name):
    """The file without comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def overlapped():
    """The sources of kernels that are launched behind one that may still run, and the
    headers that these share."""
    names = [os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*"))]
    return sorted(n for n in names if re.search(r"wait_for_previous_kernel|launch_after|decode_paged\.cuh|Fp8Pools", source(n)))


def test_the_launches_are_found():
    assert {"attn_packed.cu", "decode_paged.cu", "decode_fp8.cu", "decode_shared.cu", "kv_cache.cu", "kv_cache_fp8.cu",
            "decode_paged_kernel.cuh", "launch.cuh"} <= set(overlapped())


@pytest.mark.parametrize("name", overlapped())
def test_no_promise_that_memory_does_not_change(name):
    assert not re.findall(r"__restrict__|__restrict\b|__ldg\b|ld\.global\.nc|\.global\.nc", source(name))
