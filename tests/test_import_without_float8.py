"""The package on a PyTorch that lacks the 8-bit types: everything but the 8-bit cache is there."""

import os
import subprocess
import sys

import pytest

from pass_attention_gb300 import build_lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import torch
for name in sys.argv[1:]:
    delattr(torch, name)
import pass_attention_gb300 as oss
assert oss.abi_version() == 1
q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
pages = torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16)
bytes_, scales = torch.zeros(3, 2, 16, 128, dtype=torch.uint8), torch.zeros(3, 2, 16, dtype=torch.uint8)
table, n = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
for call, error, text in (
        (lambda: oss.attention_decode_paged(q, pages, pages, table, n), ValueError, "CUDA tensor"),
        (lambda: oss.attention_decode_shared(q, pages, pages, table[:1], n[:1], table, n), ValueError, "CUDA tensor"),
        (lambda: oss.kv_cache_read_fp8(bytes_, bytes_, scales, scales, table, n, n, 2), RuntimeError, "float8_e8m0fnu")):
    try:
        call()
    except error as e:
        assert text in str(e), e
    else:
        raise AssertionError("taken")
print("ok")
"""


@pytest.mark.parametrize("missing", [["float8_e8m0fnu"], ["float8_e4m3fn", "float8_e8m0fnu"]])
def test_import_without_the_8_bit_types(missing):
    build_lib.build()
    r = subprocess.run([sys.executable, "-c", CHILD, *missing], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), r.stdout + r.stderr
