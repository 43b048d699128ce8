"""Importing the package, and its argument checks, on a PyTorch without CUDA."""

import os
import subprocess
import sys

from pass_attention_gb300 import build_lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import torch
# what a build of PyTorch without CUDA does not have
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import pass_attention_gb300 as oss
lib = oss.load()
assert oss.abi_version() == 1
assert lib.os_kv_cache_append(None, None, 0, 0, 0, None, None, None) == 1
q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
pages = torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16)
table, n = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
for call in (lambda: oss.attention_decode_paged(q, pages, pages, table, n),
             lambda: oss.kv_cache_append(q[:, :2], q[:, :2], pages, pages, table, n),
             lambda: oss.attention_fwd_packed(q, q, q, table[:, 0])):
    try:
        call()
    except ValueError as e:
        assert "CUDA tensor" in str(e), e
    else:
        raise AssertionError("a CPU tensor was taken")
print("ok")
"""


def test_import_without_cuda_in_pytorch():
    build_lib.build()
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), r.stdout + r.stderr
