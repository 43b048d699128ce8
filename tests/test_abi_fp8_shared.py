"""The 8-bit cache's and the shared prefixes' entry points without a GPU: argument
errors through ctypes, the binding's own checks, and the index and scale arithmetic of
csrc/paged.h compiled for the host."""

import ctypes
import os
import random
import shutil
import subprocess

import numpy as np
import pytest
import torch

import pass_attention_gb300 as oss
from pass_attention_gb300 import build_lib
from test_abi_paged import A, BAD_CACHES, Cache, INVALID, MISALIGNED, UNSUPPORTED, cache

CSRC = os.path.join(os.path.dirname(build_lib.__file__), "csrc")


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return oss.load()


class Cache8(ctypes.Structure):
    """os_paged_cache_fp8, declared on its own: the binding's packed form has to agree with it."""

    _fields_ = [("pages", Cache), ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("ld_scale_page", ctypes.c_int64), ("ld_scale_head", ctypes.c_int64)]


def test_packed_struct_agrees():
    values = list(range(1, 20))
    assert oss._PAGED_CACHE_FP8.pack(*values) == bytes(Cache8(Cache(*values[:15]), *values[15:]))


def cache8(scales=None, **change):
    s = dict(k_scales=A, v_scales=A, ld_scale_page=32, ld_scale_head=16)
    return Cache8(cache(**change), *{**s, **(scales or {})}.values())


def append(lib, c, k=A, v=A, ld=(256, 128), tokens=5, cu=A):
    return lib.os_kv_cache_append_fp8(k, v, ld[0], ld[1], tokens, cu, c, None)


def read(lib, c, k=A, v=A, ld=(256, 128), tokens=5, cu=A):
    return lib.os_kv_cache_read_fp8(c, cu, tokens, k, v, ld[0], ld[1], None)


def decode(lib, c, q=A, ld=(512, 128), H=4, scale=0.1, o=A, lse=A, ws=A, nbytes=1 << 40):
    return lib.os_attention_decode_paged_fp8(q, ld[0], ld[1], H, c, scale, o, lse, ws, nbytes, None)


def shared(lib, c, q=A, ld=(512, 128), H=4, table=A, ldt=4, n=A, pages=4, cu=A, groups=2, scale=0.1, o=A, lse=A, ws=A,
           nbytes=1 << 40):
    return lib.os_attention_decode_shared(q, ld[0], ld[1], H, c, table, ldt, n, pages, cu, groups, scale, o, lse, ws, nbytes,
                                          None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, change, status):
    c = ctypes.byref(cache8(**change))
    assert append(lib, c) == status
    assert read(lib, c) == status
    assert decode(lib, c) == status
    assert shared(lib, ctypes.byref(cache(**change))) == status


@pytest.mark.parametrize("scales,status", [
    (dict(k_scales=None), INVALID), (dict(v_scales=None), INVALID), (dict(ld_scale_page=0), INVALID),
    (dict(ld_scale_head=0), INVALID), (dict(ld_scale_page=-16), INVALID), (dict(k_scales=A + 8), MISALIGNED),
    (dict(v_scales=A + 1), MISALIGNED), (dict(ld_scale_page=40), MISALIGNED), (dict(ld_scale_head=8), MISALIGNED)])
def test_every_call_refuses_bad_scales(lib, scales, status):
    c = ctypes.byref(cache8(scales))
    assert append(lib, c) == read(lib, c) == decode(lib, c) == status


def test_rows_of_bytes_stand_on_16(lib):
    # strides that 16-bit pools may have, and 8-bit ones may not
    for change in (dict(ld_slot=136), dict(ld_head=2056), dict(ld_page=4104)):
        c = ctypes.byref(cache8(**change))
        assert append(lib, c) == read(lib, c) == decode(lib, c) == MISALIGNED


def test_null_caches(lib):
    assert append(lib, None) == read(lib, None) == decode(lib, None) == shared(lib, None) == INVALID
    assert lib.os_attention_decode_paged_fp8_workspace_bytes(4, None) == 0
    assert lib.os_attention_decode_shared_workspace_bytes(4, None, 4, 1) == 0


def test_append_and_read_reject_bad_arguments(lib):
    c = ctypes.byref(cache8())
    for call in (append, read):
        assert call(lib, c, k=None) == call(lib, c, v=None) == call(lib, c, tokens=-1) == INVALID
        assert call(lib, c, cu=None) == INVALID                  # three sequences, one token each
        assert call(lib, c, ld=(-8, 128)) == INVALID
        assert call(lib, c, k=A + 8) == call(lib, c, ld=(260, 128)) == call(lib, c, cu=A + 1) == MISALIGNED
        assert call(lib, c, tokens=2 ** 31) == UNSUPPORTED
        assert call(lib, c, tokens=0, k=None, v=None) == 0       # nothing to do
    assert read(lib, c, ld=(0, 128)) == read(lib, c, ld=(256, 0)) == INVALID   # rows on top of one another
    assert read(lib, c, cu=None, tokens=3) == INVALID


def test_decodes_reject_bad_arguments(lib):
    for call, c in ((decode, cache8()), (shared, cache())):
        c = ctypes.byref(c)
        for bad in (dict(q=None), dict(o=None), dict(ws=None), dict(H=0), dict(H=5), dict(scale=0.0),
                    dict(scale=float("nan")), dict(ld=(-8, 128))):
            assert call(lib, c, **bad) == INVALID, bad
        for bad in (dict(q=A + 2), dict(o=A + 8), dict(ws=A + 4), dict(ld=(512, 132)), dict(lse=A + 2)):
            assert call(lib, c, **bad) == MISALIGNED, bad
        assert call(lib, c, H=65538) == UNSUPPORTED
    c = ctypes.byref(cache())
    for bad in (dict(table=None), dict(n=None), dict(ldt=-1), dict(pages=0), dict(groups=0), dict(cu=None), dict(ld=(0, 128)),
                dict(ld=(512, 0))):
        assert shared(lib, c, **bad) == INVALID, bad
    for bad in (dict(table=A + 2), dict(n=A + 1), dict(cu=A + 3)):
        assert shared(lib, c, **bad) == MISALIGNED, bad
    for bad in (dict(groups=65536), dict(pages=2 ** 27)):
        assert shared(lib, c, **bad) == UNSUPPORTED, bad


def test_workspaces_of_refused_shapes(lib):
    c, c8 = ctypes.byref(cache()), ctypes.byref(cache8())
    assert lib.os_attention_decode_paged_fp8_workspace_bytes(5, c8) == 0
    for bad in ((5, 4, 1), (4, 0, 1), (4, 4, 0), (4, 2 ** 27, 1), (4, 4, 65536)):
        assert lib.os_attention_decode_shared_workspace_bytes(bad[0], c, bad[1], bad[2]) == 0
    for change in (dict(head_dim=96), dict(batch=0), dict(heads=0), dict(max_pages=2 ** 27)):
        assert lib.os_attention_decode_paged_fp8_workspace_bytes(4, ctypes.byref(cache8(**change))) == 0
        assert lib.os_attention_decode_shared_workspace_bytes(4, ctypes.byref(cache(**change)), 4, 1) == 0


def test_the_binding_refuses_cpu_tensors_and_other_types():
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    pages = torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16)
    p8, s8 = pages.to(torch.float8_e4m3fn), torch.zeros(3, 2, 16, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    table, n, cu = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        oss.attention_decode_shared(q, pages, pages, table[:1], n[:1], table, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        oss.kv_cache_append_fp8(q[:, :2], q[:, :2], p8, p8, s8, s8, table, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        oss.attention_decode_paged_fp8(q, p8, p8, s8, s8, table, n)
    with pytest.raises(ValueError, match="CUDA tensor"):
        oss.kv_cache_read_fp8(p8, p8, s8, s8, table, n, cu, 2)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        oss.kv_cache_read_fp8(pages, pages, s8, s8, table, n, cu, 2)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        oss.attention_decode_paged_fp8(q.float(), p8, p8, s8, s8, table, n)


PROBE = r"""
#include <cstdio>
#include "paged.h"
using namespace oss;
int main() {
  char op;
  while (std::scanf(" %c", &op) == 1) {
    if (op == 'e') {
      unsigned u;
      std::scanf("%u", &u);
      std::printf("%u\n", fp8_scale_byte(u));
    } else if (op == 'v') {
      unsigned u;
      std::scanf("%u", &u);
      std::printf("%u\n", fp8_scale_bits(u));
    } else if (op == 'g') {
      int b, groups; static int32_t cu[4096];
      std::scanf("%d %d", &b, &groups);
      for (int i = 0; i <= groups; ++i) std::scanf("%d", &cu[i]);
      const PrefixTables p{nullptr, 0, nullptr, cu, groups, 1}, all{nullptr, 0, nullptr, nullptr, 1, 1};
      std::printf("%d %d\n", prefix_group(p, b), prefix_group(all, b));
    }
  }
}
"""


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    d = tmp_path_factory.mktemp("fp8")
    (d / "probe.cpp").write_text(PROBE)
    exe = str(d / "probe")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wno-unused-result", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-I", CSRC, str(d / "probe.cpp"), "-o", exe], check=True, capture_output=True, text=True)

    def ask(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        return r.stdout.split("\n")[:-1]
    return ask


def test_scales_by_the_definition(probe):
    # the smallest power of two with which the largest magnitude is at most 448
    r = random.Random(3)
    values = [0.0, 2.0 ** -149, 2.0 ** -133, 2.0 ** -126, 448.0, np.nextafter(np.float32(448), np.float32(449)), 447.0, 1.0, 1.75,
              1.7578125, 3.3895314e38, 65504.0, 2.0 ** -24]
    values += [448.0 * 2.0 ** n for n in range(-140, 119, 7)]
    values += [float(np.float32(r.uniform(1, 2) * 2.0 ** r.randint(-140, 127))) for _ in range(500)]
    bits = [int(np.float32(x).view(np.uint32)) for x in values]
    for x, got in zip(values, probe([f"e {b}" for b in bits])):
        e = int(got) - 127
        x = float(np.float32(x))
        assert x <= 448.0 * 2.0 ** e
        assert e == -127 or x > 448.0 * 2.0 ** (e - 1)
    assert probe([f"e {0x7f800000}", f"e {0x7fc00000}", f"e {0x7f800001}"]) == ["255"] * 3
    got = np.array([int(x) for x in probe([f"v {b}" for b in range(256)])], np.uint32).view(np.float32)
    assert np.array_equal(got[:255], np.exp2(np.arange(255) - 127.0)) and np.isnan(got[255])


def test_groups_of_sequences(probe):
    r = random.Random(4)
    lines, want = [], []
    for _ in range(200):
        groups = r.randint(1, 20)
        cu = [r.randint(0, 3)]
        for _ in range(groups):
            cu.append(cu[-1] + r.choice((0, 0, 1, 5)))
        b = r.randint(0, cu[-1] + 4)
        lines.append(f"g {b} {groups} " + " ".join(map(str, cu)))
        want.append(f"{next((g for g in range(groups) if cu[g] <= b < cu[g + 1]), -1)} 0")
    assert probe(lines) == want
