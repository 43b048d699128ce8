"""os_kv_cache_evict refuses outputs that overlap what it reads, or each other
(through ctypes, without a GPU)."""

import ctypes

import pytest
import torch

from test_abi_paged import INVALID, MISALIGNED, UNSUPPORTED, cache, evict, lib  # noqa: F401  (lib: the fixture)

MB = 1 << 20
# batch 2, 2 heads, 64 positions, budget 32, rows of 4 pages with a stride of 6
CACHE = dict(page_table=MB, ld_table=6, kv_len=2 * MB, batch=2, heads=2, page_size=16, max_pages=4)
CALL = dict(w=3 * MB, ldw=(128, 64), table=4 * MB, ld=6, kept=5 * MB, n=6 * MB, nw=7 * MB)
BYTES = dict(w=2 * 2 * 64 * 4, table=(6 + 4) * 4, page_table=(6 + 4) * 4, kv_len=2 * 4, kept=2 * 2 * 32 * 4, n=2 * 4,
             nw=2 * 2 * 64 * 4)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls that are not refused would run on stand-in addresses")
@pytest.mark.parametrize("out,other", [(x, y) for x in ("kept", "n", "nw") for y in BYTES if x != y])
def test_overlaps(lib, out, other):  # noqa: F811
    c = ctypes.byref(cache(**CACHE))
    no_device = evict(lib, c, **CALL)
    assert no_device not in (0, INVALID, MISALIGNED, UNSUPPORTED)
    at = {**CALL, **CACHE}[other]
    for apart in (-BYTES[out], BYTES[other]):
        assert evict(lib, c, **{**CALL, out: at + apart}) == no_device
    for inside in (4 - BYTES[out], 0, BYTES[other] - 4):
        assert evict(lib, c, **{**CALL, out: at + inside}) == INVALID
