"""The paged-cache entry points without a GPU: argument errors through ctypes,
and the index arithmetic of csrc/paged.h compiled for the host."""

import ctypes
import os
import random
import shutil
import subprocess

import pytest
import torch

import pass_attention_gb300 as oss
from pass_attention_gb300 import build_lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "pass_attention_gb300", "csrc")

INVALID, MISALIGNED, UNSUPPORTED = 1, 2, 3
A = 4096  # a 16-byte-aligned stand-in address; never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return oss.load()


class Cache(ctypes.Structure):
    """os_paged_cache, declared on its own: the binding's packed form has to agree with it."""

    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("ld_page", ctypes.c_int64),
                ("ld_head", ctypes.c_int64), ("ld_slot", ctypes.c_int64), ("page_table", ctypes.c_void_p),
                ("ld_table", ctypes.c_int64), ("kv_len", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


def test_packed_struct_agrees():
    values = list(range(1, 16))
    assert oss._PAGED_CACHE.pack(*values) == bytes(Cache(*values))[:oss._PAGED_CACHE.size]


def cache(**change):
    fields = dict(k_pages=A, v_pages=A, ld_page=4096, ld_head=2048, ld_slot=128, page_table=A, ld_table=4, kv_len=A,
                  num_pages=10, heads=2, page_size=16, head_dim=128, dtype=1, batch=3, max_pages=4)
    return Cache(**{**fields, **change})


BAD_CACHES = [(dict(k_pages=None), INVALID), (dict(v_pages=None), INVALID), (dict(page_table=None), INVALID),
              (dict(kv_len=None), INVALID), (dict(num_pages=0), INVALID), (dict(heads=0), INVALID),
              (dict(page_size=0), INVALID), (dict(head_dim=0), INVALID), (dict(dtype=0), INVALID), (dict(dtype=3), INVALID),
              (dict(batch=0), INVALID), (dict(max_pages=0), INVALID), (dict(ld_page=-8), INVALID), (dict(ld_slot=-8), INVALID),
              (dict(ld_page=0), INVALID), (dict(ld_head=0), INVALID), (dict(ld_slot=0), INVALID),
              (dict(ld_table=-1), INVALID), (dict(k_pages=A + 8), MISALIGNED), (dict(v_pages=A + 2), MISALIGNED),
              (dict(ld_slot=132), MISALIGNED), (dict(ld_head=4), MISALIGNED), (dict(kv_len=A + 2), MISALIGNED),
              (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED),
              (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED),
              (dict(max_pages=2 ** 27), UNSUPPORTED)]


def append(lib, c, k=A, v=A, ld=(256, 128), tokens=5, cu=A):
    return lib.os_kv_cache_append(k, v, ld[0], ld[1], tokens, cu, c, None)


def decode(lib, c, q=A, ld=(512, 128), H=4, scale=0.1, o=A, lse=A, w=None, ldw=(128, 64), ws=A, nbytes=1 << 40):
    return lib.os_attention_decode_paged(q, ld[0], ld[1], H, c, scale, o, lse, w, ldw[0], ldw[1], ws, nbytes, None)


def evict(lib, c, w=A, ldw=(128, 64), table=A, ld=4, pages=4, budget=32, recent=4, kept=A, n=A, nw=A):
    return lib.os_kv_cache_evict(c, w, ldw[0], ldw[1], table, ld, pages, budget, recent, kept, n, nw, None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, change, status):
    c = ctypes.byref(cache(**change))
    assert append(lib, c) == status
    assert decode(lib, c) == status
    assert evict(lib, c) == status


def test_null_cache(lib):
    assert append(lib, None) == INVALID
    assert decode(lib, None) == INVALID
    assert evict(lib, None) == INVALID
    assert lib.os_attention_decode_paged_workspace_bytes(4, None, 0) == 0


def test_append_rejects_bad_arguments(lib):
    c = ctypes.byref(cache())
    assert append(lib, c, k=None) == INVALID
    assert append(lib, c, v=None) == INVALID
    assert append(lib, c, tokens=-1) == INVALID
    assert append(lib, c, tokens=5, cu=None) == INVALID      # three sequences, one token each
    assert append(lib, c, ld=(-8, 128)) == INVALID
    assert append(lib, c, k=A + 8) == MISALIGNED
    assert append(lib, c, ld=(260, 128)) == MISALIGNED
    assert append(lib, c, cu=A + 1) == MISALIGNED
    assert append(lib, c, tokens=2 ** 31) == UNSUPPORTED
    assert append(lib, c, tokens=0, k=None, v=None) == 0     # nothing to do


def test_decode_rejects_bad_arguments(lib):
    c = ctypes.byref(cache())
    for bad in (dict(q=None), dict(o=None), dict(ws=None), dict(H=0), dict(H=5), dict(scale=0.0), dict(scale=float("nan")),
                dict(ld=(-8, 128)), dict(w=A, ldw=(-1, 64)), dict(w=A, ldw=(0, 64)),
                dict(w=A, ldw=(128, 0))):
        assert decode(lib, c, **bad) == INVALID, bad
    for bad in (dict(q=A + 2), dict(o=A + 8), dict(ws=A + 4), dict(ld=(512, 132)), dict(lse=A + 2), dict(w=A + 1)):
        assert decode(lib, c, **bad) == MISALIGNED, bad
    assert decode(lib, c, H=65538) == UNSUPPORTED
    assert lib.os_attention_decode_paged_workspace_bytes(5, c, 0) == 0


def test_packed_rejects_bad_arguments(lib):
    def call(q=A, ldq=(512, 128), k=A, v=A, ldk=(256, 128), o=A, lse=A, cq=A, ck=A, batch=2, tq=20, tk=30, Hq=4, Hkv=2,
             D=128, dtype=1, scale=0.1, ws=A, nbytes=1 << 40):
        return lib.os_attention_fwd_packed(q, ldq[0], ldq[1], k, v, ldk[0], ldk[1], o, lse, cq, ck, batch, tq, tk, Hq, Hkv, D,
                                           dtype, scale, 1, ws, nbytes, None)
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(cq=None), dict(ck=None), dict(batch=0), dict(tq=-1),
                dict(tk=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(D=0), dict(dtype=0), dict(dtype=3), dict(scale=0.0),
                dict(scale=float("inf")), dict(ws=None), dict(ldq=(-8, 128)), dict(ldk=(256, -8)), dict(ldq=(0, 128)),
                dict(ldq=(512, 0)), dict(ldk=(0, 128)), dict(ldk=(256, 0))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(q=A + 8), dict(k=A + 2), dict(o=A + 4), dict(ws=A + 8), dict(ldq=(516, 128)), dict(ldk=(256, 4)),
                dict(cq=A + 2), dict(lse=A + 1)):
        assert call(**bad) == MISALIGNED, bad
    for bad in (dict(D=32), dict(D=256), dict(batch=65536), dict(tq=2 ** 31), dict(tk=2 ** 31)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(tq=0, q=None, o=None) == 0
    assert lib.os_attention_fwd_packed_workspace_bytes(20, 2, 96) == 0
    assert lib.os_attention_fwd_packed_workspace_bytes(-1, 2, 128) == 0
    assert lib.os_attention_fwd_packed_workspace_bytes(20, 0, 128) == 0


def test_evict_rejects_bad_arguments(lib):
    c = ctypes.byref(cache())
    for bad in (dict(w=None), dict(table=None), dict(kept=None), dict(n=None), dict(nw=None), dict(pages=0), dict(budget=0),
                dict(budget=65), dict(recent=-1), dict(recent=33), dict(ldw=(-1, 4)), dict(ld=-1)):
        assert evict(lib, c, **bad) == INVALID, bad
    for bad in (dict(w=A + 1), dict(table=A + 2), dict(kept=A + 3), dict(n=A + 1), dict(nw=A + 2)):
        assert evict(lib, c, **bad) == MISALIGNED, bad


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls that are not refused would run on stand-in addresses")
def test_evict_refuses_what_it_would_overwrite(lib):
    # batch 2, 2 heads, 64 positions: weights and new_weights of 1024 bytes each
    MB = 1 << 20
    c = ctypes.byref(cache(page_table=MB, kv_len=2 * MB, batch=2, heads=2, page_size=16, max_pages=4))
    free = dict(w=3 * MB, ldw=(128, 64), table=4 * MB, kept=5 * MB, n=6 * MB, nw=7 * MB)
    no_device = evict(lib, c, **free)
    assert no_device not in (0, INVALID, MISALIGNED, UNSUPPORTED)
    for n in (-8, 8):
        assert evict(lib, c, **{**free, "n": 2 * MB + n}) == no_device
    for n in (-4, 0, 4):
        assert evict(lib, c, **{**free, "n": 2 * MB + n}) == INVALID
    for n in (-1024, 1024):
        assert evict(lib, c, **{**free, "nw": 3 * MB + n}) == no_device
    for n in (-1020, 0, 1020):
        assert evict(lib, c, **{**free, "nw": 3 * MB + n}) == INVALID
    assert evict(lib, c, **{**free, "table": MB}) == INVALID


PROBE = r"""
#include <cstdio>
#include "paged.h"
using namespace oss;
// commands on stdin: what paged.h answers, one line each
int main() {
  char op;
  while (std::scanf(" %c", &op) == 1) {
    if (op == 'l') {
      int n, pages, shift;
      std::scanf("%d %d %d", &n, &pages, &shift);
      std::printf("%d\n", paged_length(n, pages, shift));
    } else if (op == 'p') {
      int page, pages;
      std::scanf("%d %d", &page, &pages);
      std::printf("%d\n", page_ok(page, pages) ? 1 : 0);
    } else if (op == 'o') {
      int page, head, slot; long long a, b, c;
      std::scanf("%d %d %d %lld %lld %lld", &page, &head, &slot, &a, &b, &c);
      std::printf("%lld\n", static_cast<long long>(pool_offset(page, head, slot, a, b, c)));
    } else if (op == 's') {
      long long t; int batch; static int32_t cu[4096];
      std::scanf("%lld %d", &t, &batch);
      for (int i = 0; i <= batch; ++i) std::scanf("%d", &cu[i]);
      std::printf("%d\n", sequence_of(t, cu, batch));
    } else if (op == 'r') {
      int b, e, n;
      std::scanf("%d %d %d", &b, &e, &n);
      const RowRange r = row_range(b, e, n);
      std::printf("%d %d %d\n", r.start, r.len, r.clamped ? 1 : 0);
    } else if (op == 'w') {
      unsigned u;
      std::scanf("%u", &u);
      std::printf("%u\n", weight_key_bits(u));
    }
  }
}
"""


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    d = tmp_path_factory.mktemp("paged")
    (d / "probe.cpp").write_text(PROBE)
    exe = str(d / "probe")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wno-unused-result", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-I", CSRC, str(d / "probe.cpp"), "-o", exe], check=True, capture_output=True, text=True)

    def ask(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        return r.stdout.split("\n")[:-1]
    return ask


def test_lengths_pages_and_offsets_stay_inside(probe):
    big = 2 ** 31 - 1
    got = probe([f"l {n} {p} {s}" for n in (-big - 1, -1, 0, 5, 64, 65, big) for p, s in ((4, 4), (1, 10), (2 ** 20, 10))])
    want = [str(min(max(n, 0), p << s)) for n in (-big - 1, -1, 0, 5, 64, 65, big) for p, s in ((4, 4), (1, 10), (2 ** 20, 10))]
    assert got == want
    ids = (-big - 1, -1, 0, 9, 10, big)
    assert probe([f"p {i} 10" for i in ids]) == [str(int(0 <= i < 10)) for i in ids]
    assert probe([f"o {2 ** 20} 7 1023 {2 ** 20} {2 ** 17} 128"]) == [str(2 ** 40 + 7 * 2 ** 17 + 1023 * 128)]


def test_sequence_search_and_ranges(probe):
    r = random.Random(1)
    lines, want = [], []
    for _ in range(200):
        batch = r.randint(1, 40)
        cu = [r.randint(0, 3)]
        for _ in range(batch):
            cu.append(cu[-1] + r.choice((0, 0, 1, 5)))
        t = r.randint(0, cu[-1] + 4)
        lines.append(f"s {t} {batch} " + " ".join(map(str, cu)))
        want.append(next((b for b in range(batch) if cu[b] <= t < cu[b + 1]), -1))
    assert [int(x) for x in probe(lines)] == want
    # offsets in any order: never a sequence whose range the row is outside of
    lines, cases = [], []
    for _ in range(200):
        cu = [r.randint(-9, 50) for _ in range(r.randint(2, 9))]
        t = r.randint(0, 50)
        cases.append((t, cu))
        lines.append(f"s {t} {len(cu) - 1} " + " ".join(map(str, cu)))
    for (t, cu), x in zip(cases, probe(lines)):
        b = int(x)
        assert b == -1 or cu[b] <= t < cu[b + 1]
    edges = (-2 ** 31, -1, 0, 7, 99, 100, 101, 2 ** 31 - 1)
    pairs = [(b, e) for b in edges for e in edges]
    for (b, e), line in zip(pairs, probe([f"r {b} {e} 100" for b, e in pairs])):
        start, n, clamped = map(int, line.split())
        assert 0 <= start <= 100 and 0 <= n <= 100 - start
        assert clamped == int(not 0 <= b <= e <= 100)
        if not clamped:
            assert (start, n) == (b, e - b)


def test_weight_order(probe):
    import numpy as np
    w = np.array([np.nan, np.inf, 3.4e38, 1.5, 1e-45, 0.0, -1e-45, -1.5, -np.inf], np.float32)
    key = [int(x) for x in probe([f"w {int(u)}" for u in w.view(np.uint32)])]
    assert key == sorted(key, reverse=True) and len(set(key)) == len(key)
    zero, minus, nan = probe([f"w {0}", f"w {0x80000000}", f"w {0xffc00000}"])
    assert zero == minus and int(nan) == key[0]


PLAN = r"""
#include <cassert>
#include <cstdio>
#include <cstdlib>
#include <utility>
#include <vector>
#include "packed_plan.h"
using namespace oss;
// Random sequences: the closed forms against sums tile by tile, and the shares
// against a walk over all items.
int main() {
  srand(1);
  for (int it = 0; it < 3000; ++it) {
    const int ps = rand() % 8, B = 1 + rand() % 12, packs = 1 + rand() % 6, ctas = rand() % 2 ? 152 : 1 + rand() % 40;
    const int rounds = 1 + rand() % 4;
    const bool causal = rand() % 4 != 0;
    std::vector<PackedSeq> seqs;
    int64_t total = 0, items = 0;
    for (int b = 0; b < B; ++b) {
      const int ql = rand() % 4 == 0 ? 0 : rand() % (1 << (rand() % 11 + 1));
      const int kl = rand() % 3 == 0 ? rand() % 2000 : ql + (rand() % 2 ? rand() % 3000 : 0);
      const PackedSeq s = packed_seq(row_range(0, ql, 1 << 30), row_range(0, kl, 1 << 30), ps);
      int64_t sum = 0;
      for (int t = 0; t < s.tiles; ++t) {
        int last = ((t + 1) << ps) - 1;
        if (last >= ql) last = ql - 1;
        int vis = causal ? last + 1 + kl - ql : kl;
        if (vis > kl) vis = kl;
        const int want = vis > 0 ? (vis + 127) / 128 : 1;
        assert(kv_tiles(s, t, ps, causal) == want);
        assert(length_before(s, t, ps, causal) == sum);
        assert(tile_at(s, sum, ps, causal) == t && tile_at(s, sum + want + kTileWeight - 1, ps, causal) == t);
        sum += want + kTileWeight;
      }
      assert(length_before(s, s.tiles, ps, causal) == sum);
      seqs.push_back(s);
      total += sum * packs;
      items += static_cast<int64_t>(s.tiles) * packs;
    }
    if (!items) continue;
    const int n = share_count(total, items, ctas, rounds);
    assert(n >= 1 && n <= ctas * rounds && n <= total && (n <= ctas || n % ctas == 0));
    const ShareCut cut = share_cut(total, n);
    struct Item { int64_t w; int steps; };
    std::vector<Item> all;
    int64_t w = 0;
    for (auto& s : seqs)
      for (int p = 0; p < packs; ++p)
        for (int t = 0; t < s.tiles; ++t) {
          all.push_back({w, kv_tiles(s, t, ps, causal)});
          w += all.back().steps + kTileWeight;
        }
    // every share's beginning as (item, step); the last one is the end
    std::vector<std::pair<int, int>> at;
    size_t i = 0;
    for (int c = 0; c < n; ++c) {
      const int64_t x = share_begin(cut, c);
      while (i + 1 < all.size() && all[i + 1].w <= x) ++i;
      const int st = cut_step(x - all[i].w, all[i].steps);
      at.push_back(st == all[i].steps ? std::make_pair(static_cast<int>(i) + 1, 0) : std::make_pair(static_cast<int>(i), st));
    }
    at.push_back({static_cast<int>(all.size()), 0});
    assert(share_begin(cut, n) == total);
    assert(at[0].first == 0 && at[0].second == 0);
    for (int c = 0; c < n; ++c) {
      assert(at[c] <= at[c + 1]);
      const auto e = at[c + 1];
      if (e.second == 0) continue;
      assert(e.second >= kMinSteps && all[e.first].steps - e.second >= kMinSteps);
      if (at[c].first == e.first && at[c].second > 0) continue;
      // the item begins in share c and is cut at its end: its parts
      const int64_t last = last_boundary(cut, all[e.first].w + kTileWeight + all[e.first].steps - kMinSteps);
      int parts = 1;
      for (int d = c + 1; d < n; ++d) parts += at[d].first == e.first && at[d].second > 0;
      assert(parts == last - c + 1);
      for (int d = c + 1; d <= last; ++d) assert(at[d].first == e.first && at[d].second > 0 && at[d] < at[d + 1]);
    }
  }
  // cuts of long rows, and small quotients
  for (int it = 0; it < 20000; ++it) {
    const int64_t total = (int64_t(rand()) << (rand() % 20)) + rand() % 1000 + 1300;
    const int n = 1 + rand() % 1216;
    const ShareCut cut = share_cut(total, n);
    assert(share_begin(cut, 0) == 0 && share_begin(cut, n) == total);
    const int c = rand() % n;
    const int64_t x = share_begin(cut, c);
    assert(x < share_begin(cut, c + 1));
    assert(last_boundary(cut, x) == static_cast<uint32_t>(c));
    assert(last_boundary(cut, share_begin(cut, c + 1) - 1) == static_cast<uint32_t>(c));
    const int64_t y = 1 + (int64_t(rand()) << (rand() % 12)), q = rand() % 65536;
    assert(small_quotient(q * y + rand() % y, y) == q);
  }
  std::puts("ok");
}
"""


def test_packed_plan(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    (tmp_path / "plan.cpp").write_text(PLAN)
    exe = str(tmp_path / "plan")
    subprocess.run(["g++", "-std=c++17", "-O2", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC,
                    str(tmp_path / "plan.cpp"), "-o", exe], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr
