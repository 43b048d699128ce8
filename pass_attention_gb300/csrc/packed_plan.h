// How the packed attention forward divides its work: arithmetic shared by
// the kernel and by a host-compiled test.
//
// A work item is one tile of 128 query rows: `positions` consecutive queries of a
// sequence times a pack of 128 / positions query heads that share a key head.
// It visits kv_tiles tiles of 128 keys. The items of a launch stand in a row,
// (sequence, pack, tile)-major, each kTileWeight + kv_tiles long (a hand-over
// costs about as much as two KV steps, by a fit over the CTAs' times of a ragged batch: 8
// sequences of 77 to 2500 tokens take 160 us with 2, 187 with 1, 164 with 3), and the
// row is cut into equal shares, one or a few per CTA. A share's boundary that
// falls inside an item cuts it along the keys, unless one side would get fewer
// than kMinSteps KV steps: then the boundary moves to the item's edge.
#pragma once

#include <cstdint>

#include "paged.h"

namespace oss {

constexpr int kTileWeight = 2;
constexpr int kMinSteps = 3;
constexpr int kLeastShareShift = 3;
// The same for prefixes, whose states are joined in any case.
// (4 sequences behind 1000 tokens: 17.0 us with shares of 4 units and cuts after one step, 20.6 with the
// values above; 64 behind 8192: 68.4 and 66.0.)
constexpr int kPrefixMinSteps = 1, kPrefixShareShift = 2;
constexpr int kKeysPerTile = 128;
constexpr int kTileShift = 7;

// One packed sequence: its rows and keys, and its query tiles per pack.
struct PackedSeq {
  int32_t q_start, q_len, k_start, k_len, tiles;
};

OSS_HD PackedSeq packed_seq(RowRange q, RowRange k, int pos_shift) {
  PackedSeq s;
  s.q_start = q.start;
  s.q_len = q.len;
  s.k_start = k.start;
  s.k_len = k.len;
  s.tiles = static_cast<int32_t>((static_cast<int64_t>(q.len) + (int64_t(1) << pos_shift) - 1) >> pos_shift);
  return s;
}

// Keys that query i of the sequence sees (it may be <= 0).
OSS_HD int32_t visible_keys(const PackedSeq& s, int32_t i, bool causal) {
  if (!causal) return s.k_len;
  const int64_t n = static_cast<int64_t>(i) + 1 + s.k_len - s.q_len;
  return n < s.k_len ? static_cast<int32_t>(n) : s.k_len;
}

// KV tiles that query tile t visits: those its last query sees, at least one
// (a tile whose queries see no key visits a fully masked one).
OSS_HD int32_t kv_tiles(const PackedSeq& s, int32_t t, int pos_shift, bool causal) {
  const int64_t last = ((static_cast<int64_t>(t) + 1) << pos_shift) - 1;
  const int32_t n = visible_keys(s, last < s.q_len ? static_cast<int32_t>(last) : s.q_len - 1, causal);
  return n > 0 ? static_cast<int32_t>((static_cast<uint32_t>(n) + kKeysPerTile - 1) >> kTileShift) : 1;
}

// sum over n = 1 .. N of ceil(n / 2^q)
OSS_HD int64_t sum_of_ceils(int64_t N, int q) {
  const int64_t k = N >> q;
  return ((k * (k + 1)) << q) / 2 + (N - (k << q)) * (k + 1);
}

// Length of the items of query tiles 0 .. T - 1 of one pack (T <= tiles). In
// causal sequences tile t's last query sees off + (t + 1) P keys, off = k_len -
// q_len, P = 2^pos_shift queries a tile. Tiles with no key count 1; for the
// others, P divides 128, so the sum of the ceilings of (off + x P) / 128 is one
// over consecutive integers. The sequence's last tile may be short and is
// added by itself.
OSS_HD int64_t length_before(const PackedSeq& s, int32_t T, int pos_shift, bool causal) {
  if (T <= 0) return 0;
  const bool all = T == s.tiles;
  const int64_t last = causal && !all ? 0 : kv_tiles(s, s.tiles - 1, pos_shift, causal);
  int64_t sum = static_cast<int64_t>(T) * kTileWeight;
  if (!causal) return sum + T * last;
  int64_t n = all ? T - 1 : T;
  const int64_t off = static_cast<int64_t>(s.k_len) - s.q_len, from = off > 0 ? off : 0;
  int64_t none = (from - off) >> pos_shift;  // tiles whose queries see no key
  if (none > n) none = n;
  n -= none;
  const int64_t b = ((from & (kKeysPerTile - 1)) + (int64_t(1) << pos_shift) - 1) >> pos_shift;
  return sum + last + none + n * (from >> kTileShift) + sum_of_ceils(b + n, kTileShift - pos_shift) - b;
}

// The query tile that place `at` of a pack's items (0 <= at < length) lies in.
OSS_HD int32_t tile_at(const PackedSeq& s, int64_t at, int pos_shift, bool causal) {
  int32_t lo = 0, hi = s.tiles - 1;
  OSS_ROLLED
  while (lo < hi) {
    const int32_t mid = lo + (hi - lo + 1) / 2;
    if (length_before(s, mid, pos_shift, causal) <= at)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Shares of a row of items for `ctas` CTAs that take up to `rounds` each: no
// fewer than there are items where the CTAs reach; beyond that, a share holds at
// least 2^least_shift units (8: 6 KV steps, less is not worth a joined tile); and more than
// one round only as whole rounds, so that every CTA has the same number.
OSS_HD int32_t share_count(int64_t total, int64_t items, int32_t ctas, int32_t rounds, int least_shift = kLeastShareShift) {
  int64_t want = total >> least_shift;
  if (want < items) want = items;
  const int32_t most = ctas * rounds;
  int32_t n = want < most ? static_cast<int32_t>(want) : most;
  if (n > ctas) n -= static_cast<int32_t>(static_cast<uint32_t>(n) % static_cast<uint32_t>(ctas));
  return n;
}

// The boundaries: share c begins at place begin(c). 32-bit divisions only (the
// kernels run this once per launch, where a 64-bit one is a hundred instructions to
// fetch): a row of 2^32 units or more is cut in units of a power of two.
struct ShareCut {
  int64_t total;
  uint32_t count, per, rem;  // rem shares of per + 1 units, then shares of per
  int shift;
};

OSS_HD ShareCut share_cut(int64_t total, int32_t count) {
  ShareCut c;
  c.total = total;
  c.count = static_cast<uint32_t>(count);
  c.shift = 0;
  OSS_ROLLED
  while ((total >> c.shift) >> 31) ++c.shift;
  const uint32_t units = static_cast<uint32_t>((total + (int64_t(1) << c.shift) - 1) >> c.shift);
  c.per = count > 0 ? units / c.count : 0;
  c.rem = units - c.per * c.count;
  return c;
}

OSS_HD int64_t share_begin(const ShareCut& s, uint32_t c) {
  const int64_t x = static_cast<int64_t>(static_cast<uint64_t>(c) * s.per + (c < s.rem ? c : s.rem)) << s.shift;
  return x < s.total ? x : s.total;
}

// The last share that begins at or before place x (x < total).
OSS_HD uint32_t last_boundary(const ShareCut& s, int64_t x) {
  const uint32_t u = static_cast<uint32_t>(x >> s.shift), longer = s.rem * (s.per + 1);
  return u < longer ? u / (s.per + 1) : s.rem + (u - longer) / s.per;
}

// floor(x / y) for a quotient below 2^20.
OSS_HD int32_t small_quotient(int64_t x, int64_t y) {
  int32_t q = static_cast<int32_t>(static_cast<float>(x) / static_cast<float>(y));
  OSS_ROLLED
  while (q * y > x) --q;
  OSS_ROLLED
  while ((q + 1) * y <= x) ++q;
  return q;
}

// KV step at which a boundary `into` units inside an item cuts it: 0 moves the
// boundary to the item's start, `steps` to its end.
OSS_HD int32_t cut_step(int64_t into, int32_t steps, int32_t min_steps = kMinSteps) {
  const int64_t step = into - kTileWeight;
  if (step < min_steps) return 0;
  if (steps - step < min_steps) return steps;
  return static_cast<int32_t>(step);
}

}  // namespace oss
