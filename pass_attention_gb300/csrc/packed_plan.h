// How the packed attention forward divides its work: arithmetic shared by
// the kernel and by a host-compiled test.
//
// A work item is one tile of 128 query rows: `positions` consecutive queries of a
// sequence times a pack of 128 / positions query heads that share a key head.
// It visits kv_tiles tiles of 128 keys. The items of a launch stand in a row,
// (sequence, pack, tile)-major, each kTileWeight + kv_tiles long (a tile's
// fill, epilogue and hand-over cost about as much as three KV steps), and the
// row is cut into equal shares, one or a few per CTA. A share's boundary that
// falls inside an item cuts it along the keys, unless one side would get fewer
// than kMinSteps KV steps: then the boundary moves to the item's edge.
#pragma once

#include <cstdint>

#include "paged.h"

namespace oss {

constexpr int kTileWeight = 3;
constexpr int kMinSteps = 3;
constexpr int kKeysPerTile = 128;

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
  return n > 0 ? (n + kKeysPerTile - 1) / kKeysPerTile : 1;
}

// sum over n = 1 .. N of ceil(n / q)
OSS_HD int64_t sum_of_ceils(int64_t N, int64_t q) {
  const int64_t k = N / q;
  return q * k * (k + 1) / 2 + (N - k * q) * (k + 1);
}

// Length of the items of query tiles 0 .. T - 1 of one pack (T <= tiles). In
// causal sequences tile t's last query sees off + (t + 1) P keys, off = k_len -
// q_len, P = 2^pos_shift queries a tile; P divides 128, so the sum of the
// ceilings is one over consecutive integers. The sequence's last tile may be short
// and is added by itself.
OSS_HD int64_t length_before(const PackedSeq& s, int32_t T, int pos_shift, bool causal) {
  if (T <= 0) return 0;
  int64_t sum = static_cast<int64_t>(T) * kTileWeight;
  if (!causal) return sum + static_cast<int64_t>(T) * kv_tiles(s, 0, pos_shift, false);
  int64_t n = T;
  if (T == s.tiles) {
    sum += kv_tiles(s, T - 1, pos_shift, true);
    --n;
  }
  const int64_t off = static_cast<int64_t>(s.k_len) - s.q_len;
  const int64_t q = kKeysPerTile >> pos_shift;
  if (off < 0) {
    int64_t none = -off >> pos_shift;  // tiles whose queries see no key
    if (none > n) none = n;
    return sum + none + sum_of_ceils(n - none, q);
  }
  const int64_t whole = off / kKeysPerTile, rest = off % kKeysPerTile;
  const int64_t b = (rest + (int64_t(1) << pos_shift) - 1) >> pos_shift;
  return sum + n * whole + sum_of_ceils(b + n, q) - sum_of_ceils(b, q);
}

// The query tile that place `at` of a pack's items (0 <= at < length) lies in.
OSS_HD int32_t tile_at(const PackedSeq& s, int64_t at, int pos_shift, bool causal) {
  int32_t lo = 0, hi = s.tiles - 1;
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
// least 8 units (5 KV steps), less is not worth a joined tile; and more than
// one round only as whole rounds, so that every CTA has the same number.
OSS_HD int32_t share_count(int64_t total, int64_t items, int32_t ctas, int32_t rounds) {
  int64_t n = total / 8;
  if (n < items) n = items;
  if (n > static_cast<int64_t>(ctas) * rounds) n = static_cast<int64_t>(ctas) * rounds;
  if (n > ctas) n = n / ctas * ctas;
  return static_cast<int32_t>(n);
}

OSS_HD int64_t share_begin(int64_t c, int64_t total, int64_t shares) { return c * total / shares; }

// The last share boundary at or before place x.
OSS_HD int64_t last_boundary(int64_t x, int64_t total, int64_t shares) {
  return ((x + 1) * shares - 1) / total;
}

// KV step at which a boundary `into` units inside an item cuts it: 0 moves the
// boundary to the item's start, `steps` to its end.
OSS_HD int32_t cut_step(int64_t into, int32_t steps) {
  const int64_t step = into - kTileWeight;
  if (step < kMinSteps) return 0;
  if (steps - step < kMinSteps) return steps;
  return static_cast<int32_t>(step);
}

}  // namespace oss
