// How the prefixes' kernel of os_attention_decode_shared divides its work, and which SMs
// it leaves to the kernel of the sequences' own tokens: both kernels work this out, from
// the same lengths.
#pragma once

#include <cstdint>

#include "packed_plan.h"
#include "paged.h"

namespace oss {

// With several query tiles on one prefix, `count` CTAs (lanes) take the same shares, each with a
// tile of its own (tile number at * count + lane), and so read the same K and V at the
// same time, which then come from HBM once. As items of their own the tiles were half a
// share apart: 64 sequences, 4 heads a key head, behind 65536 tokens read the prefix's
// 268 MB twice (87 us, the kernel alone, against 62).
struct Lanes {
  int32_t count, lane;
  uint32_t sets, set;  // sets of `count` CTAs, and this CTA's
};

// As many lanes as the group with the most tiles has tiles, up to 8 (beyond that in equal
// shares of them), if that leaves at most a fifth of the CTAs' time idle in groups of
// fewer tiles; else 1.
constexpr int kMaxLanes = 8;

__device__ __forceinline__ int lane_count(int tiles) {
  const int per = (tiles + kMaxLanes - 1) / kMaxLanes;
  return (tiles + per - 1) / per;
}

// real, padded: steps of all tiles, and with the lanes' idle ones.
__device__ __forceinline__ bool too_many_lanes(int lanes, int ctas, int64_t real, int64_t padded) {
  return lanes > ctas || padded * 4 > real * 5;
}

__device__ __forceinline__ Lanes this_lane(int count, uint32_t sets) {
  Lanes x;
  x.count = count;
  x.sets = sets;
  x.set = blockIdx.x / count;
  x.lane = static_cast<int>(blockIdx.x - x.set * count);
  return x;
}

// Inclusive scan over a warp.
__device__ __forceinline__ int64_t warp_scan(int64_t x) {
  const int lane = threadIdx.x & 31;
  OSS_ROLLED
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  return x;
}

// Query tiles and keys of group b: its prefix is the "sequence".
__device__ __forceinline__ PackedSeq prefix_seq(const PrefixTables& t, int b, int32_t batch, int page_shift, int pos_shift) {
  const RowRange q = t.cu ? row_range(t.cu[b], t.cu[b + 1], batch) : RowRange{0, batch, false};
  return packed_seq(q, RowRange{0, paged_length(t.len[b], t.max_pages, page_shift), false}, pos_shift);
}

// What both kernels know of a launch.
struct PrefixLaunch {
  PrefixTables tables;
  int32_t batch, page_shift, pos_shift, packs;
  int32_t sms;
  int32_t per_seq;  // items of a sequence's own tokens: key heads and blocks of query heads
  int32_t step_cost, unit_cost, bytes_cost;  // see below; bytes_cost 0: no division (own tokens of few pages)
};

// Units of 64 keys of an item of the own tokens.
__device__ __forceinline__ int32_t own_units(int32_t len) { return (len + 63) / 64; }

// Groups up to which a warp divides a launch, a lane each. (Launches of more take all SMs for
// the prefixes, and then all for the own tokens.)
constexpr int kWarpGroups = 32;

struct PrefixDivision {
  PackedSeq s;      // this lane's group; tiles: of a lane
  int32_t places;   // of one of its items
  int64_t upto;     // inclusive sum over the groups' places, of one pack
  int64_t total;    // places of all packs
  int32_t count;    // lanes
  uint32_t sets;
  bool split;       // the own tokens' kernel runs beside this one, on the SMs that it leaves
  ShareCut cut;
};

// What the two kernels' parts cost, in sixteenths of a microsecond of an SM (fits of their
// times at D 128, unless it says otherwise).
constexpr int kStepCost = 18;       // a KV step of a tile
constexpr int kStepCost64 = 12;     // the same, D 64
constexpr int kItemCost = 28;       // an item of the own tokens, beside its units
constexpr int kUnitCost = 6;        // a unit, for up to 8 query heads
constexpr int kUnitCost64 = 4;      // the same, D 64
constexpr int kWideUnitCost = 18;   // for up to 16: these are bound by their arithmetic
constexpr int kUnitBytesCost = 12;  // a unit's bytes, when all SMs share HBM

// The SMs that the prefixes get. Where the own tokens are bound by HBM and the prefixes
// by the chain of a KV step, each kernel alone leaves idle what the other lacks: they run
// side by side, on SMs divided by what either asks of an SM, so that both end together.
// Otherwise the prefixes take what they can use, and the own tokens come behind them. One
// behind the other against side by side, us (sequences, heads, prefix, own tokens up to): 64, 32 /
// 8, 8192, 1000: 54.5 / 46.4; 64, 32 / 8, 65536, 2500: 119 / 111; 8, 32 / 8, 32768, 8192: 76.9 /
// 63.8; 4, 8 / 1, 100000, 3000: 53.3 / 42.7; and where the rule keeps them apart, forced:
// 64, 64 / 4, 16384, 1000: 62 / 71; 256, 32 / 8, 16384, 512: 130 / 154.
__device__ __forceinline__ int prefix_ctas(const PrefixLaunch& x, float steps, float units) {
  const float own = static_cast<float>(kItemCost * x.per_seq) * static_cast<float>(x.batch) + static_cast<float>(x.unit_cost) * units;
  if (static_cast<float>(x.bytes_cost) * units <= own) return x.sms;
  const float mine = static_cast<float>(x.step_cost) * steps;
  return static_cast<int>(static_cast<float>(x.sms) * __fdividef(mine, mine + own));
}

// One warp, converged. s: of this lane's group, or without tiles (one group: the same for all
// lanes); units: of all own tokens. This runs at the front of both kernels, where every
// instruction is fetched for the first time: the split of the SMs in floats, no scans for
// one group (3.2 us of a launch with 64-bit divisions and scans in any case).
__device__ __forceinline__ PrefixDivision divide_prefix(const PrefixLaunch& x, PackedSeq s, float units) {
  constexpr uint32_t kAll = 0xffffffffu;
  const bool one = x.tables.groups == 1;
  PrefixDivision d;
  d.places = kTileWeight + kv_tiles(s, 0, x.pos_shift, false);
  const int32_t tiles = s.tiles;
  d.count = lane_count(max(1, one ? tiles : __reduce_max_sync(kAll, tiles)));
  s.tiles = (tiles + d.count - 1) / d.count;
  int64_t real = static_cast<int64_t>(tiles) * d.places;
  d.upto = static_cast<int64_t>(s.tiles) * d.places;
  d.total = d.upto;
  if (!one) {
    real = __shfl_sync(kAll, warp_scan(real), 31);
    d.upto = warp_scan(d.upto);
    d.total = __shfl_sync(kAll, d.upto, 31);
  }
  if (too_many_lanes(d.count, x.sms, real, d.total * d.count)) {
    d.count = 1;
    s.tiles = tiles;
    d.upto = d.total = static_cast<int64_t>(tiles) * d.places;
    if (!one) {
      d.upto = warp_scan(d.upto);
      d.total = real;
    }
  }
  d.s = s;
  d.total *= x.packs;
  const int ctas = prefix_ctas(x, static_cast<float>(d.total) * static_cast<float>(d.count), units);
  d.split = ctas < x.sms;
  d.sets = static_cast<uint32_t>(max(1, min((ctas + d.count / 2) / d.count, x.sms / d.count)));
  const uint32_t all_tiles = one ? static_cast<uint32_t>(s.tiles) : __reduce_add_sync(kAll, static_cast<uint32_t>(s.tiles));
  d.cut = share_cut(d.total, share_count(d.total, static_cast<int64_t>(all_tiles) * x.packs, d.sets, 1, kPrefixShareShift));
  return d;
}

// Sum over a warp, in every lane.
__device__ __forceinline__ float sum_of_warp(float x) {
  OSS_ROLLED
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

}  // namespace oss
