// Attention forward over packed sequences with grouped key heads, on the
// tcgen05 tensor cores.
//
// The recurrence, the tensor-memory layout and most roles of the warps are those
// of the dense attention forward (attn_fwd.cu): 8 softmax warps, a TMA producer,
// one thread that issues S = Q K^T and one that issues O += P V, three score
// buffers in tensor memory, the O rescale past a threshold of 2^8. What bounds
// it is the same chain; what is different here:
//
// Hand-over. Packed sequences are often short, and then the step from one query
// tile to the next counts. Four warps of their own read O out of tensor memory,
// scale and store it while the softmax warps are at the next tile's scores
// already, Q is two deep, and V has a load thread of its own: a hand-over costs
// two KV steps instead of three (8 causal sequences of up to 2500 tokens, 32 heads over 8:
// 159 us against 172 with the dense kernel's roles; 48 of up to 96: 23 against 26).
// Registers move to where they are needed: 184 a thread for the softmax, 80 for the
// epilogue, 64 for the others (512 threads x 128 at launch).
//
// What it reaches: one causal sequence of 16384 in 1.52-1.59 ms (1400 TFLOP/s, 0.73
// of the measured bf16 rate, 0.81 of the sustained one). A KV step takes about 1650
// cycles where its MMAs need 1024 and its exponentials 514 (31.9 a clock and SM):
// neither bounds it, but the chain scores - maximum - weights - P V of the one
// query tile in flight. With 64 dims the MMAs need 512 cycles, and the step stays. In turns
// with the dense kernel on that sequence with 32 key heads: 1.58 against 1.48 ms (1.56
// with 8 key heads). How much of the difference is the K ring, two stages here for the
// second Q buffer and three there, and how much the waits, has not been separated.
//
// Rows. A tile's 128 rows are 128 / P' consecutive queries times P' query heads of
// one key head, P' the largest power of two that divides G = Hq / Hkv (up to
// 128): row r is query r / P', head r % P'. The tile arrives by one 4-D TMA box.
// A group's heads share each K and V tile, and sequences shorter than 128 tokens
// fill more of a tile (32 queries x 4 heads instead of 128 x 1).
//
// Division. Lengths are known on the device only. The items (query tile x KV
// tiles) stand in a row, each as long as its KV tiles and a constant, and every
// CTA takes equal shares of the length (packed_plan.h): no tile list, no sorting, no
// idle CTA behind the longest sequence, and one query tile behind a long prefix
// spreads over the GPU. A share that begins or ends inside an item leaves an
// unnormalised (m, l, O) in the workspace; a second kernel joins the parts in
// share order. No atomics: every run gives the same bits. The shares of a
// round are neighbours, so the K and V that the CTAs read at one time stay in L2
// (rounds in launch_attn_packed).
//
// Prefixes. The same kernel reads prefixes that groups of sequences share (decode_shared.cu):
// a group's queries are one sequence, its keys are in pages, and items end in states for
// another kernel's join (kPrefix; lanes and the division of the SMs: prefix_split.cuh). 64 sequences, 4
// heads a key head, behind 65536 tokens of 8 key heads: 54 KV steps a CTA at 0.93 us, 62 us.
//
// Foreign rows. The last KV tile of a sequence reaches into the next sequence's
// rows, or into rows that nobody wrote. Their scores are replaced by -inf; their V
// rows are set to zero in shared memory, since a weight of 0 times NaN or
// infinity would still reach O.

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "device_common.cuh"
#include "launch.cuh"
#include "oss_internal.h"
#include "packed_plan.h"
#include "prefix_split.cuh"
#include "tcgen05.cuh"

namespace oss {
namespace {

constexpr int kBM = 128;          // rows per query tile (= tensor-memory lanes)
constexpr int kBN = 128;          // keys per KV tile
constexpr int kScores = 3;        // score buffers, and stages of the V ring
constexpr int kKStages = 2;       // K ring, and Q buffers
constexpr int kSoftWarps = 8;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kProducerWarp = 8;
constexpr int kQkWarp = 9;
constexpr int kPvWarp = 10;
constexpr int kVWarp = 11;
constexpr int kEpiWarp = 12;      // warps 12..15: epilogue, 32 rows each
constexpr int kEpiThreads = 128;
constexpr int kThreads = 512;
// registers a thread after the split; the warpgroups' sum is what the launch holds
constexpr int kSoftRegs = 184, kIssueRegs = 64, kEpiRegs = 80;
static_assert(256 * kSoftRegs + 128 * kIssueRegs + 128 * kEpiRegs <= kThreads * 128, "register split");
constexpr int kHalf = 128 * 128;  // 128 rows x 64 dims x 2 bytes
constexpr int kMaxRounds = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 384;
constexpr float kRescaleSlack = 8.0f;
constexpr float kLn2 = 0.69314718055994530942f;
static_assert(kBN == kKeysPerTile, "the plan counts KV tiles of this size");
__device__ __forceinline__ uint32_t col_s(int b) { return 128u * b; }

template <int D>
struct Smem {
  static constexpr int kTile = (D / 64) * kHalf;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kKStages * kTile;
  static constexpr int kOffV = kOffK + kKStages * kTile;
  static constexpr int kBytes = kOffV + kScores * kTile + 1024;  // + alignment slack
};

// What the prefix kernels read and write beside the others' parameters: KV tiles come
// from pages, and states go to a join with the sequences' own tokens.
struct PrefixOut {
  PrefixLaunch launch;
  const int32_t* kv_len;  // of the sequences' own tokens
  int32_t own_max_pages;
  int32_t num_pages, box_shift;  // a TMA box: 2^box_shift slots of a page
  int4* where;      // [tokens_q][packs]: {first slot / 2, parts (0: not cut), row of the first head in the tile, lanes}
  float* state_o;   // [tokens_q][Hq][D]: unnormalised O of items that are not cut
  float2* state_ml;  // [tokens_q][Hq]
};

struct PackedParams {
  uint16_t* o;
  float* lse;
  const int32_t *cu_q, *cu_k;
  int32_t batch, tokens_q, tokens_k, Hq, packs, packs_per_key_head, pos_shift, rounds;
  float C;  // scale * log2(e)
  int causal;
  unsigned int* err;
  uint32_t wait_cycles;  // limit of every wait
  int skip_v_step;  // test hook: the producer skips the V load of this step (-1: none)
  // workspace
  float4* part_o;   // [2 shares][D / 4][128 rows]: unnormalised O, 4 dims of a row
  float2* part_ml;  // [2 shares][128 rows]: base-2 m, l
  int4* meta;       // [shares]: {parts, first query row, queries, pack} of the item cut at its end
  PrefixOut prefix;  // of the prefix kernels
};

// Bounded wait, small: it is inlined some twenty times, the step and hand-over
// code of all roles has to stay in the instruction cache (with polls that read the
// error word inlined, warps waited for instructions most of the time), and a
// kernel that moves registers between warps makes no calls. A wait that runs out
// leaves its site in the abort flag, which ends the other waits of the CTA and is
// reported when all roles have stopped.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort_flag, int site,
                                           uint32_t limit /* cycles */) {
  const uint32_t t0 = static_cast<uint32_t>(clock());
  OSS_ROLLED
  do {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
  } while (static_cast<uint32_t>(clock()) - t0 < limit);
  *abort_flag = site;
  return false;
}
#define wait_bar(bar, parity, site) wait_phase((bar), (parity), abort_flag, (site), p.wait_cycles)

// Wait used while draining: ignores the abort flag.
__device__ __forceinline__ void drain_phase(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const uint32_t t0 = static_cast<uint32_t>(clock());
  OSS_ROLLED
  do {
    if (mbar_try_wait(bar, parity)) return;
  } while (static_cast<uint32_t>(clock()) - t0 < static_cast<uint32_t>(kDrainNs * 2));
  *abort_flag = kSiteDrain;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

constexpr int kUnits = 4;  // ring of units ahead of the slowest role
constexpr int kUnitReaders = 3 + kSoftWarps + kEpiThreads / 32;  // Q K^T, P V and V threads, warps: each lets a unit go once

// Place of KV step g in a ring of kDepth: g % kDepth, and the parity of g / kDepth.
template <int kDepth>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == kDepth) {
      at = 0;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ void st_shared_u4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
  uint4 x;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr));
  return x;
}

struct Barriers {
  uint64_t q_full[kKStages];  // Q tile landed
  uint64_t q_free[kKStages];  // every QK^T of the item in the Q buffer is done, and its O has left through it
  uint64_t k_full[kKStages];
  uint64_t v_full[kScores];
  uint64_t s_full[kScores];
  uint64_t p_ready[2][kScores];  // P of keys 0..63 / 64..127 written
  uint64_t o_done[kScores];      // P V done, for the steps of each buffer
  uint64_t o_free;               // the epilogue has read O out of tensor memory
  uint64_t ml_full, ml_free;     // m and l of an item's rows, for the epilogue
  uint64_t unit_full[kUnits], unit_free[kUnits];
  uint64_t drain[2];
};

// Where a share begins and ends: the item at place w of the row of items, and
// the KV step inside it.
struct ShareStart {
  int64_t w;
  int32_t seq, pack, tile, step;
};
struct ShareEnd {
  int64_t w;
  int32_t step;
};
struct Shares {
  ShareStart start[kMaxRounds];
  ShareEnd end[kMaxRounds];
  ShareCut cut;
  Lanes lanes;
  PackedSeq first;  // the sequence that the share begins in (prefix)
};

// (Prefix: sequence b is a group, its keys the group's prefix, and a tile one of every lane.)
template <bool kPrefix>
__device__ __forceinline__ PackedSeq load_seq(const PackedParams& p, int b, int lanes) {
  if constexpr (kPrefix) {
    const PrefixLaunch& x = p.prefix.launch;
    PackedSeq s = prefix_seq(x.tables, b, x.batch, x.page_shift, x.pos_shift);
    s.tiles = (s.tiles + lanes - 1) / lanes;
    return s;
  }
  return packed_seq(row_range(p.cu_q[b], p.cu_q[b + 1], p.tokens_q),
                    row_range(p.cu_k[b], p.cu_k[b + 1], p.tokens_k), p.pos_shift);
}

// Length of the items of sequences [b0, b1), in one pack, and their tiles.
template <bool kPrefix>
__device__ __forceinline__ int64_t run_length(const PackedParams& p, int lanes, int b0, int b1, uint32_t* tiles) {
  int64_t sum = 0;
  uint32_t n = 0;
  OSS_ROLLED
  for (int b = b0; b < b1; ++b) {
    const PackedSeq s = load_seq<kPrefix>(p, b, lanes);
    sum += length_before(s, s.tiles, p.pos_shift, p.causal != 0);
    n += static_cast<uint32_t>(s.tiles);
  }
  *tiles = n;
  return sum;
}

// The lanes where a warp does not hold the groups. `sums` [3] is shared and cleared here.
__device__ __forceinline__ Lanes find_lanes(const PackedParams& p, unsigned long long* sums) {
  if (threadIdx.x < 3) sums[threadIdx.x] = 0;
  __syncthreads();
  OSS_ROLLED
  for (int b = threadIdx.x; b < p.batch; b += kThreads) atomicMax(&sums[0], static_cast<unsigned long long>(load_seq<true>(p, b, 1).tiles));
  __syncthreads();
  int count = lane_count(max(1, static_cast<int>(sums[0])));
  OSS_ROLLED
  for (int b = threadIdx.x; b < p.batch; b += kThreads) {
    const PackedSeq s = load_seq<true>(p, b, 1);
    const unsigned long long steps = kTileWeight + kv_tiles(s, 0, p.pos_shift, false);
    atomicAdd(&sums[1], s.tiles * steps);
    atomicAdd(&sums[2], (s.tiles + count - 1) / count * count * steps);
  }
  __syncthreads();
  if (too_many_lanes(count, gridDim.x, static_cast<int64_t>(sums[1]), static_cast<int64_t>(sums[2]))) count = 1;
  return this_lane(count, gridDim.x / count);
}

// The same as find_shares, for up to kWarpGroups groups: one way to memory and two CTA
// barriers. Warp 0 looks for the share's beginning, warp 1 for its end. (find_shares took
// 4.2 of the 16 us of a small launch of one group.) `scratch` [kThreads / 32].
__device__ __forceinline__ void find_prefix_share(const PackedParams& p, Shares* sh, float* scratch) {
  constexpr uint32_t kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = warp;
  const PrefixLaunch& x = p.prefix.launch;
  PackedSeq s = packed_seq(RowRange{0, 0, false}, RowRange{0, 0, false}, p.pos_shift);
  const int mine = p.batch == 1 ? 0 : lane;
  if (warp < 2 && mine < p.batch) s = prefix_seq(x.tables, mine, x.batch, x.page_shift, x.pos_shift);
  float own = 0.f;
  if (x.bytes_cost > 0) {
    OSS_ROLLED
    for (int b = threadIdx.x; b < x.batch; b += kThreads)
      own += static_cast<float>(own_units(paged_length(p.prefix.kv_len[b], p.prefix.own_max_pages, x.page_shift)));
    own = sum_of_warp(own);
    if (lane == 0) scratch[warp] = own;
    __syncthreads();
    own = sum_of_warp(lane < kThreads / 32 ? scratch[lane] : 0.f) * static_cast<float>(x.per_seq);
  }
  if (warp < 2) {
    if (e == 0 && blockIdx.x == 0 && p.cu_q && lane < p.batch && row_range(p.cu_q[lane], p.cu_q[lane + 1], p.tokens_q).clamped)
      report_error(p.err, kKernelPaged | (kSiteBadOffsets << 8));
    const PrefixDivision d = divide_prefix(x, s, own);
    const Lanes lanes = this_lane(d.count, d.sets);
    if (lane == 0 && e == 0) {
      sh->cut = d.cut;
      sh->lanes = lanes;
    }
    ShareStart start{0, 0, 0, 0, 0};
    ShareEnd end{0, 0};
    int k = 0;  // the group
    if (lanes.set < d.cut.count) {
      const int64_t at = share_begin(d.cut, lanes.set + e);
      if (at == d.total) {
        end = ShareEnd{d.total, 0};
      } else {
        int64_t len = static_cast<int64_t>(d.s.tiles) * d.places, before = (d.upto - len) * p.packs;
        int each = d.places;
        if (p.batch > 1) {
          k = __ffs(__ballot_sync(kAll, d.upto * p.packs > at)) - 1;
          len = __shfl_sync(kAll, len, k);
          before = __shfl_sync(kAll, before, k);
          each = __shfl_sync(kAll, each, k);
        }
        const int steps = each - kTileWeight;
        const int pack = small_quotient(at - before, len);
        const int64_t in_pack = at - before - pack * len;
        const int tile = small_quotient(in_pack, each);
        const int64_t into = in_pack - static_cast<int64_t>(tile) * each, w = at - into;
        const int step = cut_step(into, steps, kPrefixMinSteps);
        start = ShareStart{w, k, pack, tile, step};
        end = step == steps ? ShareEnd{w + each, 0} : ShareEnd{w, step};
      }
    }
    if (e == 0 && lane == k) {
      sh->start[0] = start;
      sh->first = d.s;
    }
    if (e == 1 && lane == 0) sh->end[0] = end;
  }
  __syncthreads();
}

// Finds this CTA's shares. The sequences are cut into a run per warp, and each of
// those into a run per lane. All warps measure theirs; then warp 2 r + e looks
// for the beginning (e = 0) or the end (e = 1) of the share of round r: the warp's
// run that holds it, that run's lane, and so on down to a sequence, then the query
// tile, 32 candidates at a time. (One thread that searched alone took 7 us of a
// launch; rolled loops, because code that runs once is paid for in instruction
// fetches.)
static_assert(2 * kMaxRounds <= kThreads / 32, "a warp for every boundary");
template <bool kPrefix>
__device__ __forceinline__ void find_shares(const PackedParams& p, Shares* sh, int64_t* scratch /* [kThreads / 32] */, uint32_t* tile_scratch) {
  constexpr int kWarps = kThreads / 32;
  constexpr uint32_t kAll = 0xffffffffu;
  int64_t* warp_len = scratch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool causal = p.causal != 0;
  Lanes lanes{1, 0, gridDim.x, blockIdx.x};
  if constexpr (kPrefix) {
    lanes = find_lanes(p, reinterpret_cast<unsigned long long*>(tile_scratch + kWarps));
    if (threadIdx.x == 0) sh->lanes = lanes;
  }
  const int per_warp = (p.batch + kWarps - 1) / kWarps;
  int lo = min(p.batch, warp * per_warp), hi = min(p.batch, lo + per_warp);  // the run in hand
  int64_t before = 0, at = 0, sum = 0;
  uint32_t tiles = 0;
  const int r = warp >> 1, e = warp & 1;
  OSS_ROLLED
  for (int level = 0;; ++level) {
    // the lanes' runs of [lo, hi)
    const int per = (hi - lo + 31) / 32;
    const int b0 = min(hi, lo + lane * per), b1 = min(hi, b0 + per);
    sum = run_length<kPrefix>(p, lanes.count, b0, b1, &tiles);
    const int64_t upto = warp_scan(sum);
    if (level == 0) {
      if (blockIdx.x == 0) {
        OSS_ROLLED
        for (int b = b0; b < b1; ++b)
          if ((!kPrefix || p.cu_q) && (row_range(p.cu_q[b], p.cu_q[b + 1], p.tokens_q).clamped ||
                                       (!kPrefix && row_range(p.cu_k[b], p.cu_k[b + 1], p.tokens_k).clamped)))
            report_error(p.err, kKernelPaged | (kSiteBadOffsets << 8));
      }
      tiles = __reduce_add_sync(kAll, tiles);
      if (lane == 31) {
        warp_len[warp] = upto;
        tile_scratch[warp] = tiles;
      }
      if (threadIdx.x < kMaxRounds) {
        sh->start[threadIdx.x] = ShareStart{0, 0, 0, 0, 0};
        sh->end[threadIdx.x] = ShareEnd{0, 0};
      }
      __syncthreads();
      const int64_t len = warp_scan(lane < kWarps ? warp_len[lane] : 0);
      const int64_t items = static_cast<int64_t>(__reduce_add_sync(kAll, lane < kWarps ? tile_scratch[lane] : 0u)) * p.packs;
      const int64_t total = __shfl_sync(kAll, len, 31) * p.packs;
      const ShareCut cut = share_cut(total, share_count(total, items, lanes.sets, p.rounds, kPrefix ? kPrefixShareShift : kLeastShareShift));
      if (threadIdx.x == 0) sh->cut = cut;
      const uint32_t share = r * lanes.sets + lanes.set;
      if (r >= p.rounds || share >= cut.count) break;
      at = share_begin(cut, share + e);
      if (at == total) {
        if (lane == 0) sh->end[r] = ShareEnd{total, 0};
        break;
      }
      // the first warp's run that ends behind the boundary
      const int w = __ffs(__ballot_sync(kAll, len * p.packs > at)) - 1;
      lo = min(p.batch, w * per_warp);
      hi = min(p.batch, lo + per_warp);
      before = w > 0 ? __shfl_sync(kAll, len, w - 1) * p.packs : 0;
      continue;
    }
    const int k = __ffs(__ballot_sync(kAll, before + upto * p.packs > at)) - 1;
    lo = __shfl_sync(kAll, b0, k);
    hi = __shfl_sync(kAll, b1, k);
    before += __shfl_sync(kAll, upto - sum, k) * p.packs;
    if (hi - lo > 1) continue;
    // the sequence: its pack, then its query tile among T0 + lane * stride
    const int64_t len = __shfl_sync(kAll, sum, k);
    const int pack = small_quotient(at - before, len);
    before += pack * len;
    const PackedSeq s = load_seq<kPrefix>(p, lo, lanes.count);
    int tile = 0;
    int64_t stride = 1;
    while (stride * 32 < s.tiles) stride *= 32;
    int64_t place = 0;
    OSS_ROLLED
    for (; stride > 0; stride /= 32) {
      const int64_t T = tile + static_cast<int64_t>(lane) * stride;
      const int64_t x = T < s.tiles ? length_before(s, static_cast<int>(T), p.pos_shift, causal) : INT64_MAX;
      const int last = 31 - __clz(__ballot_sync(kAll, x <= at - before));
      tile += static_cast<int>(last * stride);
      place = __shfl_sync(kAll, x, last);
    }
    if (lane == 0) {
      const int64_t w = before + place;
      if (kPrefix && e == 0) sh->first = s;
      const int steps = kv_tiles(s, tile, p.pos_shift, causal);
      const int step = cut_step(at - w, steps, kPrefix ? kPrefixMinSteps : kMinSteps);
      if (e == 0)
        sh->start[r] = ShareStart{w, lo, pack, tile, step};
      else
        sh->end[r] = step == steps ? ShareEnd{w + kTileWeight + steps, 0} : ShareEnd{w, step};
    }
    break;
  }
  __syncthreads();
}

// A piece of an item: KV steps [s0, s1) of its n_kv.
struct Unit {
  int q_row, n_pos;       // first query row, queries of the tile
  int k_row, k_len, vis;  // first key row (or row of the prefix table), keys, keys that the tile's first query sees
  int n_kv, n_diag, s0, s1, pack, share;
  int parts;              // parts of the item, if it begins here and is cut
  int end;                // no unit: the shares are done
};

// The walk of a CTA over its shares.
struct Walk {
  PackedSeq s;
  int64_t w, end_w;
  int seq, pack, tile, s0, end_step, round;
  bool fetch;  // the next item belongs to a later sequence

  __device__ __forceinline__ void begin() {
    round = -1;
    w = end_w = 0;
    end_step = 0;
  }
  template <bool kPrefix>
  __device__ __forceinline__ bool next(const PackedParams& p, const Shares& sh, Unit& u) {
    const bool causal = p.causal != 0;
    OSS_ROLLED
    for (;;) {
      if (w > end_w || (w == end_w && end_step == 0)) {  // the share of the next round
        if (++round >= p.rounds) return false;
        const ShareStart a = sh.start[round];
        w = a.w;
        seq = kPrefix ? a.seq : a.seq - 1;
        pack = a.pack;
        tile = a.tile;
        s0 = a.step;
        end_w = sh.end[round].w;
        end_step = sh.end[round].step;
        fetch = !kPrefix;
        if constexpr (kPrefix) s = sh.first;
        continue;
      }
      if (fetch) {
        fetch = false;
        OSS_ROLLED
        do {
          s = load_seq<kPrefix>(p, ++seq, kPrefix ? sh.lanes.count : 1);
        } while (s.tiles == 0 && seq + 1 < p.batch);
      }
      const int steps = kv_tiles(s, tile, p.pos_shift, causal);
      const int s1 = w == end_w ? end_step : steps;
      const int from = s0;
      const int pos0 = (kPrefix ? tile * sh.lanes.count + sh.lanes.lane : tile) << p.pos_shift;
      const bool some = from < s1 && (!kPrefix || pos0 < s.q_len);  // (a lane may have no tile of a group)
      if (some) {
        u.q_row = s.q_start + pos0;
        u.n_pos = min(1 << p.pos_shift, s.q_len - pos0);
        u.k_row = kPrefix ? seq : s.k_start;
        u.k_len = s.k_len;
        u.vis = visible_keys(s, pos0, causal);
        u.n_kv = steps;
        // KV tiles that the first query does not see whole are visited first
        u.n_diag = causal ? max(0, steps - max(0, u.vis) / kBN) : 0;
        u.s0 = from;
        u.s1 = s1;
        u.pack = pack;
        u.share = kPrefix ? static_cast<int>(sh.lanes.set) : round * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
        u.parts = 0;
        if (from == 0 && s1 < steps)
          u.parts = static_cast<int>(last_boundary(sh.cut, w + kTileWeight + steps - (kPrefix ? kPrefixMinSteps : kMinSteps))) - u.share + 1;
        if constexpr (kPrefix) u.share = u.share * sh.lanes.count + sh.lanes.lane;
        u.end = 0;
      }
      w += kTileWeight + steps;
      s0 = 0;
      if (++tile == s.tiles) {
        tile = 0;
        if (++pack == p.packs) {
          pack = 0;
          fetch = true;
        }
      }
      if (some) return true;
    }
  }
};

// KV tile visited at step j of an item.
__device__ __forceinline__ int kv_tile(const Unit& u, int j) {
  return j < u.n_diag ? u.n_kv - 1 - j : j - u.n_diag;
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t w;
  if constexpr (kF16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// Row r of a tile, as a row of o and lse.
__device__ __forceinline__ int64_t out_row(const PackedParams& p, int q_row, int pack, int r) {
  const int head_shift = 7 - p.pos_shift;
  return static_cast<int64_t>(q_row + (r >> head_shift)) * p.Hq + (pack << head_shift) + (r & ((1 << head_shift) - 1));
}

constexpr int kBadRing = 8;  // steps whose masks of bad pages are kept: no reader is more than 4 behind

// A prefix's KV tile comes in pieces of 2^box_shift rows, a lane's each: its page, or
// num_pages (a box outside the pool: zeros) for pieces behind the last key and bad
// pages. *bad: a bit for every 16 keys that belong to the prefix and whose page is
// outside the pool.
__device__ __forceinline__ int piece_page(const PrefixOut& x, int group, int tile, int k_len, uint32_t* bad) {
  const int lane = threadIdx.x & 31, key = tile * kBN + (lane << x.box_shift);
  const bool mine = lane < (kBN >> x.box_shift) && key < k_len;
  const int page = mine ? x.launch.tables.table[group * x.launch.tables.ld_table + (key >> x.launch.page_shift)] : x.num_pages;
  const bool ok = page_ok(page, x.num_pages);
  const uint32_t pieces = __ballot_sync(0xffffffffu, mine && !ok);
  *bad = __ballot_sync(0xffffffffu, lane < kBN / 16 && ((pieces >> (lane >> (x.box_shift - 4))) & 1u));
  return ok ? page : x.num_pages;
}

// Loads this lane's piece of a KV tile (its halves of 64 dims) to `dst`, when the
// barrier knows of the tile's bytes.
template <int D>
__device__ __forceinline__ void load_piece(const PrefixOut& x, const CUtensorMap* map, uint32_t dst, uint32_t bar, int page,
                                           int head, int tile) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) mbar_expect_tx(bar, (D / 64) * kHalf);
  __syncwarp();
  if (lane < (kBN >> x.box_shift)) {
    const int slot = (tile * kBN) & ((1 << x.launch.page_shift) - 1);  // 0 for pages of a tile or less
#pragma unroll
    for (int h = 0; h < D / 64; ++h) tma_load_4d(dst + h * kHalf + (lane << (x.box_shift + 7)), map, bar, h * 64, slot, head, page);
  }
  __syncwarp();
}

template <int D, bool kF16, bool kPrefix>
__global__ void __launch_bounds__(kThreads, 1)
attn_packed_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const PackedParams p) {
  using L = Smem<D>;
  constexpr int kHalves = D / 64;
  constexpr uint32_t kIdescQK = make_idesc(kBM, kBN, false, kF16);
  constexpr uint32_t kIdescPV = make_idesc(kBM, D, true, kF16);
  extern __shared__ uint8_t smem_raw[];
  __shared__ Barriers bars;
  __shared__ Shares shares;
  __shared__ __align__(16) float2 row_ml[kBM];  // find_shares uses it first
  __shared__ Unit units[kUnits];
  __shared__ uint32_t tmem_base_slot;
  __shared__ int abort_flag_s;
  __shared__ uint32_t bad_keys[kBadRing];  // of the steps' KV tiles (prefix)
  volatile int* abort_flag = &abort_flag_s;
  if constexpr (!kPrefix) let_next_kernel_start();

  const uint32_t sbase = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(smem_addr(&bars.q_full[i]), 1);
      mbar_init(smem_addr(&bars.q_free[i]), 1 + kEpiThreads / 32);
      mbar_init(smem_addr(&bars.k_full[i]), 1);
    }
    for (int b = 0; b < kScores; ++b) {
      mbar_init(smem_addr(&bars.v_full[b]), 1);
      mbar_init(smem_addr(&bars.s_full[b]), 1);
      mbar_init(smem_addr(&bars.p_ready[0][b]), kSoftThreads);
      mbar_init(smem_addr(&bars.p_ready[1][b]), kSoftThreads);
      mbar_init(smem_addr(&bars.o_done[b]), 1);
    }
    mbar_init(smem_addr(&bars.o_free), kEpiThreads);
    mbar_init(smem_addr(&bars.ml_full), kSoftThreads);
    mbar_init(smem_addr(&bars.ml_free), kEpiThreads);
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(smem_addr(&bars.unit_full[i]), 1);
      mbar_init(smem_addr(&bars.unit_free[i]), kUnitReaders);
    }
    mbar_init(smem_addr(&bars.drain[0]), 1);
    mbar_init(smem_addr(&bars.drain[1]), 1);
    abort_flag_s = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  // (Before the wait: a CTA of this kernel takes the SM's whole register file, so none of
  // the kernel before it that holds tensor memory can share the SM with it.)
  if (warp == kQkWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&tmem_base_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  wait_for_previous_kernel();
  // (Prefix: the kernel behind this one reads nothing of it, and may begin once all that
  // came before this one has ended. It waits for this one at its own end.)
  if constexpr (kPrefix) let_next_kernel_start();
  if (!kPrefix && threadIdx.x < p.rounds) p.meta[threadIdx.x * gridDim.x + blockIdx.x] = make_int4(0, 0, 0, 0);
  if (kPrefix && p.batch <= kWarpGroups)
    find_prefix_share(p, &shares, reinterpret_cast<float*>(row_ml));
  else
    find_shares<kPrefix>(p, &shares, reinterpret_cast<int64_t*>(row_ml), reinterpret_cast<uint32_t*>(row_ml + 2 * kThreads / 32));  // its barriers publish the set-up above
  tc_fence_after();
  const uint32_t tbase = tmem_base_slot;

  // Every role takes the same units in turn and counts KV steps g across them: step
  // g uses score buffer and V stage g % 3 and K stage g % 2, unit kt Q buffer kt % 2.
  //
  // Unit kt, copied (the fields that the role uses) and let go at once. False:
  // there is none, or a wait gave up.
  auto take_unit = [&](int kt, Unit& u) -> bool {
    const int slot = kt % kUnits;
    if (!wait_bar(smem_addr(&bars.unit_full[slot]), (kt / kUnits) & 1, kSiteUnitFull)) return false;
    u = units[slot];
    mbar_arrive(smem_addr(&bars.unit_free[slot]));
    return !u.end;
  };
  // The same for a whole warp.
  auto take_unit_warp = [&](int kt, Unit& u) -> bool {
    const int slot = kt % kUnits;
    if (!__all_sync(0xffffffffu, wait_bar(smem_addr(&bars.unit_full[slot]), (kt / kUnits) & 1, kSiteUnitFull)))
      return false;
    u = units[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&bars.unit_free[slot]));
    return !u.end;
  };
  if (warp >= kProducerWarp && warp < kEpiWarp)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
  if (kPrefix && warp == kProducerWarp) {
    // ------------------------------------------- the same as below, with K in pieces
    // Lane 0 walks; every lane has a piece of the tile. A lane's page number is on its way
    // while the warp waits for the stage.
    Ring<kKStages> rk;
    Ring<kScores> sk;
    Walk walk;
    walk.begin();
    int kt = 0, g = 0;
    bool ok = true;
    OSS_ROLLED
    for (;; ++kt) {
      const int slot = kt % kUnits, buf = kt & 1;
      if (kt >= kUnits && !__all_sync(0xffffffffu, wait_bar(smem_addr(&bars.unit_free[slot]), (kt / kUnits - 1) & 1, kSiteUnitFree))) break;
      if (lane == 0) {
        Unit u;
        u.end = 1;
        walk.next<kPrefix>(p, shares, u);
        units[slot] = u;
        mbar_arrive(smem_addr(&bars.unit_full[slot]));
      }
      __syncwarp();
      const Unit u = units[slot];
      if (u.end) break;
      const uint32_t qb = smem_addr(&bars.q_full[buf]);
      if (kt >= kKStages && !__all_sync(0xffffffffu, wait_bar(smem_addr(&bars.q_free[buf]), ((kt >> 1) - 1) & 1, kSiteQEmpty))) break;
      if (lane == 0) {
        mbar_expect_tx(qb, L::kTile);
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          tma_load_4d(sbase + L::kOffQ + buf * L::kTile + h * kHalf, &tmap_q, qb, h * 64, 0, u.pack, u.q_row);
      }
      const int head = u.pack / p.packs_per_key_head;
      OSS_ROLLED
      for (int j = u.s0; j < u.s1; ++j, ++g, rk.next()) {
        uint32_t bad;
        const int tile = kv_tile(u, j), page = piece_page(p.prefix, u.k_row, tile, u.k_len, &bad);
        if (g >= kKStages) {
          if (!(ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.s_full[sk.at]), sk.phase, kSiteKEmpty)))) break;
          sk.next();
        }
        if (lane == 0) {
          bad_keys[g % kBadRing] = bad;
          if (bad) report_error(p.err, kKernelPaged | (kSiteBadPage << 8));
        }
        load_piece<D>(p.prefix, &tmap_k, sbase + L::kOffK + rk.at * L::kTile, smem_addr(&bars.k_full[rk.at]), page, head, tile);
      }
      if (!ok) {
        ++kt;  // its Q load has been issued
        break;
      }
    }
    if (lane == 0) {
      OSS_ROLLED
      for (int i = max(0, kt - kKStages); i < kt; ++i)
        drain_phase(smem_addr(&bars.q_full[i & 1]), (i >> 1) & 1, abort_flag);
      OSS_ROLLED
      for (int i = max(0, g - kKStages); i < g; ++i)
        drain_phase(smem_addr(&bars.k_full[i & 1]), (i >> 1) & 1, abort_flag);
    }
  } else if (kPrefix && warp == kVWarp) {
    Ring<kScores> r;
    Unit u;
    int g = 0, skipped = -1;
    bool ok = true;
    OSS_ROLLED
    for (int kt = 0; ok && take_unit_warp(kt, u); ++kt) {
      const int head = u.pack / p.packs_per_key_head;
      OSS_ROLLED
      for (int j = u.s0; j < u.s1; ++j, ++g, r.next()) {
        uint32_t bad;
        const int tile = kv_tile(u, j), page = piece_page(p.prefix, u.k_row, tile, u.k_len, &bad);
        if (g >= kScores && !(ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.o_done[r.at]), r.phase ^ 1, kSiteVEmpty)))) break;
        if (g == p.skip_v_step) {
          skipped = g;  // test hook: this V tile never arrives
          continue;
        }
        load_piece<D>(p.prefix, &tmap_v, sbase + L::kOffV + r.at * L::kTile, smem_addr(&bars.v_full[r.at]), page, head, tile);
      }
    }
    if (lane == 0) {
      OSS_ROLLED
      for (int i = max(0, g - kScores); i < g; ++i)
        if (i != skipped) drain_phase(smem_addr(&bars.v_full[i % kScores]), (i / kScores) & 1, abort_flag);
    }
  } else if (warp == kProducerWarp) {
    // ------------------------------------------- walk over the shares, Q and K
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_q)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
      // K_g goes to its stage when QK_{g-2} is done (s_full)
      static_assert(kKStages == 2, "sk below lags by two steps");
      Ring<kKStages> rk;
      Ring<kScores> sk;
      Walk walk;
      walk.begin();
      Unit u;
      int kt = 0, g = 0;
      bool ok = true;
      OSS_ROLLED
      for (;; ++kt) {
        const int slot = kt % kUnits, buf = kt & 1;
        if (kt >= kUnits && !wait_bar(smem_addr(&bars.unit_free[slot]), (kt / kUnits - 1) & 1, kSiteUnitFree)) break;
        u.end = 1;
        const bool have = walk.next<kPrefix>(p, shares, u);
        units[slot] = u;
        mbar_arrive(smem_addr(&bars.unit_full[slot]));
        if (!have) break;
        const uint32_t qb = smem_addr(&bars.q_full[buf]);
        if (kt >= kKStages && !wait_bar(smem_addr(&bars.q_free[buf]), ((kt >> 1) - 1) & 1, kSiteQEmpty)) break;
        mbar_expect_tx(qb, L::kTile);
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
          tma_load_4d(sbase + L::kOffQ + buf * L::kTile + h * kHalf, &tmap_q, qb, h * 64, 0, u.pack, u.q_row);
        const int head = u.pack / p.packs_per_key_head;
        OSS_ROLLED
        for (int j = u.s0; j < u.s1; ++j, ++g, rk.next()) {
          if (g >= kKStages) {
            if (!(ok = wait_bar(smem_addr(&bars.s_full[sk.at]), sk.phase, kSiteKEmpty))) break;
            sk.next();
          }
          const uint32_t kb = smem_addr(&bars.k_full[rk.at]);
          mbar_expect_tx(kb, L::kTile);
          const int row = u.k_row + kv_tile(u, j) * kBN;
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tma_load_3d(sbase + L::kOffK + rk.at * L::kTile + h * kHalf, &tmap_k, kb, h * 64, head, row);
        }
        if (!ok) {
          ++kt;  // its Q load has been issued
          break;
        }
      }
      // drain: every issued copy must land before the CTA may exit
      OSS_ROLLED
      for (int i = max(0, kt - kKStages); i < kt; ++i)
        drain_phase(smem_addr(&bars.q_full[i & 1]), (i >> 1) & 1, abort_flag);
      OSS_ROLLED
      for (int i = max(0, g - kKStages); i < g; ++i)
        drain_phase(smem_addr(&bars.k_full[i & 1]), (i >> 1) & 1, abort_flag);
    }
  } else if (warp == kVWarp) {
    // ------------------------------------------------------------------- V
    // V_g goes to its stage when P_{g-3} V is done (o_done). A thread of its own: behind
    // K it would wait for score buffers and Q buffers that the step it serves
    // does not need, which in items of a step or two is most of their time.
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
      Ring<kScores> r;
      Unit u;
      int g = 0, skipped = -1;
      bool ok = true;
      OSS_ROLLED
      for (int kt = 0; ok && take_unit(kt, u); ++kt) {
        const int head = u.pack / p.packs_per_key_head;
        OSS_ROLLED
        for (int j = u.s0; j < u.s1; ++j, ++g, r.next()) {
          if (g >= kScores && !(ok = wait_bar(smem_addr(&bars.o_done[r.at]), r.phase ^ 1, kSiteVEmpty))) break;
          if (g == p.skip_v_step) {
            skipped = g;  // test hook: this V tile never arrives
            continue;
          }
          const uint32_t vb = smem_addr(&bars.v_full[r.at]);
          mbar_expect_tx(vb, L::kTile);
          const int row = u.k_row + kv_tile(u, j) * kBN;
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tma_load_3d(sbase + L::kOffV + r.at * L::kTile + h * kHalf, &tmap_v, vb, h * 64, head, row);
        }
      }
      OSS_ROLLED
      for (int i = max(0, g - kScores); i < g; ++i)
        if (i != skipped) drain_phase(smem_addr(&bars.v_full[i % kScores]), (i / kScores) & 1, abort_flag);
    }
  } else if (warp == kQkWarp) {
    // ------------------------------------------------------------ QK issuer
    if (lane == 0) {
      bool ok = true;
      Ring<kScores> r;
      Ring<kKStages> rk;
      int g = 0;
      Unit u;
      OSS_ROLLED
      for (int kt = 0; ok && take_unit(kt, u); ++kt) {
        const int buf = kt & 1;
        if (!(ok = wait_bar(smem_addr(&bars.q_full[buf]), (kt >> 1) & 1, kSiteQFull))) break;
        const uint64_t dq = smem_desc(sbase + L::kOffQ + buf * L::kTile, 16, 1024);
        OSS_ROLLED
        for (int j = u.s0; j < u.s1; ++j, ++g, r.next(), rk.next()) {
          if (!(ok = wait_bar(smem_addr(&bars.k_full[rk.at]), rk.phase, kSiteKFull))) break;
          if (g >= kScores && !(ok = wait_bar(smem_addr(&bars.o_done[r.at]), r.phase ^ 1, kSiteODone))) break;
          tc_fence_after();
          const uint64_t dk = smem_desc(sbase + L::kOffK + rk.at * L::kTile, 16, 1024);
          const uint32_t d_s = tbase + col_s(r.at);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(d_s, dq + kstep_kmajor(kk, kHalf), dk + kstep_kmajor(kk, kHalf), kIdescQK, kk > 0 ? 1u : 0u);
          tc_commit(smem_addr(&bars.s_full[r.at]));
        }
        if (ok) tc_commit(smem_addr(&bars.q_free[buf]));
      }
      tc_commit(smem_addr(&bars.drain[0]));
      drain_phase(smem_addr(&bars.drain[0]), 0, abort_flag);
    }
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------ PV issuer
    if (lane == 0) {
      bool ok = true;
      const uint32_t d_o = tbase + kColO;
      Ring<kScores> r;
      Unit u;
      OSS_ROLLED
      for (int kt = 0; ok && take_unit(kt, u); ++kt) {
        OSS_ROLLED
        for (int j = u.s0; j < u.s1; ++j, r.next()) {
          if (!(ok = wait_bar(smem_addr(&bars.v_full[r.at]), r.phase, kSiteVFull))) break;
          if (j == u.s0 && kt > 0 && !(ok = wait_bar(smem_addr(&bars.o_free), (kt - 1) & 1, kSiteOFree))) break;
          const uint64_t dv = smem_desc(sbase + L::kOffV + r.at * L::kTile, kHalf, 1024);
          const uint32_t a_p = tbase + col_s(r.at);
          OSS_ROLLED
          for (int hp = 0; hp < 2; ++hp) {  // keys 0..63, 64..127 of the tile
            if (!(ok = wait_bar(smem_addr(&bars.p_ready[hp][r.at]), r.phase, kSitePReady))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ts(d_o, a_p + (4 * hp + kk) * 8, dv + static_cast<uint64_t>((4 * hp + kk) * (2048 >> 4)), kIdescPV,
                     (j > u.s0 || hp > 0 || kk > 0) ? 1u : 0u);
          }
          if (!ok) break;
          tc_commit(smem_addr(&bars.o_done[r.at]));
        }
      }
      tc_commit(smem_addr(&bars.drain[1]));
      drain_phase(smem_addr(&bars.drain[1]), 0, abort_flag);
    }
  } else if (warp >= kEpiWarp) {
    // ------------------------------------------------------------ epilogue
    // Thread: one row, 32 dims at a time. The scaled and rounded rows go to the
    // item's Q buffer, which nothing reads any more (128-byte rows, chunks swizzled), and
    // from there out in whole rows: stores of 16 bytes a row straight from here
    // kept the load/store unit busy for as long as a KV step, and the softmax warps'
    // barriers with it. Rolled loops: this code shares the instruction cache with
    // the softmax's.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int row0 = (warp - kEpiWarp) * 32;
    const uint32_t t_o = tbase + (static_cast<uint32_t>(row0) << 16) + kColO;
    const int head_shift = 7 - p.pos_shift;
    bool ok = true;
    int g = 0;  // steps of the items so far
    Unit u;
    OSS_ROLLED
    for (int kt = 0; ok && take_unit_warp(kt, u); ++kt) {
      g += u.s1 - u.s0;
      ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.ml_full), kt & 1, kSiteMlFull));
      if (!ok) break;
      const float2 ml = row_ml[row0 + lane];
      mbar_arrive(smem_addr(&bars.ml_free));
      ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.o_done[(g - 1) % kScores]), ((g - 1) / kScores) & 1, kSiteODone));
      if (!ok) break;
      tc_fence_after();
      const uint32_t stage = sbase + L::kOffQ + (kt & 1) * L::kTile + (warp - kEpiWarp) * (L::kTile / 4);  // [half][32 rows][128 bytes]
      if (kPrefix && u.s0 == 0) {
        // where the rows' states lie, for the kernel that joins them with the sequences' own tokens
        const int at = threadIdx.x - kEpiWarp * 32;
        if (at < u.n_pos) p.prefix.where[static_cast<int64_t>(u.q_row + at) * p.packs + u.pack] = make_int4(u.share, u.parts, at << head_shift, shares.lanes.count);
      }
      if (kPrefix && u.s0 == 0 && u.s1 == u.n_kv) {
        // The state as it is. 16 rows x 64 dims a load, of which 4 threads store the
        // 32 bytes of a row's sector.
        OSS_ROLLED
        for (int part = 0; part < 2 * kHalves; ++part) {
          const int half = part & 1, h = part >> 1;
          uint32_t v[32];
          tmem_ld16x256_x8(t_o + (static_cast<uint32_t>(16 * half) << 16) + 64 * h, v);
          tmem_ld_wait(v);
          if (part == 2 * kHalves - 1) {
            tc_fence_before();
            mbar_arrive(smem_addr(&bars.o_free));
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = row0 + 16 * half + 8 * e + (lane >> 2);
            if ((row >> head_shift) >= u.n_pos) continue;
            float* dst = p.prefix.state_o + out_row(p, u.q_row, u.pack, row) * D + 64 * h + 2 * (lane & 3);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<float2*>(dst + 8 * k) = make_float2(__uint_as_float(v[4 * k + 2 * e]), __uint_as_float(v[4 * k + 2 * e + 1]));
          }
        }
        if (((row0 + lane) >> head_shift) < u.n_pos) p.prefix.state_ml[out_row(p, u.q_row, u.pack, row0 + lane)] = ml;
      } else if (!kPrefix && u.s0 == 0 && u.s1 == u.n_kv) {
        // (a row without keys has O = 0: its weights are zeros and V is finite)
        const float inv = ml.y != 0.f ? 1.0f / ml.y : 0.f;
        OSS_ROLLED
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32x32_x32(t_o + 32 * c, v);
          tmem_ld_wait(v);
          const uint32_t dst = stage + (c >> 1) * (32 * 128) + lane * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack16<kF16>(__uint_as_float(v[8 * i + 2 * k]) * inv, __uint_as_float(v[8 * i + 2 * k + 1]) * inv);
            st_shared_u4(dst + (((4 * (c & 1) + i) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
          }
        }
        tc_fence_before();
        mbar_arrive(smem_addr(&bars.o_free));  // the next item's first P V may overwrite O
        __syncwarp();
        constexpr int kChunks = D / 8, kRows = 32 / kChunks;  // chunks of a row, rows of a pass
        uint4* base = reinterpret_cast<uint4*>(p.o + out_row(p, u.q_row, u.pack, 0) * D);
        const int c = lane % kChunks;
        const uint32_t from = stage + (c >> 3) * (32 * 128);
#pragma unroll 4
        for (int row = lane / kChunks; row < 32; row += kRows) {
          const uint4 x = ld_shared_u4(from + row * 128 + (((c & 7) ^ (row & 7)) << 4));
          const int at = (row0 + row) >> head_shift, head = (row0 + row) & ((1 << head_shift) - 1);
          if (at < u.n_pos) base[static_cast<int64_t>(at * p.Hq + head) * kChunks + c] = x;
        }
        __syncwarp();
        // (__log2f: off by at most 2^-22 for l in 0.5 .. 2, by 2 units in the last place
        // elsewhere. With log2f, which the join uses, 8 sequences of up to 2500 take 161.9
        // against 161.2 us.)
        if (p.lse && ((row0 + lane) >> head_shift) < u.n_pos)
          p.lse[out_row(p, u.q_row, u.pack, row0 + lane)] = ml.y != 0.f ? (ml.x + __log2f(ml.y)) * kLn2 : neg_inf();
      } else {
        const int64_t slot = 2 * static_cast<int64_t>(u.share) + (u.s0 == 0 ? 1 : 0);
        float4* dst = p.part_o + slot * (D / 4) * kBM + row0 + lane;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          tmem_ld32x32_x32(t_o + 32 * c, v);
          tmem_ld_wait(v);
          if (c == D / 32 - 1) {
            tc_fence_before();
            mbar_arrive(smem_addr(&bars.o_free));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[(8 * c + i) * kBM] = make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                                 __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3]));
        }
        p.part_ml[slot * kBM + row0 + lane] = ml;
        if (!kPrefix && u.parts > 0 && threadIdx.x == kEpiWarp * 32) p.meta[u.share] = make_int4(u.parts, u.q_row, u.n_pos, u.pack);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the next Q tile lands where O's rows were
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bars.q_free[kt & 1]));
    }
  } else if (warp < kSoftWarps) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // Warp w owns rows 32 (w % 4) + 16 (w / 4) .. + 15; thread t holds rows
    // ra = t/4 and rb = 8 + t/4 of them, columns 8k + cq + {0, 1}.
    const int lane0 = (warp & 3) * 32 + (warp >> 2) * 16;
    const int ra = lane0 + (lane >> 2);
    const int rb = ra + 8;
    const int cq = 2 * (lane & 3);
    const int head_shift = 7 - p.pos_shift;
    const int pos_a = ra >> head_shift, pos_b = rb >> head_shift;
    const uint32_t tl = tbase + (static_cast<uint32_t>(lane0) << 16);
    const float C = p.C;
    bool ok = true;
    Ring<kScores> r, before;  // of this step and of the one before
    int g = 0;                // steps so far (prefix)
    Unit u;
    OSS_ROLLED
    for (int kt = 0; ok && take_unit_warp(kt, u); ++kt) {
      float m_a = neg_inf(), m_b = neg_inf();  // reference maxima, base 2
      float l_a = 0.f, l_b = 0.f;              // this thread's share of the row sums
      const int vis_a = p.causal ? min(u.k_len, u.vis + pos_a) : u.k_len;  // keys the rows see
      const int vis_b = p.causal ? min(u.k_len, u.vis + pos_b) : u.k_len;
      // Rows behind the tile's queries hold another sequence's, or none: they have no
      // vote on the rescale, which would change how the warp's own rows are rounded
      // (-inf + inf is NaN, and no maximum exceeds either).
      const float slack_a = pos_a < u.n_pos ? kRescaleSlack : -neg_inf();
      const float slack_b = pos_b < u.n_pos ? kRescaleSlack : -neg_inf();
      OSS_ROLLED
      for (int j = u.s0; j < u.s1; ++j, before = r, r.next()) {
        const int b = r.at;
        const uint32_t colS = col_s(b);
        ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.s_full[b]), r.phase, kSiteSFull));
        if (!ok) break;
        tc_fence_after();
        uint32_t r0[32], r1[32];
        tmem_ld16x256_x8(tl + colS, r0);
        tmem_ld16x256_x8(tl + colS + 64, r1);
        tmem_ld_wait(r0);
        tmem_ld_wait(r1);
        float sa[32], sb[32];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sa[2 * k + e] = __uint_as_float(r0[4 * k + e]);
            sb[2 * k + e] = __uint_as_float(r0[4 * k + 2 + e]);
            sa[16 + 2 * k + e] = __uint_as_float(r1[4 * k + e]);
            sb[16 + 2 * k + e] = __uint_as_float(r1[4 * k + 2 + e]);
          }
        }
        const int key0 = kv_tile(u, j) * kBN;
        if constexpr (kPrefix) {
          const uint32_t bad = bad_keys[g++ % kBadRing];
          if (bad) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((bad >> (4 * (i >> 4) + ((i >> 2) & 3))) & 1u) sa[i] = sb[i] = neg_inf();
          }
        }
        if (key0 + kBN > (p.causal ? u.vis : u.k_len)) {
          const int lim_a = vis_a - key0, lim_b = vis_b - key0;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int col = (i >> 4) * 64 + ((i >> 1) & 7) * 8 + cq + (i & 1);
            if (col >= lim_a) sa[i] = neg_inf();
            if (col >= lim_b) sb[i] = neg_inf();
          }
        }
        float xa0 = neg_inf(), xa1 = neg_inf(), xb0 = neg_inf(), xb1 = neg_inf();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          xa0 = fmax3(xa0, sa[i], sa[i + 1]);
          xa1 = fmax3(xa1, sa[i + 2], sa[i + 3]);
          xb0 = fmax3(xb0, sb[i], sb[i + 1]);
          xb1 = fmax3(xb1, sb[i + 2], sb[i + 3]);
        }
        float xa = fmaxf(xa0, xa1), xb = fmaxf(xb0, xb1);
        xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
        xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
        xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2));
        xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2));
        const float mnew_a = fmaxf(m_a, xa * C), mnew_b = fmaxf(m_b, xb * C);
        const bool rescale = __any_sync(0xffffffffu, (mnew_a > m_a + slack_a) || (mnew_b > m_b + slack_b));
        float corr_a = 1.f, corr_b = 1.f;
        if (rescale) {
          corr_a = ex2(m_a - ((mnew_a == neg_inf()) ? 0.f : mnew_a));  // 0 while m = -inf
          corr_b = ex2(m_b - ((mnew_b == neg_inf()) ? 0.f : mnew_b));
          m_a = mnew_a;
          m_b = mnew_b;
        }
        if (rescale && j > u.s0) {
          // wait for P_{j-1} V (its completion implies every earlier one), then
          // rescale this warp's rows of O
          ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.o_done[before.at]), before.phase, kSiteODone));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < kHalves; ++h) {
            uint32_t ov[32];
            tmem_ld16x256_x8(tl + kColO + 64 * h, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float2 oa = __fmul2_rn(make_float2(__uint_as_float(ov[4 * k]), __uint_as_float(ov[4 * k + 1])),
                                           make_float2(corr_a, corr_a));
              const float2 ob = __fmul2_rn(make_float2(__uint_as_float(ov[4 * k + 2]), __uint_as_float(ov[4 * k + 3])),
                                           make_float2(corr_b, corr_b));
              ov[4 * k] = __float_as_uint(oa.x);
              ov[4 * k + 1] = __float_as_uint(oa.y);
              ov[4 * k + 2] = __float_as_uint(ob.x);
              ov[4 * k + 3] = __float_as_uint(ob.y);
            }
            tmem_st16x256_x8(tl + kColO + 64 * h, ov);
          }
        }
        if (key0 + kBN > u.k_len) {
          // rows of V behind the sequence's keys: zeros (a 16-byte chunk's place
          // in its 128-byte row does not matter for them)
          ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.v_full[r.at]), r.phase, kSiteVFull));
          if (!ok) break;
          const int first = max(0, u.k_len - key0);
          uint8_t* vt = smem_raw + (sbase - smem_addr(smem_raw)) + L::kOffV + b * L::kTile;
          for (int i = first * 8 + static_cast<int>(threadIdx.x); i < kBN * 8; i += kSoftThreads)
#pragma unroll
            for (int h = 0; h < kHalves; ++h)
              *reinterpret_cast<uint4*>(vt + h * kHalf + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        const float2 Cv = make_float2(C, C);
        const float ref_a = (m_a == neg_inf()) ? 0.f : m_a, ref_b = (m_b == neg_inf()) ? 0.f : m_b;
        const float2 mva = make_float2(-ref_a, -ref_a), mvb = make_float2(-ref_b, -ref_b);
        float2 acc_a = make_float2(0.f, 0.f), acc_b = acc_a;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int kk = 8 * h + k;
            const float2 ta = __ffma2_rn(make_float2(sa[2 * kk], sa[2 * kk + 1]), Cv, mva);
            const float2 tb = __ffma2_rn(make_float2(sb[2 * kk], sb[2 * kk + 1]), Cv, mvb);
            const float2 ea = make_float2(ex2(ta.x), ex2(ta.y));
            const float2 eb = make_float2(ex2(tb.x), ex2(tb.y));
            acc_a = __fadd2_rn(acc_a, ea);
            acc_b = __fadd2_rn(acc_b, eb);
            pk[2 * k] = pack16<kF16>(ea.x, ea.y);
            pk[2 * k + 1] = pack16<kF16>(eb.x, eb.y);
          }
          tmem_st16x128_x8(tl + colS + 32 * h, pk);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(smem_addr(&bars.p_ready[h][b]));
        }
        l_a = fmaf(l_a, corr_a, acc_a.x + acc_a.y);
        l_b = fmaf(l_b, corr_b, acc_b.x + acc_b.y);
      }
      l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
      l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
      if (!ok) break;
      if (kt > 0) {
        ok = __all_sync(0xffffffffu, wait_bar(smem_addr(&bars.ml_free), (kt - 1) & 1, kSiteMlFree));
        if (!ok) break;
      }
      if ((lane & 3) == 0) {
        row_ml[ra] = make_float2(m_a, l_a);
        row_ml[rb] = make_float2(m_b, l_b);
      }
      mbar_arrive(smem_addr(&bars.ml_full));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) report_error(p.err, kKernelAttnPacked | (static_cast<unsigned>(*abort_flag) << 8));
  if (warp == kQkWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(kTmemCols) : "memory");
  }
}

// The join: CTA (share, c) merges dims 32 c .. 32 c + 31 of the item that is
// cut at the share's end. Part 0 lies in slot 2 share + 1, part i in slot 2 (share
// + i). Thread: a row, 16 dims.
constexpr int kJoinThreads = 2 * kBM;

template <int D, bool kF16>
__global__ void __launch_bounds__(kJoinThreads) attn_packed_join_kernel(const PackedParams p) {
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int share = blockIdx.x;
  const int4 meta = p.meta[share];
  const int parts = meta.x;
  if (parts == 0) return;
  const int row = threadIdx.x & (kBM - 1), q4 = 8 * blockIdx.y + 4 * (threadIdx.x >> 7);  // first vector of 4 dims
  if ((row >> (7 - p.pos_shift)) >= meta.z) return;
  auto slot = [&](int i) -> int64_t { return 2 * (static_cast<int64_t>(share) + i) + (i == 0 ? 1 : 0); };
  float M = neg_inf();
  for (int i = 0; i < parts; ++i) M = fmaxf(M, p.part_ml[slot(i) * kBM + row].x);
  const float ref = M == neg_inf() ? 0.f : M;
  float L = 0.f, acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float2 ml = p.part_ml[slot(i) * kBM + row];
    const float4* src = p.part_o + (slot(i) * (D / 4) + q4) * kBM + row;
    float4 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = src[e * kBM];
    // a part in which the row sees no key has l = 0 and adds nothing; one whose scores
    // are NaN has NaN, although its maximum is -inf too
    if (ml.y == 0.f) continue;
    const float f = ex2(ml.x - ref);
    L = fmaf(ml.y, f, L);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[4 * e] = fmaf(v[e].x, f, acc[4 * e]);
      acc[4 * e + 1] = fmaf(v[e].y, f, acc[4 * e + 1]);
      acc[4 * e + 2] = fmaf(v[e].z, f, acc[4 * e + 2]);
      acc[4 * e + 3] = fmaf(v[e].w, f, acc[4 * e + 3]);
    }
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;
  const int64_t at = out_row(p, meta.y, meta.w, row);
  uint4* dst = reinterpret_cast<uint4*>(p.o + at * D + 4 * q4);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    dst[i] = make_uint4(pack16<kF16>(acc[8 * i] * inv, acc[8 * i + 1] * inv), pack16<kF16>(acc[8 * i + 2] * inv, acc[8 * i + 3] * inv),
                        pack16<kF16>(acc[8 * i + 4] * inv, acc[8 * i + 5] * inv), pack16<kF16>(acc[8 * i + 6] * inv, acc[8 * i + 7] * inv));
  if (q4 == 0 && p.lse) p.lse[at] = L != 0.f ? (M + log2f(L)) * kLn2 : neg_inf();
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// A tensor of `rank` dimensions, boxes of 64 x box[1] x ... elements, 128B
// swizzle. strides in elements, from dimension 1 on; a dimension of size 1 takes
// any stride.
bool make_map(CUtensorMap* map, const uint16_t* base, bool f16, int rank, const int64_t* dims, const int64_t* strides,
              const int* boxes) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t gd[4], gs[3];
  cuuint32_t box[4], es[4];
  for (int i = 0; i < rank; ++i) {
    gd[i] = static_cast<cuuint64_t>(dims[i]);
    box[i] = static_cast<cuuint32_t>(boxes[i]);
    es[i] = 1;
    if (i > 0) gs[i - 1] = static_cast<cuuint64_t>(dims[i] > 1 ? strides[i - 1] * 2 : dims[0] * 2);
  }
  return enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank),
             const_cast<uint16_t*>(base), gd, gs, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

// Heads of one key head that a tile packs: a power of two, at most 128.
int pack_heads(int group) {
  int n = 1;
  while (n < kBM && group % (2 * n) == 0) n *= 2;
  return n;
}

// Shares a CTA takes one after the other. The CTAs' shares of one round are
// neighbours in the row of items, so that the K and V they read at one time are
// about 1 / rounds of all; that part should stay in L2 (half of its 129 MB), since
// every query tile reads it again.
int round_count(int64_t tokens_k, int Hkv, int D) {
  const int64_t bytes = tokens_k * Hkv * D * 4, part = int64_t(64) << 20;
  const int64_t n = (bytes + part - 1) / part;
  return n < 1 ? 1 : (n > kMaxRounds ? kMaxRounds : static_cast<int>(n));
}

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

template <int D, bool kF16, bool kPrefix>
cudaError_t launch_shape(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PackedParams& p,
                         int ctas, cudaStream_t stream) {
  static std::atomic<bool> smem_set[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !smem_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(attn_packed_kernel<D, kF16, kPrefix>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) smem_set[dev].store(true, std::memory_order_release);
  }
  e = launch_after(attn_packed_kernel<D, kF16, kPrefix>, dim3(ctas), kThreads, Smem<D>::kBytes, stream, mq, mk, mv, p);
  if (e != cudaSuccess || kPrefix) return e;
  return launch_after(attn_packed_join_kernel<D, kF16>, dim3(ctas * p.rounds, D / 32), kJoinThreads, 0, stream, p);
}

template <bool kPrefix>
cudaError_t launch_kernel(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PackedParams& p, int D,
                          bool f16, int ctas, cudaStream_t stream) {
  if (D == 128)
    return f16 ? launch_shape<128, true, kPrefix>(mq, mk, mv, p, ctas, stream) : launch_shape<128, false, kPrefix>(mq, mk, mv, p, ctas, stream);
  return f16 ? launch_shape<64, true, kPrefix>(mq, mk, mv, p, ctas, stream) : launch_shape<64, false, kPrefix>(mq, mk, mv, p, ctas, stream);
}

// Query positions of a tile whose rows hold `heads` heads each, as a shift.
int tile_positions(int heads) {
  int pos_shift = 7;
  while ((kBM >> pos_shift) < heads) --pos_shift;
  return pos_shift;
}

bool make_q_map(CUtensorMap* map, const uint16_t* q, bool f16, int D, int H, int heads, int64_t tokens, int64_t ld_head,
                int64_t ld_token) {
  const int64_t dims[4] = {D, heads, H / heads, tokens}, strides[3] = {ld_head, ld_head * heads, ld_token};
  const int box[4] = {64, heads, 1, kBM / heads};
  return make_map(map, q, f16, 4, dims, strides, box);
}

uint32_t wait_limit(const AttnFault& fault) {
  const uint64_t timeout_ns = fault.timeout_ns > 0 ? static_cast<uint64_t>(fault.timeout_ns) : kTimeoutNs;
  return static_cast<uint32_t>(timeout_ns < kTimeoutNs ? timeout_ns * 2 : kTimeoutNs * 2);  // about 2 GHz
}

}  // namespace

int device_sms() {
  static std::atomic<int> cached[kMaxDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  if ((sms = cached[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  cached[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

int64_t attn_packed_workspace_bytes(int64_t tokens_k, int Hkv, int D) {
  const int sms = device_sms();
  if (sms < 1) return -1;
  const int64_t shares = static_cast<int64_t>(sms) * round_count(tokens_k, Hkv, D);
  return round256(2 * shares * D * kBM * 4) + round256(2 * shares * kBM * 8) + round256(shares * 16);
}

cudaError_t launch_attn_packed(const PackedArgs& a, void* workspace, unsigned int* err, const AttnFault& fault,
                               cudaStream_t stream) {
  const int sms = device_sms();
  if (sms < 1) return cudaErrorInvalidDevice;
  const int group = a.Hq / a.Hkv, heads = pack_heads(group);
  CUtensorMap mq, mk, mv;
  // without keys nothing of k and v is read: any mapped row stands in for them
  const bool keys = a.tokens_k > 0;
  const int64_t k_dims[3] = {a.D, keys ? a.Hkv : 1, keys ? a.tokens_k : 1};
  const int64_t k_strides[2] = {a.ld_kv_head, a.ld_kv_token};
  const int k_box[3] = {64, 1, kBN};
  if (!make_q_map(&mq, a.q, a.f16, a.D, a.Hq, heads, a.tokens_q, a.ld_q_head, a.ld_q_token) ||
      !make_map(&mk, keys ? a.k : a.q, a.f16, 3, k_dims, k_strides, k_box) ||
      !make_map(&mv, keys ? a.v : a.q, a.f16, 3, k_dims, k_strides, k_box))
    return cudaErrorInvalidValue;

  PackedParams p = {};
  p.o = a.o;
  p.lse = a.lse;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.batch = a.batch;
  p.tokens_q = static_cast<int32_t>(a.tokens_q);
  p.tokens_k = static_cast<int32_t>(a.tokens_k);
  p.Hq = a.Hq;
  p.packs = a.Hq / heads;
  p.packs_per_key_head = group / heads;
  p.pos_shift = tile_positions(heads);
  p.rounds = round_count(a.tokens_k, a.Hkv, a.D);
  p.C = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634074);
  p.causal = a.causal ? 1 : 0;
  p.err = err;
  p.wait_cycles = wait_limit(fault);
  p.skip_v_step = fault.skip_v_step;
  const int64_t shares = static_cast<int64_t>(sms) * p.rounds;
  char* ws = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float4*>(ws);
  ws += round256(2 * shares * a.D * kBM * 4);
  p.part_ml = reinterpret_cast<float2*>(ws);
  ws += round256(2 * shares * kBM * 8);
  p.meta = reinterpret_cast<int4*>(ws);
  return launch_kernel<false>(mq, mk, mv, p, a.D, a.f16, sms, stream);
}

PrefixPlan prefix_plan(int H, const os_paged_cache& c) {
  PrefixPlan pl;
  const int heads = pack_heads(H / c.heads);
  pl.head_shift = 7 - tile_positions(heads);
  pl.packs = H / heads;
  pl.shares = device_sms();
  int64_t at = 0;
  const auto take = [&](int64_t n) {
    const int64_t here = at;
    at += round256(n);
    return here;
  };
  const int64_t rows = static_cast<int64_t>(c.batch) * H;
  pl.part_o = take(2 * static_cast<int64_t>(pl.shares) * c.head_dim * kBM * 4);
  pl.part_ml = take(2 * static_cast<int64_t>(pl.shares) * kBM * 8);
  pl.where = take(static_cast<int64_t>(c.batch) * pl.packs * 16);
  pl.state_o = take(rows * c.head_dim * 4);
  pl.state_ml = take(rows * 8);
  pl.bytes = at;
  return pl;
}

cudaError_t launch_attn_prefix(const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head, int H, const os_paged_cache& c,
                               const PrefixLaunch& x, float scale, const PrefixPlan& pl, void* workspace,
                               unsigned int* err, const AttnFault& fault, cudaStream_t stream) {
  const int sms = device_sms();
  if (sms < 1) return cudaErrorInvalidDevice;
  const int heads = 1 << pl.head_shift, box_rows = c.page_size < kBN ? c.page_size : kBN;
  const bool f16 = c.dtype == OS_DTYPE_F16;
  CUtensorMap mq, mk, mv;
  const int64_t dims[4] = {c.head_dim, c.page_size, c.heads, c.num_pages}, strides[3] = {c.ld_slot, c.ld_head, c.ld_page};
  const int box[4] = {64, box_rows, 1, 1};
  if (!make_q_map(&mq, q, f16, c.head_dim, H, heads, c.batch, ld_q_head, ld_q_batch) ||
      !make_map(&mk, static_cast<const uint16_t*>(c.k_pages), f16, 4, dims, strides, box) ||
      !make_map(&mv, static_cast<const uint16_t*>(c.v_pages), f16, 4, dims, strides, box))
    return cudaErrorInvalidValue;
  char* ws = static_cast<char*>(workspace);
  PackedParams p = {};
  p.cu_q = x.tables.cu;
  p.batch = x.tables.groups;
  p.tokens_q = c.batch;
  p.Hq = H;
  p.packs = pl.packs;
  p.packs_per_key_head = pl.packs / c.heads;
  p.pos_shift = 7 - pl.head_shift;
  p.rounds = 1;
  p.C = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  p.err = err;
  p.wait_cycles = wait_limit(fault);
  p.skip_v_step = fault.skip_v_step;
  p.part_o = reinterpret_cast<float4*>(ws + pl.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_ml);
  p.prefix.launch = x;
  p.prefix.kv_len = c.kv_len;
  p.prefix.own_max_pages = c.max_pages;
  p.prefix.num_pages = c.num_pages;
  while ((1 << p.prefix.box_shift) < box_rows) ++p.prefix.box_shift;
  p.prefix.where = reinterpret_cast<int4*>(ws + pl.where);
  p.prefix.state_o = reinterpret_cast<float*>(ws + pl.state_o);
  p.prefix.state_ml = reinterpret_cast<float2*>(ws + pl.state_ml);
  return launch_kernel<true>(mq, mk, mv, p, c.head_dim, f16, sms, stream);
}

}  // namespace oss
