// What the kernels of the paged decode share: a walk in equal shares over the cached
// tokens, the products' instructions, the states' merge, and the workspace. The reasons
// stand in decode_paged.cu.
#pragma once

#include <atomic>
#include <cstdint>

#include "device_common.cuh"
#include "launch.cuh"
#include "oss_internal.h"
#include "packed_plan.h"
#include "paged.h"
#include "prefix_split.cuh"

namespace oss {
namespace decode {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxDevices = 64;
constexpr int kTileKeys = 16;
constexpr int kUnitTiles = kWarps;  // a unit: one tile per warp
constexpr int kMaxHeadBlock = 16;
constexpr int kCtasPerSm = 2;  // of the 16-bit decode
// Items are not cut, and nothing is joined, when a row of the page table holds at
// most kWholeKeys tokens, or at most kWholeKeysMany and there are as many items
// as shares. Replayed from a graph, 32 heads over 8, whole against cut: 1 x 128 tokens
// 4.9 against 7.4 us, 1 x 333 7.8 / 7.6 (but 3 us of the host for the second launch),
// 64 x 256 12 / 18, 64 x 512 26 / 33; and 1 x 512 9.2 / 7.5. On the GPU the two meet
// before 333; up to 384 it is the host's second launch that decides. The rule goes by
// the table's width, because the lengths are on the device: short sequences in a wide
// table are cut.
constexpr int kWholeKeys = 384;
constexpr int kWholeKeysMany = 512;
constexpr float kLn2 = 0.69314718055994530942f;
// kMode other than kPlain: what an item costs beside its units, in units: its queries' way from memory
// and the warps' merge. Without it, shares of many short items took twice as long as others:
// 8-bit decode of 64 sequences of up to 8192 tokens 111.9 us with 0, 107.6 with 1, 106.6 with 2,
// 107.0 with 4; 64 of up to 1000 behind a prefix 68.8, 61.9, 58.2 and (3) 58.1. (The 16-bit
// decode keeps 0.)
constexpr int kItemWeight = 2;
// The reference maximum moves only when a score exceeds it by more than
// 2^kSlack: any reference gives the same quotient O / l, and weights up to 2^8 are
// as exact in bf16 and fp16 as weights up to 1.
constexpr float kSlack = 8.0f;

struct DecodeParams {
  PagedCache c;
  const uint16_t* q;
  int64_t ld_q_batch, ld_q_head;
  int32_t H, group, head_blocks, block_heads;  // block_heads: 8 or 16
  int32_t unit_tiles;                          // tiles of a unit: 4, or all of an item
  int32_t item_weight;  // what an item costs beside its units, in units
  float scale2;                                // scale * log2(e)
  uint16_t* o;
  float* lse;
  // workspace
  float* part_o;    // [2 N][block_heads][D]
  float2* part_ml;  // [2 N][block_heads]
  int4* meta;       // [N]: {sequence, key head and head block, parts, first slot}
  float* lse2;      // [batch][H], base 2: of items that were not cut (only with scores)
  int2* item_meta;  // [batch][heads * head_blocks]: {first share, parts}, or null
  // of the decode behind shared prefixes
  PrefixLaunch prefix;
  float* state_o;   // [sequences][H][D]: O of whole items (kPairs, kBehind)
  float2* state_ml;  // [sequences][H]: m, l
  float* scores;    // [batch][heads * head_blocks][capacity][score_heads], or null
  int32_t score_heads;
  unsigned int* err;
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 bytes from global to shared memory, zeros when !there.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <bool kF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What exponents are taken relative to where the maximum is m: 0 in place of -inf.
// A part without a key then adds zeros, and one whose scores are NaN (which no
// maximum shows) adds NaN instead of nothing.
__device__ __forceinline__ float reference(float m) { return m == neg_inf() ? 0.f : m; }

// What a launch of the decode is.
enum Mode {
  kPlain,   // the 16-bit decode: items have no weight, and end in o and lse
  kWeighed,  // the 8-bit decode: items have one
  // of the decode behind shared prefixes, ending in states:
  kPairs,   // two sequences for each of the batch: 2 b is the prefix of b's group, 2 b + 1 its own tokens
  kBehind,  // the own tokens, beside or behind the prefixes' kernel
};

// What an item costs beside its units, in units.
template <Mode kMode>
__device__ __forceinline__ int item_weight(const DecodeParams& p) {
  return kMode == kPlain ? 0 : p.item_weight;
}

// The sequences that a launch walks.
template <Mode kMode>
__device__ __forceinline__ int seq_count(const DecodeParams& p) {
  return kMode == kPairs ? 2 * p.c.batch : p.c.batch;
}

template <Mode kMode>
__device__ __forceinline__ int seq_len(const DecodeParams& p, int v) {
  if constexpr (kMode == kPairs) {
    const PrefixTables& t = p.prefix.tables;
    if ((v & 1) == 0) {
      const int g = prefix_group(t, v >> 1);
      return g < 0 ? 0 : paged_length(t.len[g], t.max_pages, p.c.page_shift);
    }
    v >>= 1;
  }
  return paged_length(p.c.kv_len[v], p.c.max_pages, p.c.page_shift);
}

// The sequence's row of its page table (of a sequence with tokens).
template <Mode kMode>
__device__ __forceinline__ const int32_t* seq_table(const DecodeParams& p, int v) {
  if constexpr (kMode == kPairs) {
    const PrefixTables& t = p.prefix.tables;
    if ((v & 1) == 0) return t.table + max(prefix_group(t, v >> 1), 0) * t.ld_table;
    v >>= 1;
  }
  return p.c.table + v * p.c.ld_table;
}

// Units [r0, r1) of an item: sequence b, key head and head block j.
struct Segment {
  int b, j, len, units, r0, r1;
};

// The walk of one CTA over its share of the row of items. An item takes
// item_weight + units places of the row, and unit k of an item that begins at place `at`
// lies at at + item_weight + k.
// kKeys: keys of a tile.
template <int kKeys, Mode kMode>
struct Walk {
  Segment s;
  int64_t at, end;  // where the segment's item and the share's end lie

  // (an empty sequence has a unit, to be answered)
  __device__ __forceinline__ static int units_of(const DecodeParams& p, int len) {
    if (p.unit_tiles != kUnitTiles) return 1;
    const int n = (len + kKeys * kUnitTiles - 1) / (kKeys * kUnitTiles);
    return n > 0 ? n : 1;
  }
  // The segment from unit r0 of the item at hand; false when the share ends before that.
  __device__ __forceinline__ bool clip(const DecodeParams& p, int64_t r0) {
    const int64_t r1 = end - at - item_weight<kMode>(p);
    s.r0 = static_cast<int>(r0);
    s.r1 = r1 < s.units ? static_cast<int>(r1 > 0 ? r1 : 0) : s.units;
    return s.r0 < s.r1;
  }
  // The next segment of the share; false when there is none.
  __device__ __forceinline__ bool next(const DecodeParams& p) {
    at += s.units + item_weight<kMode>(p);
    if (at + item_weight<kMode>(p) >= end) return false;
    if (++s.j == p.c.heads * p.head_blocks) {
      s.j = 0;
      ++s.b;
      s.len = seq_len<kMode>(p, s.b);
      s.units = units_of(p, s.len);
    }
    return clip(p, 0);
  }
  // One past the last tile of the segment that holds a key.
  __device__ __forceinline__ int tile_end(const DecodeParams& p) const {
    return min(s.r1 * p.unit_tiles, (s.len + kKeys - 1) / kKeys);
  }
};

// This CTA's share, from the lengths: every thread sums a run of sequences, a
// block scan places the runs, and the thread whose run holds the first unit
// finds the sequence in it. False when the CTA has no share.
template <int kKeys, Mode kMode>
__device__ __forceinline__ bool find_share(const DecodeParams& p, Walk<kKeys, kMode>* w, ShareCut* share) {
  using Walk = decode::Walk<kKeys, kMode>;
  __shared__ int64_t warp_sum[kWarps];
  __shared__ Walk found;
  __shared__ bool some;  // a share may lie within an item's weight
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int count = seq_count<kMode>(p), per = (count + kThreads - 1) / kThreads;
  const int b0 = min(count, static_cast<int>(threadIdx.x) * per), b1 = min(count, b0 + per);
  int64_t mine = 0;
  float own = 0.f;
  PackedSeq group = packed_seq(RowRange{0, 0, false}, RowRange{0, 0, false}, 0);
  const bool split = kMode == kBehind && p.prefix.bytes_cost > 0 && p.prefix.tables.groups <= kWarpGroups;  // SMs are left to the prefixes
  const int g = p.prefix.tables.groups == 1 ? 0 : threadIdx.x;
  if (split && warp == 0 && g < p.prefix.tables.groups)
    group = prefix_seq(p.prefix.tables, g, p.prefix.batch, p.prefix.page_shift, p.prefix.pos_shift);
  if constexpr (kMode == kPairs) {
    const PrefixTables& t = p.prefix.tables;
    for (int g = threadIdx.x; t.cu && blockIdx.x == 0 && g < t.groups; g += kThreads)
      if (row_range(t.cu[g], t.cu[g + 1], p.c.batch).clamped) report_error(p.err, kKernelPaged | (kSiteBadOffsets << 8));
  }
  for (int b = b0; b < b1; ++b) {
    const int len = seq_len<kMode>(p, b);
    mine += Walk::units_of(p, len) + item_weight<kMode>(p);
    if (split) own += static_cast<float>(own_units(len));
  }
  int64_t upto = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, upto, off);
    if (lane >= off) upto += y;
  }
  if (lane == 31) warp_sum[warp] = upto;
  __syncthreads();
  int64_t before = upto - mine, all = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += warp_sum[i];
    all += warp_sum[i];
  }
  const int per_seq = p.c.heads * p.head_blocks;
  const int64_t W = all * per_seq;
  int ctas = gridDim.x;
  if (split) {
    __shared__ float warp_own[kWarps];
    __shared__ int left;
    own = sum_of_warp(own);
    if (lane == 0) warp_own[warp] = own;
    __syncthreads();
    if (warp == 0) {
      own = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) own += warp_own[i];
      const PrefixDivision d = divide_prefix(p.prefix, group, own * static_cast<float>(p.prefix.per_seq));
      if (lane == 0) left = d.split ? p.prefix.sms - static_cast<int>(d.cut.count) * d.count : 0;
    }
    __syncthreads();
    // (0: the own tokens come behind the prefixes, on every SM)
    if (left > 0) ctas = min(ctas, kCtasPerSm * left);
  }
  const ShareCut cut = share_cut(W, W < ctas ? static_cast<int>(W) : ctas);
  *share = cut;
  if (blockIdx.x >= cut.count) return false;
  const int64_t first = share_begin(cut, blockIdx.x), last = share_begin(cut, blockIdx.x + 1);
  if (first >= before * per_seq && first < (before + mine) * per_seq) {
    int64_t at = before * per_seq;
    for (int b = b0; b < b1; ++b) {
      const int len = seq_len<kMode>(p, b);
      const int units = Walk::units_of(p, len), places = units + item_weight<kMode>(p);
      if (first < at + static_cast<int64_t>(places) * per_seq) {
        Walk f;
        f.s.b = b;
        f.s.j = small_quotient(first - at, places);
        f.s.len = len;
        f.s.units = units;
        f.at = at + static_cast<int64_t>(f.s.j) * places;
        f.end = last;
        const int64_t into = first - f.at - item_weight<kMode>(p);
        some = f.clip(p, into > 0 ? into : 0) || f.next(p);
        found = f;
        break;
      }
      at += static_cast<int64_t>(places) * per_seq;
    }
  }
  __syncthreads();
  *w = found;
  return some;
}

// Rows of the warps' outputs in shared memory, in floats: conflict-free for the
// accumulators' layouts.
template <int D>
constexpr int kMergeLd = D + 4;
template <int D>
constexpr int kMergeBytes = kWarps * 8 * kMergeLd<D> * 4;

// The four warps' states of 8 query heads, from head0 on (`heads` of them are live), as they
// lie in `merge` [warp][8][kMergeLd], m and l: the answer of an item that one CTA has
// seen whole (kPairs, kBehind: its state), else its part in `slot`.
template <bool kF16, int D, Mode kMode>
__device__ __forceinline__ void merge_warps(const DecodeParams& p, const Segment& s, bool whole, int slot, int head0,
                                            int in_block, int heads, const float* merge, const float (*merge_m)[8],
                                            const float (*merge_l)[8]) {
  // thread: head threadIdx.x / 16 of the 8, D / 16 dims
  constexpr int kDims = D / 16;
  const int hh = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * kDims;
  if (in_block + hh >= heads) return;
  float M = neg_inf(), L = 0.f, acc[kDims];
#pragma unroll
  for (int i = 0; i < kWarps; ++i) M = fmaxf(M, merge_m[i][hh]);
#pragma unroll
  for (int k = 0; k < kDims; ++k) acc[k] = 0.f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const float f = ex2(merge_m[i][hh] - reference(M));
    L = fmaf(merge_l[i][hh], f, L);
    const float4* src = reinterpret_cast<const float4*>(merge + (i * 8 + hh) * kMergeLd<D> + d0);
#pragma unroll
    for (int k = 0; k < kDims / 4; ++k) {
      const float4 x = src[k];
      acc[4 * k] = fmaf(x.x, f, acc[4 * k]);
      acc[4 * k + 1] = fmaf(x.y, f, acc[4 * k + 1]);
      acc[4 * k + 2] = fmaf(x.z, f, acc[4 * k + 2]);
      acc[4 * k + 3] = fmaf(x.w, f, acc[4 * k + 3]);
    }
  }
  const int64_t row = static_cast<int64_t>(s.b) * p.H + head0 + in_block + hh;
  constexpr bool kStates = kMode == kPairs || kMode == kBehind;
  if (whole && !kStates) {
    const float inv = L != 0.f ? 1.f / L : 0.f;
    uint32_t out[kDims / 2];
#pragma unroll
    for (int k = 0; k < kDims / 2; ++k) out[k] = pack2<kF16>(acc[2 * k] * inv, acc[2 * k + 1] * inv);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + d0);
    if constexpr (kDims == 8)
      *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
    if ((threadIdx.x & 15) == 0) {
      const float e2 = L != 0.f ? M + log2f(L) : neg_inf();
      if (p.lse) p.lse[row] = e2 * kLn2;
      if (p.scores) p.lse2[row] = e2;
    }
  } else {
    const int64_t at = whole ? row : static_cast<int64_t>(slot) * p.block_heads + in_block + hh;
    float4* dst = reinterpret_cast<float4*>((whole ? p.state_o : p.part_o) + at * D + d0);
#pragma unroll
    for (int k = 0; k < kDims / 4; ++k)
      dst[k] = make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
    if ((threadIdx.x & 15) == 0) (whole ? p.state_ml : p.part_ml)[at] = make_float2(M, L);
  }
}

// The part of an item that begins in this CTA's share: 2 blockIdx.x + 1, of others 2
// blockIdx.x. Where the item begins and is cut, thread 0 leaves its number of
// parts behind, for the join.
template <int kKeys, Mode kMode>
__device__ __forceinline__ int open_segment(const DecodeParams& p, const Walk<kKeys, kMode>& w, const ShareCut& share, bool whole) {
  const Segment& s = w.s;
  const int slot = 2 * blockIdx.x + (s.r0 == 0 ? 1 : 0);
  if (s.r0 == 0 && threadIdx.x == 0) {
    int parts = 1;
    if (!whole) {
      // the item's last unit lies in the last of its shares
      parts = static_cast<int>(last_boundary(share, w.at + item_weight<kMode>(p) + s.units - 1) - blockIdx.x) + 1;
      p.meta[blockIdx.x] = make_int4(s.b, s.j, parts, slot);
    }
    // (behind prefixes, parts < 0: no group names the sequence)
    if (kMode == kBehind && prefix_group(p.prefix.tables, s.b) < 0) parts = -parts;
    if (p.item_meta) p.item_meta[static_cast<int64_t>(s.b) * p.c.heads * p.head_blocks + s.j] = make_int2(blockIdx.x, parts);
  }
  return slot;
}

// Slot of part i of an item that begins in share c: part 0 in 2 c + 1, part i > 0 in 2 (c + i).
__device__ __forceinline__ int64_t part_slot(int c, int i) {
  return 2 * (static_cast<int64_t>(c) + i) + (i == 0 ? 1 : 0);
}

// Layout of the workspace, the same for its size and its use.
struct Plan {
  int shares, block_heads, head_blocks, score_heads, unit_tiles, item_weight;
  bool whole;  // items are not cut
  int64_t part_o, part_ml, meta, lse2, item_meta, scores, bytes;  // offsets, then the size
};

// Query heads that share one read of the cache.
inline int heads_of_block(int group) { return group <= 8 ? 8 : kMaxHeadBlock; }

// What the plan adds to the cache's tables: the parts of cut items, and optionally the scores
// and what else the weights' sums need.
// (ctas: of an SM; tile_keys: of the kernel's Walk; item_weight: as in DecodeParams, of items
// that may be cut.)
bool make_plan(int H, const os_paged_cache& c, int ctas, int tile_keys, int item_weight, bool weights, Plan* out);

// The parameters of a launch that writes o and lse, without weights and states.
DecodeParams decode_params(const Plan& pl, const PagedCache& c, const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head,
                           int H, float scale, uint16_t* o, float* lse, void* workspace, unsigned int* err);

// The second kernel of a launch that cuts items: their join.
cudaError_t launch_join(const DecodeParams& p, bool f16, int D, int shares, cudaStream_t stream);

// Raises a kernel's shared-memory limit, once per device: `done` [64] belongs to the kernel.
template <typename Kernel>
cudaError_t raise_smem(Kernel* kernel, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace decode
}  // namespace oss
