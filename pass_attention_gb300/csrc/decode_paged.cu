// Attention of one new token per sequence over a paged key-value cache.
//
//   s_t = scale q.k_t;  lse = ln sum exp s_t;  o = sum exp(s_t - lse) v_t
//
// for each query head, G = H / heads query heads reading one key head. What
// bounds it: every cached key and value row is read once from HBM (4 D bytes a
// token and key head) for 4 D G operations, so the G heads of a group have to
// share one read, and from G = 4 on the FMA pipes could not keep up with HBM.
// The products therefore run on mma.sync (m16n8k16), with the keys on the wide side
// and the heads on the narrow one, so that a group of 8 heads or fewer
// fills the instruction (up to 16 heads share a read, in two instructions; a group of
// more is cut into blocks of 16 that each read the cache):
//   S^T [16 keys x 8 heads]  = K [16 x D] Q^T [D x 8]
//   O^T [16 dims x 8 heads] += V^T [16 x 16 keys] P^T [16 x 8]
// K and V tiles come out of shared memory by ldmatrix (transposed for V), and
// P^T is the 8 x 8 transpose of S^T's registers (movmatrix). (tcgen05 wants 128
// rows of one operand; with at most 16 heads the tile would be mostly idle and
// its round trip through tensor memory longer than the 0.2 us a tile lasts.)
//
// Division of the work: a unit is 64 keys of an item, an item being one
// sequence, key head and block of up to 16 query heads. The units of all items
// stand in a row, and every CTA takes an equal share of them (share_cut): equal shares
// of the bytes whatever the lengths are, from lengths that only the device
// knows. An item inside one share is finished there; one that crosses shares
// leaves partial states (m, l, O), which a second kernel joins in share order.
// No atomics: every run gives the same bits. Short caches (kWholeKeys) are not cut:
// an item is one unit then, and there is nothing to join.
//
// With weights, the first kernel leaves its scores in the workspace, and the second
// one, beside the joins, adds 2^(s - lse) to the sums: 4 bytes a head against
// the 2 D of reading the key again.
//
// What it reaches: 64 sequences of up to 8192 tokens, 32 heads over 8, 193 us (6.4
// TB/s, 0.95 of the copy peak); 6 of up to 32768, 16 heads of 64 in fp16, 104 us
// (0.93). (A stream that is only read may exceed the copy's rate: the dense split decode
// reads 7.35 TB/s.) A step over 1.2 MB of cache takes 8 us: the chain from the lengths over the
// page table to the keys, on 8 SMs of 152.
//
// Each of a CTA's four warps streams tiles of 16 keys (every fourth one of its
// segment) through its own ring in shared memory, by 16-byte asynchronous
// copies with a cursor that runs ahead across segments, so no CTA barrier
// stands between the loads. A page holds whole tiles (page_size >= 16).

#include <atomic>
#include <cstdint>

#include "device_common.cuh"
#include "launch.cuh"
#include "oss_internal.h"
#include "packed_plan.h"
#include "paged.h"

namespace oss {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTileKeys = 16;
constexpr int kUnitTiles = kWarps;  // a unit: one tile per warp
constexpr int kCtasPerSm = 2;
constexpr int kMaxHeadBlock = 16;
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
// The reference maximum moves only when a score exceeds it by more than
// 2^kSlack: any reference gives the same quotient O / l, and weights up to 2^8 are
// as exact in bf16 and fp16 as weights up to 1.
constexpr float kSlack = 8.0f;

template <int D>
struct Shape {
  static constexpr int kStages = D == 128 ? 3 : 6;  // 24 KB of K and V in flight per warp
  static constexpr int kRowBytes = D * 2;
  static constexpr int kTileBytes = kTileKeys * kRowBytes;  // K or V
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kMergeLd = D + 4;  // floats; conflict-free for the accumulators' layout
  static constexpr int kMergeBytes = kWarps * 8 * kMergeLd * 4;
  static constexpr int kSmemBytes = kRingBytes + kMergeBytes;
};

struct DecodeParams {
  PagedCache c;
  const uint16_t* q;
  int64_t ld_q_batch, ld_q_head;
  int32_t H, group, head_blocks, block_heads;  // block_heads: 8 or 16
  int32_t unit_tiles;                          // tiles of a unit: 4, or all of an item
  float scale2;                                // scale * log2(e)
  uint16_t* o;
  float* lse;
  // workspace
  float* part_o;    // [2 N][block_heads][D]
  float2* part_ml;  // [2 N][block_heads]
  int4* meta;       // [N]: {sequence, key head and head block, parts, first slot}
  float* lse2;      // [batch][H], base 2: of items that were not cut (only with scores)
  int2* item_meta;  // [batch][heads * head_blocks]: {first share, parts} (only with scores)
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

template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t w;
  if constexpr (kF16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// What exponents are taken relative to where the maximum is m: 0 in place of -inf.
// A part without a key then adds zeros, and one whose scores are NaN (which no
// maximum shows) adds NaN instead of nothing.
__device__ __forceinline__ float reference(float m) { return m == neg_inf() ? 0.f : m; }

// Units [r0, r1) of an item: sequence b, key head and head block j.
struct Segment {
  int b, j, len, units, r0, r1;
};

// The walk of one CTA over its share [u, end) of the units.
struct Walk {
  Segment s;
  int64_t u, end;

  // (an empty sequence has a unit, to be answered)
  __device__ __forceinline__ static int units_of(const DecodeParams& p, int len) {
    if (p.unit_tiles != kUnitTiles) return 1;
    const int n = (len + kTileKeys * kUnitTiles - 1) / (kTileKeys * kUnitTiles);
    return n > 0 ? n : 1;
  }
  __device__ __forceinline__ void clip() {
    const int64_t r1 = s.r0 + (end - u);
    s.r1 = r1 < s.units ? static_cast<int>(r1) : s.units;
  }
  // The next segment of the share; false when there is none.
  __device__ __forceinline__ bool next(const DecodeParams& p) {
    u += s.r1 - s.r0;
    if (u >= end) return false;
    if (++s.j == p.c.heads * p.head_blocks) {
      s.j = 0;
      ++s.b;
      s.len = paged_length(p.c.kv_len[s.b], p.c.max_pages, p.c.page_shift);
      s.units = units_of(p, s.len);
    }
    s.r0 = 0;
    clip();
    return true;
  }
  // One past the last tile of the segment that holds a key.
  __device__ __forceinline__ int tile_end(const DecodeParams& p) const {
    return min(s.r1 * p.unit_tiles, (s.len + kTileKeys - 1) / kTileKeys);
  }
};

// This CTA's share, from the lengths: every thread sums a run of sequences, a
// block scan places the runs, and the thread whose run holds the first unit
// finds the sequence in it. False when the CTA has no share.
__device__ bool find_share(const DecodeParams& p, Walk* w, ShareCut* share) {
  __shared__ int64_t warp_sum[kWarps];
  __shared__ Walk found;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (p.c.batch + kThreads - 1) / kThreads;
  const int b0 = min(p.c.batch, static_cast<int>(threadIdx.x) * per), b1 = min(p.c.batch, b0 + per);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b)
    mine += Walk::units_of(p, paged_length(p.c.kv_len[b], p.c.max_pages, p.c.page_shift));
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
  const ShareCut cut = share_cut(W, W < gridDim.x ? static_cast<int>(W) : static_cast<int>(gridDim.x));
  *share = cut;
  if (blockIdx.x >= cut.count) return false;
  const int64_t first = share_begin(cut, blockIdx.x), last = share_begin(cut, blockIdx.x + 1);
  if (first >= before * per_seq && first < (before + mine) * per_seq) {
    int64_t at = before * per_seq;
    for (int b = b0; b < b1; ++b) {
      const int len = paged_length(p.c.kv_len[b], p.c.max_pages, p.c.page_shift);
      const int units = Walk::units_of(p, len);
      if (first < at + static_cast<int64_t>(units) * per_seq) {
        Walk f;
        f.s.b = b;
        f.s.j = small_quotient(first - at, units);
        f.s.len = len;
        f.s.units = units;
        f.s.r0 = static_cast<int>((first - at) - static_cast<int64_t>(f.s.j) * units);
        f.s.r1 = 0;
        f.u = first;
        f.end = last;
        f.clip();
        found = f;
        break;
      }
      at += static_cast<int64_t>(units) * per_seq;
    }
  }
  __syncthreads();
  *w = found;
  return true;
}

// NT: blocks of 8 query heads.
template <bool kF16, int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_paged_kernel(const DecodeParams p) {
  using S = Shape<D>;
  constexpr int kChunks = D / 8;              // 16-byte chunks of a row
  constexpr int kRowsPerCopy = 32 / kChunks;  // rows a warp's copy instruction covers
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float merge_m[kWarps][8], merge_l[kWarps][8];
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane & 3, row8 = lane >> 2;

  Walk w;
  ShareCut share;
  const bool has_share = find_share(p, &w, &share);
  if (threadIdx.x == 0) p.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (!has_share) return;

  const uint32_t ring = smem_u32(smem) + warp * kStages * S::kStageBytes;
  float* merge = reinterpret_cast<float*>(smem + S::kRingBytes);
  const int copy_row = lane / kChunks, copy_chunk = lane % kChunks;

  // ---- the loads' cursor: the tile to be loaded next, and its page
  Walk lw = w;
  int lt = lw.s.r0 * p.unit_tiles + warp;
  bool more = true;
  int page = 0;
  auto settle = [&]() {  // move to the next tile that exists, fetch its page number
    while (lt >= lw.tile_end(p)) {
      if (!(more = lw.next(p))) return;
      lt = lw.s.r0 * p.unit_tiles + warp;
    }
    page = p.c.table[static_cast<int64_t>(lw.s.b) * p.c.ld_table + ((lt * kTileKeys) >> p.c.page_shift)];
  };
  uint32_t bad = 0;  // stages whose tile has a page outside the pool
  auto load = [&](int stage) {
    if (more) {
      const int key0 = lt * kTileKeys;
      const bool ok = page_ok(page, p.c.num_pages);
      if (!ok) report_error(p.err, kKernelPaged | (kSiteBadPage << 8));
      bad = (bad & ~(1u << stage)) | (ok ? 0u : 1u << stage);
      const int g = lw.s.j / p.head_blocks;
      const int64_t at = ok ? pool_offset(page, g, (key0 & ((1 << p.c.page_shift) - 1)) + copy_row, p.c.ld_page,
                                          p.c.ld_head, p.c.ld_slot) + copy_chunk * 8
                            : 0;
      const int rows = ok ? lw.s.len - key0 : 0;  // rows of the tile that hold a token
      const uint32_t dst = ring + stage * S::kStageBytes;
#pragma unroll
      for (int i = 0; i < kTileKeys / kRowsPerCopy; ++i) {
        const int r = i * kRowsPerCopy + copy_row;
        const bool there = r < rows;
        const int64_t src = there ? at + i * kRowsPerCopy * p.c.ld_slot : 0;
        const uint32_t d = dst + r * S::kRowBytes + ((copy_chunk ^ (r & 7)) << 4);
        copy16(d, p.c.k + src, there);
        copy16(d + S::kTileBytes, p.c.v + src, there);
      }
      lt += kUnitTiles;
      settle();
    }
    copy_commit();
  };
  settle();
#pragma unroll 1
  for (int i = 0; i < kStages; ++i) load(i);

  int stage = 0;
  bool go = true;
  while (go) {
    const Segment s = w.s;
    const int g = s.j / p.head_blocks, hb = s.j - g * p.head_blocks;
    const int head0 = g * p.group + hb * p.block_heads;          // first query head of the block
    const int heads = min(p.block_heads, p.group - hb * p.block_heads);
    // Q^T fragments: head row8 of each 8, dims 16 kk + 2 quad + {0, 1} and 8 more
    uint32_t qf[NT][D / 16][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool live = nt * 8 + row8 < heads;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          p.q + s.b * p.ld_q_batch + static_cast<int64_t>(live ? head0 + nt * 8 + row8 : 0) * p.ld_q_head);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[nt][kk][0] = live ? src[8 * kk + quad] : 0u;
        qf[nt][kk][1] = live ? src[8 * kk + 4 + quad] : 0u;
      }
    }
    float m[NT][2], l[NT][2];   // heads 8 nt + 2 quad + {0, 1}; l: this thread's keys
    float od[NT][D / 16][4];    // dims 16 i + row8 (+ 8), the same heads
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = neg_inf();
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) od[nt][i][e] = 0.f;
    }
    const int t_end = w.tile_end(p);
    for (int t = s.r0 * p.unit_tiles + warp; t < t_end; t += kUnitTiles) {
      copy_wait<kStages - 1>();
      __syncwarp();
      const uint32_t kt = ring + stage * S::kStageBytes, vt = kt + S::kTileBytes;
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t a[4];
        const int r = lane & 15, ch = 2 * kk + (lane >> 4);
        ldmatrix4(a, kt + r * S::kRowBytes + ((ch ^ (r & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816<kF16>(sc[nt], a, qf[nt][kk][0], qf[nt][kk][1]);
      }
      const int key = t * kTileKeys + row8;
      const bool masked = (bad >> stage) & 1u;
      const bool live_a = key < s.len && !masked, live_b = key + 8 < s.len && !masked;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[nt][e] = live_a ? sc[nt][e] * p.scale2 : neg_inf();
          sc[nt][e + 2] = live_b ? sc[nt][e + 2] * p.scale2 : neg_inf();
          mx[nt][e] = fmaxf(sc[nt][e], sc[nt][e + 2]);
        }
      }
      if (p.scores) {
        const int64_t cap = static_cast<int64_t>(p.c.max_pages) << p.c.page_shift;
        float* out = p.scores + ((static_cast<int64_t>(s.b) * p.c.heads * p.head_blocks + s.j) * cap + key) * p.score_heads + 2 * quad;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (8 * nt + 2 * quad >= p.score_heads) continue;
          if (key < s.len) *reinterpret_cast<float2*>(out + nt * 8) = make_float2(sc[nt][0], sc[nt][1]);
          if (key + 8 < s.len)
            *reinterpret_cast<float2*>(out + 8 * p.score_heads + nt * 8) = make_float2(sc[nt][2], sc[nt][3]);
        }
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], off));
      bool rise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) rise |= mx[nt][0] > m[nt][0] + kSlack || mx[nt][1] > m[nt][1] + kSlack;
      if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float corr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float to = fmaxf(m[nt][e], mx[nt][e]);
            corr[e] = to == neg_inf() ? 1.f : ex2(m[nt][e] - to);
            m[nt][e] = to;
            l[nt][e] *= corr[e];
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) od[nt][i][e] *= corr[e & 1];
        }
      }
      uint32_t pf[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pe[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pe[e] = ex2(sc[nt][e] - reference(m[nt][e & 1]));
        }
        l[nt][0] += pe[0] + pe[2];
        l[nt][1] += pe[1] + pe[3];
        pf[nt][0] = transpose8x8(pack2<kF16>(pe[0], pe[1]));
        pf[nt][1] = transpose8x8(pack2<kF16>(pe[2], pe[3]));
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t a[4];
        const int r = (lane & 7) + ((lane >> 4) << 3), ch = 2 * i + ((lane >> 3) & 1);
        ldmatrix4_trans(a, vt + r * S::kRowBytes + ((ch ^ (r & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816<kF16>(od[nt][i], a, pf[nt][0], pf[nt][1]);
      }
      __syncwarp();
      load(stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    // ---- the four warps' states, 8 heads at a time
    const bool whole = s.r0 == 0 && s.r1 == s.units;
    const int slot = 2 * blockIdx.x + (s.r0 == 0 ? 1 : 0);
    if (s.r0 == 0 && threadIdx.x == 0) {
      int parts = 1;
      if (!whole) {
        // the item's last unit lies in the last of its shares
        parts = static_cast<int>(last_boundary(share, w.u + s.units - 1) - blockIdx.x) + 1;
        p.meta[blockIdx.x] = make_int4(s.b, s.j, parts, slot);
      }
      if (p.scores)
        p.item_meta[static_cast<int64_t>(s.b) * p.c.heads * p.head_blocks + s.j] = make_int2(blockIdx.x, parts);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int e = 0; e < 2; ++e) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
      float* mine = merge + warp * 8 * S::kMergeLd;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(2 * quad + (e & 1)) * S::kMergeLd + 16 * i + row8 + (e >> 1) * 8] = od[nt][i][e];
      if (row8 == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          merge_m[warp][2 * quad + e] = m[nt][e];
          merge_l[warp][2 * quad + e] = l[nt][e];
        }
      }
      __syncthreads();
      // thread: head threadIdx.x / 16 of the 8, D / 16 dims
      constexpr int kDims = D / 16;
      const int hh = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * kDims;
      if (nt * 8 + hh < heads) {
        float M = neg_inf(), L = 0.f, acc[kDims];
#pragma unroll
        for (int i = 0; i < kWarps; ++i) M = fmaxf(M, merge_m[i][hh]);
#pragma unroll
        for (int k = 0; k < kDims; ++k) acc[k] = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float f = ex2(merge_m[i][hh] - reference(M));
          L = fmaf(merge_l[i][hh], f, L);
          const float4* src = reinterpret_cast<const float4*>(merge + (i * 8 + hh) * S::kMergeLd + d0);
#pragma unroll
          for (int k = 0; k < kDims / 4; ++k) {
            const float4 x = src[k];
            acc[4 * k] = fmaf(x.x, f, acc[4 * k]);
            acc[4 * k + 1] = fmaf(x.y, f, acc[4 * k + 1]);
            acc[4 * k + 2] = fmaf(x.z, f, acc[4 * k + 2]);
            acc[4 * k + 3] = fmaf(x.w, f, acc[4 * k + 3]);
          }
        }
        const int h = head0 + nt * 8 + hh;
        const int64_t row = static_cast<int64_t>(s.b) * p.H + h;
        if (whole) {
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
          const int64_t at = static_cast<int64_t>(slot) * p.block_heads + nt * 8 + hh;
          float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + d0);
#pragma unroll
          for (int k = 0; k < kDims / 4; ++k)
            dst[k] = make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
          if ((threadIdx.x & 15) == 0) p.part_ml[at] = make_float2(M, L);
        }
      }
      __syncthreads();
    }
    go = w.next(p);
  }
  copy_wait<0>();
}

// The second kernel. With weights, its first CTAs add up: kAddKeys keys of one key
// head each. The others join: CTA (c, hh) merges head hh of the item that begins
// in share c and goes on into the next ones; its warps take the parts in turn.
constexpr int kFinishThreads = 256;
constexpr int kFinishWarps = kFinishThreads / 32;
constexpr int kAddKeysPerThread = 4;
constexpr int kAddKeys = kAddKeysPerThread * kFinishThreads;

// Slot of part i of an item that begins in share c: part 0 in 2 c + 1, part i > 0 in 2 (c + i).
__device__ __forceinline__ int64_t part_slot(int c, int i) {
  return 2 * (static_cast<int64_t>(c) + i) + (i == 0 ? 1 : 0);
}

template <bool kF16, int D>
__device__ __forceinline__ void join_head(const DecodeParams& p, int share, int hh) {
  constexpr int kDims = D / 32;
  __shared__ float sm[kFinishWarps], sl[kFinishWarps], so[kFinishWarps][D];
  const int4 meta = p.meta[share];
  const int parts = meta.z;
  if (parts == 0) return;
  const int g = meta.y / p.head_blocks, hb = meta.y - g * p.head_blocks;
  if (hh >= min(p.block_heads, p.group - hb * p.block_heads)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float M = neg_inf(), L = 0.f, acc[kDims];
#pragma unroll
  for (int k = 0; k < kDims; ++k) acc[k] = 0.f;
  constexpr int kBatch = 4;
  for (int i0 = warp; i0 < parts; i0 += kFinishWarps * kBatch) {
    float2 ml[kBatch];
    float x[kBatch][kDims];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kFinishWarps;
      ml[u] = make_float2(neg_inf(), 0.f);
#pragma unroll
      for (int k = 0; k < kDims; ++k) x[u][k] = 0.f;
      if (i < parts) {
        const int64_t at = part_slot(share, i) * p.block_heads + hh;
        ml[u] = p.part_ml[at];
#pragma unroll
        for (int k = 0; k < kDims; ++k) x[u][k] = p.part_o[at * D + lane + 32 * k];
      }
    }
    float to = M;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) to = fmaxf(to, ml[u].x);
    const float ref = reference(to), corr = ex2(M - ref);
    M = to;
    L *= corr;
#pragma unroll
    for (int k = 0; k < kDims; ++k) acc[k] *= corr;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float f = ex2(ml[u].x - ref);
      L = fmaf(ml[u].y, f, L);
#pragma unroll
      for (int k = 0; k < kDims; ++k) acc[k] = fmaf(x[u][k], f, acc[k]);
    }
  }
  if (lane == 0) {
    sm[warp] = M;
    sl[warp] = L;
  }
#pragma unroll
  for (int k = 0; k < kDims; ++k) so[warp][lane + 32 * k] = acc[k];
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  M = neg_inf();
  L = 0.f;
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int i = 0; i < kFinishWarps; ++i) M = fmaxf(M, sm[i]);
#pragma unroll
  for (int i = 0; i < kFinishWarps; ++i) {
    const float f = ex2(sm[i] - reference(M));
    L = fmaf(sl[i], f, L);
    a = fmaf(so[i][2 * threadIdx.x], f, a);
    b = fmaf(so[i][2 * threadIdx.x + 1], f, b);
  }
  const int64_t row = static_cast<int64_t>(meta.x) * p.H + g * p.group + hb * p.block_heads + hh;
  const float inv = L != 0.f ? 1.f / L : 0.f;
  reinterpret_cast<uint32_t*>(p.o + row * D)[threadIdx.x] = pack2<kF16>(a * inv, b * inv);
  if (threadIdx.x == 0 && p.lse) p.lse[row] = L != 0.f ? (M + log2f(L)) * kLn2 : neg_inf();
}

// weights[b, g, t] += sum over the group's heads of 2^(s - lse). Each key's sum
// has one thread and a fixed order. A cut item's lse is formed here from its
// parts, so that this does not wait for the join; the scores are on their way
// meanwhile.
__device__ __forceinline__ void add_weights(const DecodeParams& p, int b, int g, int chunk, float* __restrict__ weights) {
  __shared__ float lse2[kMaxHeadBlock];
  // (the lengths too may come from a kernel that still runs, one before the first
  // kernel: an eviction writes them)
  wait_for_previous_kernel();
  const int len = paged_length(p.c.kv_len[b], p.c.max_pages, p.c.page_shift);
  const int t0 = chunk * kAddKeys + threadIdx.x;
  if (chunk * kAddKeys >= len) return;
  const int64_t cap = static_cast<int64_t>(p.c.max_pages) << p.c.page_shift;
  float was[kAddKeysPerThread], sum[kAddKeysPerThread];
#pragma unroll
  for (int i = 0; i < kAddKeysPerThread; ++i) {
    const int t = t0 + i * kFinishThreads;
    was[i] = t < len ? weights[t] : 0.f;
    sum[i] = 0.f;
  }
  for (int hb = 0; hb < p.head_blocks; ++hb) {
    const int64_t item = (static_cast<int64_t>(b) * p.c.heads + g) * p.head_blocks + hb;
    const int heads = min(p.block_heads, p.group - hb * p.block_heads);
    const float* s = p.scores + item * cap * p.score_heads;
    if (hb > 0) __syncthreads();
    for (int h = 0; h < heads; h += 4) {
      float4 x[kAddKeysPerThread];
#pragma unroll
      for (int i = 0; i < kAddKeysPerThread; ++i) {
        const int64_t t = t0 + i * kFinishThreads;
        x[i] = t < len ? *reinterpret_cast<const float4*>(s + t * p.score_heads + h)
                       : make_float4(neg_inf(), neg_inf(), neg_inf(), neg_inf());
      }
      if (h == 0) {
        if (threadIdx.x < heads) {
          const int2 meta = p.item_meta[item];
          float e2 = neg_inf();
          if (meta.y == 1) {
            e2 = p.lse2[static_cast<int64_t>(b) * p.H + g * p.group + hb * p.block_heads + threadIdx.x];
          } else {
            float M = neg_inf(), L = 0.f;
            for (int i = 0; i < meta.y; ++i) {
              const float2 ml = p.part_ml[part_slot(meta.x, i) * p.block_heads + threadIdx.x];
              const float to = fmaxf(M, ml.x), ref = reference(to);
              L = fmaf(L, ex2(M - ref), ml.y * ex2(ml.x - ref));
              M = to;
            }
            if (L != 0.f) e2 = M + log2f(L);
          }
          lse2[threadIdx.x] = e2;
        }
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < kAddKeysPerThread; ++i) {
        const float v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (h + e < heads && v[e] != neg_inf()) sum[i] += ex2(v[e] - lse2[h + e]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kAddKeysPerThread; ++i) {
    const int t = t0 + i * kFinishThreads;
    if (t < len) weights[t] = was[i] + sum[i];
  }
}

template <bool kF16, int D>
__global__ void __launch_bounds__(kFinishThreads)
decode_finish_kernel(const DecodeParams p, int adds, int chunks, float* weights, int64_t ld_w_batch, int64_t ld_w_head) {
  let_next_kernel_start();
  int i = blockIdx.x;
  if (i < adds) {
    const int chunk = i % chunks, row = i / chunks;
    const int g = row % p.c.heads, b = row / p.c.heads;
    add_weights(p, b, g, chunk, weights + b * ld_w_batch + g * ld_w_head);
    return;
  }
  i -= adds;
  wait_for_previous_kernel();
  join_head<kF16, D>(p, i / p.block_heads, i % p.block_heads);
}

// Layout of the workspace, the same for its size and its use.
struct Plan {
  int shares, block_heads, head_blocks, score_heads;
  bool whole;  // items are not cut
  int64_t part_o, part_ml, meta, lse2, item_meta, scores, bytes;  // offsets, then the size
};

bool make_plan(int H, const os_paged_cache& c, bool weights, Plan* out) {
  const int sms = device_sms();
  if (sms < 1) return false;
  const int group = H / c.heads;
  Plan pl;
  pl.shares = sms * kCtasPerSm;
  pl.block_heads = group <= 8 ? 8 : kMaxHeadBlock;
  pl.head_blocks = (group + pl.block_heads - 1) / pl.block_heads;
  pl.score_heads = pl.head_blocks > 1 ? pl.block_heads : (group + 3) / 4 * 4;
  const int64_t capacity = static_cast<int64_t>(c.max_pages) * c.page_size;
  const int64_t items = static_cast<int64_t>(c.batch) * c.heads * pl.head_blocks;
  pl.whole = capacity <= kWholeKeys || (capacity <= kWholeKeysMany && items >= pl.shares);
  int64_t at = 0;
  auto take = [&](int64_t n) {
    const int64_t here = at;
    at += (n + 255) / 256 * 256;
    return here;
  };
  pl.part_o = take(static_cast<int64_t>(2) * pl.shares * pl.block_heads * c.head_dim * 4);
  pl.part_ml = take(static_cast<int64_t>(2) * pl.shares * pl.block_heads * 8);
  pl.meta = take(static_cast<int64_t>(pl.shares) * 16);
  pl.lse2 = pl.item_meta = pl.scores = 0;
  if (weights) {
    pl.lse2 = take(static_cast<int64_t>(c.batch) * H * 4);
    pl.item_meta = take(static_cast<int64_t>(c.batch) * c.heads * pl.head_blocks * 8);
    pl.scores = take(static_cast<int64_t>(c.batch) * c.heads * pl.head_blocks * c.max_pages * c.page_size *
                     pl.score_heads * 4);
  }
  pl.bytes = at;
  *out = pl;
  return true;
}

template <bool kF16, int D, int NT>
cudaError_t launch_shape(const DecodeParams& p, int shares, float* weights, int64_t ld_w_batch, int64_t ld_w_head,
                         cudaStream_t stream) {
  constexpr int smem = Shape<D>::kSmemBytes;
  // the kernel's shared-memory limit, raised once per device
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> smem_set[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !smem_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(decode_paged_kernel<kF16, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) smem_set[dev].store(true, std::memory_order_release);
  }
  if ((e = launch_after(decode_paged_kernel<kF16, D, NT>, dim3(shares), kThreads, smem, stream, p)) != cudaSuccess) return e;
  const int64_t joins = p.unit_tiles == kUnitTiles ? static_cast<int64_t>(shares) * p.block_heads : 0;
  const int64_t chunks = weights ? ((static_cast<int64_t>(p.c.max_pages) << p.c.page_shift) + kAddKeys - 1) / kAddKeys : 0;
  const int64_t adds = chunks * p.c.heads * p.c.batch, ctas = adds + joins;
  if (ctas > 0x7fffffff) return cudaErrorNotSupported;
  if (ctas == 0) return cudaSuccess;
  return launch_after(decode_finish_kernel<kF16, D>, dim3(static_cast<unsigned>(ctas)), kFinishThreads, 0, stream, p,
                      static_cast<int>(adds), static_cast<int>(chunks), weights, ld_w_batch, ld_w_head);
}

template <bool kF16, int D>
cudaError_t launch_heads(const DecodeParams& p, int shares, float* weights, int64_t ld_w_batch, int64_t ld_w_head,
                         cudaStream_t stream) {
  return p.block_heads == 8 ? launch_shape<kF16, D, 1>(p, shares, weights, ld_w_batch, ld_w_head, stream)
                            : launch_shape<kF16, D, 2>(p, shares, weights, ld_w_batch, ld_w_head, stream);
}

}  // namespace

int64_t decode_paged_workspace_bytes(int H, const os_paged_cache& cache, bool weights) {
  Plan pl;
  return make_plan(H, cache, weights, &pl) ? pl.bytes : -1;
}

cudaError_t launch_decode_paged(const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head, int H,
                                const os_paged_cache& cache, float scale, uint16_t* o, float* lse,
                                float* weights, int64_t ld_w_batch, int64_t ld_w_head,
                                void* workspace, unsigned int* err, cudaStream_t stream) {
  Plan pl;
  if (!make_plan(H, cache, weights != nullptr, &pl)) return cudaErrorInvalidDevice;
  char* ws = static_cast<char*>(workspace);
  DecodeParams p;
  p.c = paged_cache(cache);
  p.q = q;
  p.ld_q_batch = ld_q_batch;
  p.ld_q_head = ld_q_head;
  p.H = H;
  p.group = H / cache.heads;
  p.head_blocks = pl.head_blocks;
  p.block_heads = pl.block_heads;
  p.unit_tiles = pl.whole ? kWholeKeysMany / kTileKeys : kUnitTiles;
  p.score_heads = pl.score_heads;
  p.scale2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  p.o = o;
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_ml);
  p.meta = reinterpret_cast<int4*>(ws + pl.meta);
  p.lse2 = reinterpret_cast<float*>(ws + pl.lse2);
  p.item_meta = reinterpret_cast<int2*>(ws + pl.item_meta);
  p.scores = weights ? reinterpret_cast<float*>(ws + pl.scores) : nullptr;
  p.err = err;
  const bool f16 = cache.dtype == OS_DTYPE_F16;
  if (cache.head_dim == 128)
    return f16 ? launch_heads<true, 128>(p, pl.shares, weights, ld_w_batch, ld_w_head, stream)
               : launch_heads<false, 128>(p, pl.shares, weights, ld_w_batch, ld_w_head, stream);
  return f16 ? launch_heads<true, 64>(p, pl.shares, weights, ld_w_batch, ld_w_head, stream)
             : launch_heads<false, 64>(p, pl.shares, weights, ld_w_batch, ld_w_head, stream);
}

}  // namespace oss
