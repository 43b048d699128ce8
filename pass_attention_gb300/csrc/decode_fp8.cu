// Attention of one new token per sequence over a paged key-value cache in 8 bits.
//
//   s_t = scale 2^ek_t q.kcode_t;  lse = ln sum exp s_t;  o = sum exp(s_t - lse) 2^ev_t vcode_t
//
// The walk, the division of the work and the join are those of the 16-bit decode
// (decode_paged.cu). What differs:
//
// Products. Codes are exact in fp16 (4 significant bits, 2^-9 to 448), so both products
// run as fp16 mma.sync with fp32 sums, whatever the type of q and o. (An e4m3 MMA would want q
// and the weights in 8 bits.) A bf16 q is brought into fp16's range by a power of two per
// head: its largest element comes to 2^15 .. 2^16 (255/128 2^15 at most, fp16 ends at 2047/1024 2^15). All
// 8 bits of an element then fit down to 2^-17, 2^-32 of the largest; below that it is off by up to 2^-25,
// half of fp16's least step and 2^-40 of the largest.
//
// Scales. The key's is a factor on the score. The value's goes into the weight's
// exponent, 2^(s + ev - m'), so V needs no multiplication. Weights of values far larger
// than others would leave fp16's range if they were taken relative to the largest score
// alone; so O has a reference of its own, m' = max (s + ev), and l keeps m = max s: two
// exponentials a score. Where warps and parts meet, O comes to m.
//
// Fragments. ldmatrix moves 16-bit elements, here pairs of codes. A K register holds
// four consecutive dims of a key; the MMA's k index is permuted to fit (dims 4 q, 4 q + 1 in
// its columns 2 q, 2 q + 1, and 4 q + 2, 4 q + 3 in 2 q + 8, 2 q + 9), and q's fragments
// likewise. A transposed V register holds two dims of two keys; a byte permutation
// sorts them by dim, and rows r and r + 8 of the MMA are dims 2 r and 2 r + 1.
//
// What bounds it: HBM, at half the bytes of the 16-bit decode, so a tile may take half the
// time: 711 cycles of a scheduler for 16 keys of 128. It takes about 344 instructions (436
// with addresses formed anew for every tile, masks and guards in every weight), so three CTAs
// an SM (two: 129 against 116 us at that point) and the next tile's products beside this one's
// softmax (106.5 -> 104.5). 64 sequences of up to 8192 tokens, 32 heads over 8: 102 us (6.0 TB/s, 0.90 of
// the copy peak, 6 us of it the launch's beginning and end); 6 of up to 32768, 16 heads of 64 in
// fp16: 58 us (0.85: instructions; a tile there has 32 keys, 7 us more with 16); one of 777 tokens
// 7.2 us from a graph. Groups of 9 to 16 heads (236 registers, two CTAs an SM) wait for their instructions'
// latencies, not for HBM: 64 of up to 8192, 128 heads over 8, 145 us where 32 over 8 take 92 (16-bit: 218 and 178).

#include <atomic>
#include <cstdint>

#include "decode_paged.cuh"
#include "device_common.cuh"
#include "fp8.cuh"
#include "launch.cuh"
#include "oss_internal.h"

namespace oss {
namespace {

using namespace decode;

constexpr int ctas_per_sm(int NT) { return NT == 1 ? 3 : 2; }

template <int D, int NT>
struct Shape {
  static constexpr int kCtas = ctas_per_sm(NT);
  static constexpr int kSub = 128 / D;               // blocks of 16 keys in a tile: 4 KB of K and V either way
  static constexpr int kKeys = 16 * kSub;
  static constexpr int kStages = kCtas == 2 ? 5 : 2 + kSub;  // what fits beside the merge buffer
  static constexpr int kBlockBytes = 16 * D;         // 16 rows of K or V
  static constexpr int kTileBytes = kKeys * D;       // K or V of a tile
  static constexpr int kScaleBytes = 2 * kKeys;      // K's, then V's
  static constexpr int kRingBytes = kWarps * kStages * 2 * kTileBytes;
  static constexpr int kScaleRing = kWarps * kStages * kScaleBytes;
  static constexpr int kSmemBytes = kRingBytes + kScaleRing + kMergeBytes<D>;
};

// The references before the first key: below every finite score, so that no weight needs
// a special case (-inf - kNone is -inf still).
constexpr float kNone = -3.402823466e+38f;

// A score is its sum times one factor, of the query's and the key's powers of two: a large query over
// small keys would leave fp32's range between them. Where the factor itself does, every sum
// but 0 is far beyond it too, and 0 is to stay 0. (NaN stays NaN.)
__device__ __forceinline__ float finite(float x) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(3.402823466e+38f));
  return y;
}

// Byte offset of 16-byte chunk c of row r of a tile, so that eight rows of a chunk
// touch all banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return r * D + ((c ^ (D == 128 ? r & 7 : (r >> 1) & 3)) << 4);
}

// NT: blocks of 8 query heads.
template <bool kF16, int D, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT)) decode_fp8_kernel(const DecodeParams p, const Fp8Pools f) {
  using S = Shape<D, NT>;
  constexpr int kChunks = D / 16;             // 16-byte chunks of a row
  constexpr int kRowsPerCopy = 32 / kChunks;  // rows a warp's copy instruction covers
  constexpr int kStages = S::kStages, kSub = S::kSub;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float merge_m[kWarps][8], merge_l[kWarps][8];
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane & 3, row8 = lane >> 2;

  Walk<S::kKeys, kWeighed> w;
  ShareCut share;
  const bool has_share = find_share(p, &w, &share);
  if (threadIdx.x == 0) p.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (!has_share) return;

  const uint32_t ring = smem_u32(smem) + warp * kStages * 2 * S::kTileBytes;
  const uint8_t* scale_ring = smem + S::kRingBytes + warp * kStages * S::kScaleBytes;
  float* merge = reinterpret_cast<float*>(smem + S::kRingBytes + S::kScaleRing);
  const int copy_row = lane / kChunks, copy_chunk = lane % kChunks;

  // ---- the loads' cursor: the tile to be loaded next and its page, and what of its
  // address the segment decides
  Walk<S::kKeys, kWeighed> lw = w;
  int lt, lt_end;
  bool more = true;
  int page[kSub];
  const int32_t* row;
  int64_t head_at, scale_at;
  const int64_t lane_at = copy_row * p.c.ld_slot + copy_chunk * 16, copy_step = kRowsPerCopy * p.c.ld_slot;
  const int slot_mask = (1 << p.c.page_shift) - 1;
  auto enter = [&]() {
    const int g = lw.s.j / p.head_blocks;
    lt = lw.s.r0 * p.unit_tiles + warp;
    lt_end = lw.tile_end(p);
    row = p.c.table + static_cast<int64_t>(lw.s.b) * p.c.ld_table;
    head_at = g * p.c.ld_head + lane_at;
    scale_at = g * f.ld_head;
  };
  auto settle = [&]() {  // move to the next tile that exists, fetch its page number
    while (lt >= lt_end) {
      if (!(more = lw.next(p))) return;
      enter();
    }
#pragma unroll
    for (int b = 0; b < kSub; ++b) {
      const int key = lt * S::kKeys + 16 * b;
      page[b] = b == 0 || key < lw.s.len ? row[key >> p.c.page_shift] : 0;
    }
  };
  uint32_t bad = 0;  // a bit for every block of every stage: its page is outside the pool
  auto load = [&](int stage) {
    if (more) {
#pragma unroll
      for (int b = 0; b < kSub; ++b) {
        const int key0 = lt * S::kKeys + 16 * b, slot0 = key0 & slot_mask;
        const int rows = lw.s.len - key0;  // rows of the block that hold a token
        const uint32_t dst = ring + stage * 2 * S::kTileBytes + b * S::kBlockBytes + chunk_at<D>(copy_row, copy_chunk);
        const uint32_t sc = smem_u32(scale_ring) + stage * S::kScaleBytes + lane * S::kKeys + 16 * b;
        const uint32_t bit = 1u << (stage * kSub + b);
        // (rows kRowsPerCopy apart have the same swizzle but in D 128's second four of eight)
        auto at_copy = [&](int i) { return D == 128 && (i & 1) ? (dst ^ 64) + i * kRowsPerCopy * D : dst + i * kRowsPerCopy * D; };
        bad &= ~bit;
        if (page_ok(page[b], p.c.num_pages) && rows > 0) {
          const int64_t at = static_cast<int64_t>(page[b]) * p.c.ld_page + head_at + slot0 * p.c.ld_slot;
          const uint8_t *k = f.k + at, *v = f.v + at;
          if (rows >= 16) {
#pragma unroll
            for (int i = 0; i < 16 / kRowsPerCopy; ++i, k += copy_step, v += copy_step) {
              copy16(at_copy(i), k);
              copy16(at_copy(i) + S::kTileBytes, v);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16 / kRowsPerCopy; ++i) {
              const bool there = i * kRowsPerCopy + copy_row < rows;
              copy16(at_copy(i), there ? k + i * copy_step : f.k, there);
              copy16(at_copy(i) + S::kTileBytes, there ? v + i * copy_step : f.v, there);
            }
          }
          if (lane < 2) copy16(sc, (lane ? f.v_scales : f.k_scales) + page[b] * f.ld_page + scale_at + slot0);
        } else {
          if (rows > 0) {
            report_error(p.err, kKernelPaged | (kSiteBadPage << 8));
            bad |= bit;
          }
#pragma unroll
          for (int i = 0; i < 16 / kRowsPerCopy; ++i) {
            copy16(at_copy(i), f.k, false);
            copy16(at_copy(i) + S::kTileBytes, f.v, false);
          }
          if (lane < 2) copy16(sc, f.k_scales, false);
        }
      }
      lt += kUnitTiles;
      settle();
    }
    copy_commit();
  };
  enter();
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
    // Q^T fragments in fp16: head row8 of each 8, dims 16 kk + 4 quad + {0, 1} and {2, 3}
    uint32_t qf[NT][D / 16][2];
    float qs[NT][2];  // factors of the scores of heads 8 nt + 2 quad + {0, 1}
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool live = nt * 8 + row8 < heads;
      const uint2* src = reinterpret_cast<const uint2*>(
          p.q + s.b * p.ld_q_batch + static_cast<int64_t>(live ? head0 + nt * 8 + row8 : 0) * p.ld_q_head);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint2 x = live ? src[4 * kk + quad] : make_uint2(0u, 0u);
        qf[nt][kk][0] = x.x;
        qf[nt][kk][1] = x.y;
      }
      float up = 1.f;
      if constexpr (!kF16) {
        uint32_t top = 0;  // the head's largest magnitude
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e) top = __vmaxu2(top, qf[nt][kk][e] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // exponent field n of the largest: times 2^(127 + 15 - n); NaN, infinity and 0 as
        // they are, and below 2^-100 no further up than from there
        const uint32_t n = max(top >> 7, 27u);
        const bool plain = top >= 0x7f80u;
        const float to = plain ? 1.f : __uint_as_float((127u + 127u + 15u - n) << 23);
        up = plain ? 1.f : __uint_as_float((n - 15u) << 23);  // 1 / to
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 x = widen2<false>(qf[nt][kk][e]);
            qf[nt][kk][e] = pack2<true>(x.x * to, x.y * to);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) qs[nt][e] = __shfl_sync(0xffffffffu, up, (2 * quad + e) * 4) * p.scale2;
    }
    float m[NT][2], l[NT][2];   // heads 8 nt + 2 quad + {0, 1}; l: this thread's keys
    float mo[NT][2];            // O's reference
    float od[NT][D / 16][4];    // dims 16 i + 2 row8 (+ 1), the same heads
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = mo[nt][0] = mo[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) od[nt][i][e] = 0.f;
    }
    const int t_end = w.tile_end(p);
    // scores of the tile in a stage, before their factors; two sums: even and odd dims' chunks
    using Sums = float[kSub][NT][2][4];
    auto products = [&](int st, Sums& sc) {
      const uint32_t kt = ring + st * 2 * S::kTileBytes;
#pragma unroll
      for (int b = 0; b < kSub; ++b) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[b][nt][0][e] = sc[b][nt][1][e] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[4];
          ldmatrix4(x, kt + b * S::kBlockBytes + chunk_at<D>(lane & 15, 2 * c + (lane >> 4)));
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t a[4] = {from_e4m3x2(x[2 * half]), from_e4m3x2(x[2 * half + 1]), from_e4m3x2(x[2 * half] >> 16),
                                   from_e4m3x2(x[2 * half + 1] >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<true>(sc[b][nt][half], a, qf[nt][2 * c + half][0], qf[nt][2 * c + half][1]);
          }
        }
      }
    };
    Sums sc;
    int t = s.r0 * p.unit_tiles + warp;
    if (t < t_end) {
      copy_wait<kStages - 1>();
      __syncwarp();
      products(stage, sc);
    }
    for (; t < t_end; t += kUnitTiles) {
      // the next tile's products beside this one's softmax (behind the segment's last
      // tile: of whatever lies in the next stage, for nothing)
      const int next_stage = stage + 1 == kStages ? 0 : stage + 1;
      Sums ahead;
      copy_wait<kStages - 2>();
      __syncwarp();
      products(next_stage, ahead);
      const uint32_t vt = ring + stage * 2 * S::kTileBytes + S::kTileBytes;
      // the keys' scales and the values' exponents, one to a lane: lanes 0 .. 15 and 16 .. 31
      // have those of one block, or all lanes both of two
      const uint8_t* bytes = scale_ring + stage * S::kScaleBytes + lane;
      const float ks = fp8_scale_value(bytes[0]);
      const uint32_t vb = bytes[kSub == 1 ? 0 : 32];
      const float ev = vb == kFp8ScaleNan ? __uint_as_float(0x7fffffffu) : __uint_as_float(0x4b000000u | vb) - 8388735.f;
      float x[kSub][NT][4], y[kSub][NT][4];  // scores in base 2, and with the value's exponent
      const int left = s.len - t * S::kKeys;  // keys from the tile's first one on
#pragma unroll
      for (int b = 0; b < kSub; ++b) {
        float kf[2], vf[2];  // of keys row8 and row8 + 8
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          kf[r] = __shfl_sync(0xffffffffu, ks, 16 * b + 8 * r + row8);
          vf[r] = __shfl_sync(0xffffffffu, ev, (kSub == 1 ? 16 : 16 * b) + 8 * r + row8);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[b][nt][e] = (sc[b][nt][0][e] + sc[b][nt][1][e]) * finite(qs[nt][e & 1] * kf[e >> 1]);
            y[b][nt][e] = x[b][nt][e] + vf[e >> 1];
          }
      }
      if (left < S::kKeys || bad) {  // some tile has a bad page, perhaps this one
#pragma unroll
        for (int b = 0; b < kSub; ++b) {
          const int live = (bad >> (stage * kSub + b)) & 1u ? 0 : left - 16 * b;  // the block's rows that hold a token
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (row8 + (e < 2 ? 0 : 8) >= live) x[b][nt][e] = y[b][nt][e] = neg_inf();
        }
      }
      float mx[NT][2], my[NT][2];  // this thread's largest
      bool rise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[nt][e] = fmaxf(x[0][nt][e], x[0][nt][e + 2]);
          my[nt][e] = fmaxf(y[0][nt][e], y[0][nt][e + 2]);
#pragma unroll
          for (int b = 1; b < kSub; ++b) {
            mx[nt][e] = fmaxf(mx[nt][e], fmaxf(x[b][nt][e], x[b][nt][e + 2]));
            my[nt][e] = fmaxf(my[nt][e], fmaxf(y[b][nt][e], y[b][nt][e + 2]));
          }
          rise |= mx[nt][e] > m[nt][e] + kSlack || my[nt][e] > mo[nt][e] + kSlack;
        }
      if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float corr[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              mx[nt][e] = fmaxf(mx[nt][e], __shfl_xor_sync(0xffffffffu, mx[nt][e], off));
              my[nt][e] = fmaxf(my[nt][e], __shfl_xor_sync(0xffffffffu, my[nt][e], off));
            }
            mx[nt][e] = fmaxf(mx[nt][e], m[nt][e]);
            my[nt][e] = fmaxf(my[nt][e], mo[nt][e]);
            l[nt][e] *= ex2(m[nt][e] - mx[nt][e]);
            corr[e] = ex2(mo[nt][e] - my[nt][e]);
            m[nt][e] = mx[nt][e];
            mo[nt][e] = my[nt][e];
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) od[nt][i][e] *= corr[e & 1];
        }
      }
      uint32_t pf[kSub][NT][2];
#pragma unroll
      for (int b = 0; b < kSub; ++b)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pe[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            l[nt][e & 1] += ex2(x[b][nt][e] - m[nt][e & 1]);
            pe[e] = ex2(y[b][nt][e] - mo[nt][e & 1]);
          }
          pf[b][nt][0] = transpose8x8(pack2<true>(pe[0], pe[1]));
          pf[b][nt][1] = transpose8x8(pack2<true>(pe[2], pe[3]));
        }
#pragma unroll
      for (int b = 0; b < kSub; ++b)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[4];
          ldmatrix4_trans(v, vt + b * S::kBlockBytes + chunk_at<D>(lane & 15, 2 * c + (lane >> 4)));
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // bytes {key, dim}: 00 01 10 11 -> 00 10 01 11
            const uint32_t lo = __byte_perm(v[2 * half], 0, 0x3120), hi = __byte_perm(v[2 * half + 1], 0, 0x3120);
            const uint32_t a[4] = {from_e4m3x2(lo), from_e4m3x2(lo >> 16), from_e4m3x2(hi), from_e4m3x2(hi >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<true>(od[nt][2 * c + half], a, pf[b][nt][0], pf[b][nt][1]);
          }
        }
      __syncwarp();
      load(stage);
      stage = next_stage;
#pragma unroll
      for (int b = 0; b < kSub; ++b)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[b][nt][0][e] = ahead[b][nt][0][e];
            sc[b][nt][1][e] = ahead[b][nt][1][e];
          }
    }
    // ---- the four warps' states, 8 heads at a time
    const bool whole = s.r0 == 0 && s.r1 == s.units;
    const int slot = open_segment(p, w, share, whole);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float to[2];  // O from its own reference to l's, in two steps: 2^-127 is no normal number
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
        to[e] = ex2(0.5f * (mo[nt][e] - m[nt][e]));
      }
      float* mine = merge + warp * 8 * kMergeLd<D>;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2*>(mine + (2 * quad + e) * kMergeLd<D> + 16 * i + 2 * row8) =
              make_float2(od[nt][i][e] * to[e] * to[e], od[nt][i][e + 2] * to[e] * to[e]);
      if (row8 == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          merge_m[warp][2 * quad + e] = m[nt][e];
          merge_l[warp][2 * quad + e] = l[nt][e];
        }
      }
      __syncthreads();
      merge_warps<kF16, D, kWeighed>(p, s, whole, slot, head0, nt * 8, heads, merge, merge_m, merge_l);
      __syncthreads();
    }
    go = w.next(p);
  }
  copy_wait<0>();
}

template <bool kF16, int D, int NT>
cudaError_t launch_shape(const DecodeParams& p, const Fp8Pools& f, int shares, cudaStream_t stream) {
  constexpr int smem = Shape<D, NT>::kSmemBytes;
  static std::atomic<bool> smem_set[kMaxDevices];
  const cudaError_t e = raise_smem(decode_fp8_kernel<kF16, D, NT>, smem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_after(decode_fp8_kernel<kF16, D, NT>, dim3(shares), kThreads, smem, stream, p, f);
}

template <bool kF16, int D>
cudaError_t launch_heads(const DecodeParams& p, const Fp8Pools& f, int shares, cudaStream_t stream) {
  const cudaError_t e = p.block_heads == 8 ? launch_shape<kF16, D, 1>(p, f, shares, stream) : launch_shape<kF16, D, 2>(p, f, shares, stream);
  return e != cudaSuccess ? e : launch_join(p, kF16, D, shares, stream);
}

bool fp8_plan(int H, const os_paged_cache& c, Plan* out) {
  return make_plan(H, c, ctas_per_sm(heads_of_block(H / c.heads) / 8), 16 * 128 / c.head_dim, kItemWeight, false, out);
}

}  // namespace

int64_t decode_paged_fp8_workspace_bytes(int H, const os_paged_cache& pages) {
  Plan pl;
  return fp8_plan(H, pages, &pl) ? pl.bytes : -1;
}

cudaError_t launch_decode_paged_fp8(const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head, int H,
                                    const os_paged_cache_fp8& cache, float scale, uint16_t* o, float* lse,
                                    void* workspace, unsigned int* err, cudaStream_t stream) {
  Plan pl;
  if (!fp8_plan(H, cache.pages, &pl)) return cudaErrorInvalidDevice;
  const DecodeParams p = decode_params(pl, paged_cache(cache.pages), q, ld_q_batch, ld_q_head, H, scale, o, lse, workspace, err);
  const Fp8Pools f = fp8_pools(cache);
  if (cache.pages.dtype == OS_DTYPE_F16)
    return cache.pages.head_dim == 128 ? launch_heads<true, 128>(p, f, pl.shares, stream)
                                       : launch_heads<true, 64>(p, f, pl.shares, stream);
  return cache.pages.head_dim == 128 ? launch_heads<false, 128>(p, f, pl.shares, stream)
                                     : launch_heads<false, 64>(p, f, pl.shares, stream);
}

}  // namespace oss
