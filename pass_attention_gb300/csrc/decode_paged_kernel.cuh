// The paged decode's first kernel, over 16-bit pools. The reasons stand in decode_paged.cu.
#pragma once

#include "decode_paged.cuh"

namespace oss {
namespace decode {

template <int D>
struct Shape {
  static constexpr int kStages = D == 128 ? 3 : 6;  // 24 KB of K and V in flight per warp
  static constexpr int kRowBytes = D * 2;
  static constexpr int kTileBytes = kTileKeys * kRowBytes;  // K or V
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  static constexpr int kSmemBytes = kRingBytes + kMergeBytes<D>;
};

// NT: blocks of 8 query heads.
template <bool kF16, int D, int NT, Mode kMode>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode_paged_kernel(const DecodeParams p) {
  using S = Shape<D>;
  constexpr int kChunks = D / 8;              // 16-byte chunks of a row
  constexpr int kRowsPerCopy = 32 / kChunks;  // rows a warp's copy instruction covers
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float merge_m[kWarps][8], merge_l[kWarps][8];
  let_next_kernel_start();
  if constexpr (kMode == kBehind)
    begin_behind_waiting_kernel();
  else
    wait_for_previous_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane & 3, row8 = lane >> 2;

  Walk<kTileKeys, kMode> w;
  ShareCut share;
  const bool has_share = find_share(p, &w, &share);
  if (threadIdx.x == 0) p.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (!has_share) {
    if (kMode == kBehind && blockIdx.x == 0) wait_for_previous_kernel();
    return;
  }

  const uint32_t ring = smem_u32(smem) + warp * kStages * S::kStageBytes;
  float* merge = reinterpret_cast<float*>(smem + S::kRingBytes);
  const int copy_row = lane / kChunks, copy_chunk = lane % kChunks;

  // ---- the loads' cursor: the tile to be loaded next, and its page
  Walk<kTileKeys, kMode> lw = w;
  int lt = lw.s.r0 * p.unit_tiles + warp;
  bool more = true;
  int page = 0;
  const int32_t* row = seq_table<kMode>(p, lw.s.b);
  auto settle = [&]() {  // move to the next tile that exists, fetch its page number
    while (lt >= lw.tile_end(p)) {
      if (!(more = lw.next(p))) return;
      lt = lw.s.r0 * p.unit_tiles + warp;
      row = seq_table<kMode>(p, lw.s.b);
    }
    page = row[(lt * kTileKeys) >> p.c.page_shift];
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
          p.q + (kMode == kPairs ? s.b >> 1 : s.b) * p.ld_q_batch + static_cast<int64_t>(live ? head0 + nt * 8 + row8 : 0) * p.ld_q_head);
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
    const int slot = open_segment(p, w, share, whole);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int e = 0; e < 2; ++e) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
      float* mine = merge + warp * 8 * kMergeLd<D>;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(2 * quad + (e & 1)) * kMergeLd<D> + 16 * i + row8 + (e >> 1) * 8] = od[nt][i][e];
      if (row8 == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          merge_m[warp][2 * quad + e] = m[nt][e];
          merge_l[warp][2 * quad + e] = l[nt][e];
        }
      }
      __syncthreads();
      merge_warps<kF16, D, kMode>(p, s, whole, slot, head0, nt * 8, heads, merge, merge_m, merge_l);
      __syncthreads();
    }
    go = w.next(p);
  }
  copy_wait<0>();
  // (behind prefixes: this kernel ends when its first CTA has seen the one before it end. The
  // others leave, so that CTAs without a share do not wait for a place on an SM.)
  if (kMode == kBehind && blockIdx.x == 0) wait_for_previous_kernel();
}

template <bool kF16, int D, int NT, Mode kMode>
cudaError_t launch_shape(const DecodeParams& p, int shares, cudaStream_t stream) {
  constexpr int smem = Shape<D>::kSmemBytes;
  static std::atomic<bool> smem_set[kMaxDevices];
  const cudaError_t e = raise_smem(decode_paged_kernel<kF16, D, NT, kMode>, smem, smem_set);
  if (e != cudaSuccess) return e;
  return launch_after(decode_paged_kernel<kF16, D, NT, kMode>, dim3(shares), kThreads, smem, stream, p);
}

template <Mode kMode>
cudaError_t launch_kernel(const DecodeParams& p, bool f16, int D, int shares, cudaStream_t stream) {
  if (p.block_heads == 8) {
    if (D == 128) return f16 ? launch_shape<true, 128, 1, kMode>(p, shares, stream) : launch_shape<false, 128, 1, kMode>(p, shares, stream);
    return f16 ? launch_shape<true, 64, 1, kMode>(p, shares, stream) : launch_shape<false, 64, 1, kMode>(p, shares, stream);
  }
  if (D == 128) return f16 ? launch_shape<true, 128, 2, kMode>(p, shares, stream) : launch_shape<false, 128, 2, kMode>(p, shares, stream);
  return f16 ? launch_shape<true, 64, 2, kMode>(p, shares, stream) : launch_shape<false, 64, 2, kMode>(p, shares, stream);
}

}  // namespace decode
}  // namespace oss
