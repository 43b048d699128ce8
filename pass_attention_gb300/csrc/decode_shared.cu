// Attention of one new token per sequence, where groups of sequences share a prefix.
//
// With sequence b's keys the prefix P of its group and its own tokens S, o and lse come from
// the states (m, l, O) of both:  m = max(m_P, m_S);  l = l_P 2^(m_P - m) + l_S 2^(m_S - m);  O
// likewise;  o = O / l.
//
// Three kernels. (1) The prefixes, on the tensor cores (attn_packed.cu, prefix
// kernels): the queries of a group, times the query heads of a key head, fill the
// 128 rows of a tile, so a prefix is read once for up to 128 rows instead of once for every
// sequence. (A tile takes 2^n heads, the largest power of two that divides the group, and the
// group's others are tiles that walk the prefix for themselves: with 12 heads a key head
// three, with 7 seven. 64 sequences behind 65536 tokens of 8 key heads, 24 query heads 178 us, 32: 110,
// 40: 258; of 4 key heads, 28: 171, 48: 131; 16 behind 32768 of 4 key heads, 28: 63, 48: 43.)
// (2) The sequences' own tokens, by the paged decode's first kernel (decode_paged.cu). (3) The join
// below, of the parts and states that the two have left.
//
// What bounds it: the first kernel the chain of a KV step (0.9 us for 128 rows of 128 keys),
// from about two tiles of rows on, HBM below that; the second HBM. They run side by side
// (prefix_split.cuh). The second reads nothing of the first, so it is launched to start when all
// that came before the first has ended, and waits for the first at its own end.
//
// Measured, 32 heads over 8 of 128: 64 sequences of up to 1000 tokens behind 8192: 46 us (183 MB:
// 27 us of HBM's time); of up to 2500 behind 65536: 107 us (566 MB: 85 us). With one table a
// sequence, every one of them with the prefix's pages in front, the paged decode takes 193
// and 1455 us. Of a launch, 5 us are the way to the first product, and 6 the join with its two
// hand-overs.

#include <cstdint>

#include "decode_paged_kernel.cuh"
#include "device_common.cuh"
#include "launch.cuh"
#include "oss_internal.h"
#include "prefix_rule.h"

namespace oss {
namespace {

using namespace decode;

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
// Rows (a sequence's query head) of a CTA. A tile's rows lie 16 bytes apart, 4 dims of each:
// four neighbours make up two sectors. (One row a CTA took 14 us for 2048 rows of 11 parts,
// every read half wasted and five dependent loads at the front; four rows and two loads
// take 7.5, in turns of 4 warps, and with 8 the whole call 0.3 to 0.9 us less.)
constexpr int kJoinRows = 4;

// What the first kernel has left.
struct PrefixStates {
  const int4* where;
  const float4* part_o;  // [2 shares][D / 4][128]
  const float2* part_ml;
  const float4* state_o;  // [batch][H][D / 4]
  const float2* state_ml;
  int32_t shares, packs, head_shift;
};

// A warp takes every eighth part of the four rows, first the prefix's, then those of the
// own tokens. Thread: row lane % 4, the vectors of 4 dims lane / 4, lane / 4 + 8, ...
// kInPairs: the prefix's parts and states are those of sequence 2 b of the decode's kernel.
template <bool kF16, int D, bool kInPairs>
__global__ void __launch_bounds__(kJoinThreads) decode_shared_join_kernel(const DecodeParams p, const PrefixStates x) {
  constexpr int kVecs = D / 32;
  __shared__ float2 sml[kJoinWarps][kJoinRows];
  __shared__ float4 so[kJoinWarps][kJoinRows][D / 4 + 1];
  let_next_kernel_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, v0 = lane >> 2;
  const int64_t rows = static_cast<int64_t>(p.c.batch) * p.H;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kJoinRows + (lane & 3);
  const bool live = row < rows;
  const int b = live ? static_cast<int>(row / p.H) : 0, h = live ? static_cast<int>(row - static_cast<int64_t>(b) * p.H) : 0;
  const int g = h / p.group, in_group = h - g * p.group, hb = in_group / p.block_heads;
  const int in_block = in_group - hb * p.block_heads;
  wait_for_previous_kernel();
  const int per_seq = p.c.heads * p.head_blocks, item = g * p.head_blocks + hb;
  int2 own, pre = make_int2(0, 0);  // kInPairs: {first share, parts} of the prefix
  int4 w = make_int4(0, 0, 0, 0);
  int parts = 0;  // of the prefix
  int64_t pre_row = row, own_row = row;
  if constexpr (kInPairs) {
    pre = p.item_meta[static_cast<int64_t>(2 * b) * per_seq + item];
    own = p.item_meta[static_cast<int64_t>(2 * b + 1) * per_seq + item];
    parts = pre.y;
    pre_row = static_cast<int64_t>(2 * b) * p.H + h;
    own_row = pre_row + p.H;
  } else {
    own = p.item_meta[static_cast<int64_t>(b) * per_seq + item];
    w = x.where[static_cast<int64_t>(b) * x.packs + (h >> x.head_shift)];
    if (own.y > 0) {
      parts = w.y != 0 ? w.y : 1;
      // (a launch that gave up on a wait has not written this)
      if (w.y != 0 && (parts < 0 || w.x < 0 || w.w < 1 || w.w > x.shares || w.x + (parts - 1) * static_cast<int64_t>(w.w) >= x.shares))
        parts = 0;
    } else {
      own.y = -own.y;  // no group names the sequence
    }
  }
  const int tile_row = (w.z + (h & ((1 << x.head_shift) - 1))) & 127;
  const int all = live ? parts + own.y : 0;

  float M = neg_inf(), L = 0.f;
  float4 acc[kVecs];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int i = warp; i < all; i += kJoinWarps) {
    float2 ml;
    const float4* src;
    int step = 8;  // vectors from one of this thread's to the next
    if (!kInPairs && i < parts) {
      if (w.y == 0) {
        ml = x.state_ml[row];
        src = x.state_o + row * (D / 4) + v0;
      } else {
        const int64_t slot = 2 * (w.x + static_cast<int64_t>(i) * w.w) + (i == 0 ? 1 : 0);
        ml = x.part_ml[slot * 128 + tile_row];
        src = x.part_o + (slot * (D / 4) + v0) * 128 + tile_row;
        step = 8 * 128;
      }
    } else {
      const bool first = i < parts;  // kInPairs
      const int2 it = first ? pre : own;
      const int64_t of = first ? pre_row : own_row;
      if (it.y == 1) {
        ml = p.state_ml[of];
        src = reinterpret_cast<const float4*>(p.state_o) + of * (D / 4) + v0;
      } else {
        const int64_t at = part_slot(it.x, first ? i : i - parts) * p.block_heads + in_block;
        ml = p.part_ml[at];
        src = reinterpret_cast<const float4*>(p.part_o) + at * (D / 4) + v0;
      }
    }
    float4 v[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) v[k] = src[k * step];
    const float to = fmaxf(M, ml.x), ref = reference(to), corr = ex2(M - ref), f = ex2(ml.x - ref);
    M = to;
    L = fmaf(ml.y, f, L * corr);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      acc[k].x = fmaf(v[k].x, f, acc[k].x * corr);
      acc[k].y = fmaf(v[k].y, f, acc[k].y * corr);
      acc[k].z = fmaf(v[k].z, f, acc[k].z * corr);
      acc[k].w = fmaf(v[k].w, f, acc[k].w * corr);
    }
  }
  if (v0 == 0) sml[warp][lane & 3] = make_float2(M, L);
#pragma unroll
  for (int k = 0; k < kVecs; ++k) so[warp][lane & 3][v0 + 8 * k] = acc[k];
  __syncthreads();
  // warp: one of the rows; lane: D / 32 dims
  if (warp >= kJoinRows) return;
  const int64_t out = static_cast<int64_t>(blockIdx.x) * kJoinRows + warp;
  if (out >= rows) return;
  M = neg_inf();
  L = 0.f;
  float y[kVecs];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) y[k] = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) M = fmaxf(M, sml[i][warp].x);
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) {
    const float2 ml = sml[i][warp];
    const float f = ex2(ml.x - reference(M)), *from = reinterpret_cast<const float*>(so[i][warp]) + lane * kVecs;
    L = fmaf(ml.y, f, L);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) y[k] = fmaf(from[k], f, y[k]);
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + out * D + lane * kVecs);
  if constexpr (kVecs == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<kF16>(y[0] * inv, y[1] * inv), pack2<kF16>(y[2] * inv, y[3] * inv));
  else
    *dst = pack2<kF16>(y[0] * inv, y[1] * inv);
  if (lane == 0 && p.lse) p.lse[out] = L != 0.f ? (M + log2f(L)) * kLn2 : neg_inf();
}

int64_t round256(int64_t n) { return (n + 255) / 256 * 256; }

// Layout of the workspace: the prefixes' part (not in pairs), the decode's, and its states.
struct SharedPlan {
  bool pairs;
  PrefixPlan prefix;
  Plan own;
  int64_t own_at, item_meta, state_o, state_ml, bytes;
};

bool make_shared_plan(int H, const os_paged_cache& c, int groups, int prefix_max_pages, SharedPlan* out) {
  const int group = H / c.heads, block_heads = heads_of_block(group);
  out->pairs = read_by_every_sequence(c.batch, groups, (group + block_heads - 1) / block_heads,
                                      static_cast<int64_t>(prefix_max_pages) * c.page_size,
                                      4 * static_cast<int64_t>(c.heads) * c.head_dim);
  os_paged_cache walked = c;  // the sequences of the decode's kernel
  if (out->pairs) {
    walked.batch = 2 * c.batch;
    if (prefix_max_pages > c.max_pages) walked.max_pages = prefix_max_pages;
  }
  if (!make_plan(H, walked, kCtasPerSm, kTileKeys, kItemWeight, false, &out->own)) return false;
  out->prefix = prefix_plan(H, c);
  const int64_t rows = static_cast<int64_t>(walked.batch) * H;
  out->own_at = out->pairs ? 0 : out->prefix.bytes;
  out->item_meta = out->own_at + out->own.bytes;
  out->state_o = out->item_meta + round256(static_cast<int64_t>(walked.batch) * c.heads * out->own.head_blocks * 8);
  out->state_ml = out->state_o + round256(rows * c.head_dim * 4);
  out->bytes = out->state_ml + round256(rows * 8);
  return true;
}

template <bool kInPairs>
cudaError_t launch_join(const DecodeParams& p, const PrefixStates& x, bool f16, int D, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.c.batch) * p.H;
  const dim3 grid(static_cast<unsigned>((rows + kJoinRows - 1) / kJoinRows));
  const auto join = [&](auto* kernel) { return launch_after(kernel, grid, kJoinThreads, 0, stream, p, x); };
  if (D == 128) return f16 ? join(decode_shared_join_kernel<true, 128, kInPairs>) : join(decode_shared_join_kernel<false, 128, kInPairs>);
  return f16 ? join(decode_shared_join_kernel<true, 64, kInPairs>) : join(decode_shared_join_kernel<false, 64, kInPairs>);
}

}  // namespace

int64_t decode_shared_workspace_bytes(int H, const os_paged_cache& cache, int groups, int prefix_max_pages) {
  SharedPlan pl;
  return make_shared_plan(H, cache, groups, prefix_max_pages, &pl) ? pl.bytes : -1;
}

cudaError_t launch_decode_shared(const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head, int H,
                                 const os_paged_cache& cache, const PrefixTables& prefix, float scale, uint16_t* o,
                                 float* lse, void* workspace, unsigned int* err, const AttnFault& fault,
                                 cudaStream_t stream) {
  SharedPlan pl;
  if (!make_shared_plan(H, cache, prefix.groups, prefix.max_pages, &pl)) return cudaErrorInvalidDevice;
  char* ws = static_cast<char*>(workspace);
  const bool f16 = cache.dtype == OS_DTYPE_F16;
  const int D = cache.head_dim;
  const PagedCache c = paged_cache(cache);
  const PrefixLaunch x{prefix, cache.batch, c.page_shift, 7 - pl.prefix.head_shift, pl.prefix.packs, device_sms(),
                       cache.heads * pl.own.head_blocks, D == 128 ? kStepCost : kStepCost64,
                       pl.own.block_heads > 8 ? kWideUnitCost : D == 128 ? kUnitCost : kUnitCost64,
                       pl.own.whole ? 0 : kUnitBytesCost * D / 128};
  cudaError_t e;
  if (!pl.pairs && (e = launch_attn_prefix(q, ld_q_batch, ld_q_head, H, cache, x, scale, pl.prefix, ws, err, fault, stream)) != cudaSuccess)
    return e;
  DecodeParams p = decode_params(pl.own, c, q, ld_q_batch, ld_q_head, H, scale, o, lse, ws + pl.own_at, err);
  p.item_meta = reinterpret_cast<int2*>(ws + pl.item_meta);
  p.state_o = reinterpret_cast<float*>(ws + pl.state_o);
  p.state_ml = reinterpret_cast<float2*>(ws + pl.state_ml);
  p.prefix = x;
  e = pl.pairs ? launch_kernel<kPairs>(p, f16, D, pl.own.shares, stream) : launch_kernel<kBehind>(p, f16, D, pl.own.shares, stream);
  if (e != cudaSuccess) return e;
  if (pl.pairs) return launch_join<true>(p, PrefixStates{}, f16, D, stream);
  const PrefixStates states{reinterpret_cast<const int4*>(ws + pl.prefix.where),
                            reinterpret_cast<const float4*>(ws + pl.prefix.part_o),
                            reinterpret_cast<const float2*>(ws + pl.prefix.part_ml),
                            reinterpret_cast<const float4*>(ws + pl.prefix.state_o),
                            reinterpret_cast<const float2*>(ws + pl.prefix.state_ml),
                            pl.prefix.shares, pl.prefix.packs, pl.prefix.head_shift};
  return launch_join<false>(p, states, f16, D, stream);
}

}  // namespace oss
