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

#include "decode_paged_kernel.cuh"
#include "device_common.cuh"
#include "launch.cuh"
#include "oss_internal.h"

namespace oss {
namespace {

using namespace decode;

// The second kernel. With weights, its first CTAs add up: kAddKeys keys of one key
// head each. The others join: CTA (c, hh) merges head hh of the item that begins
// in share c and goes on into the next ones; its warps take the parts in turn.
constexpr int kFinishThreads = 256;
constexpr int kFinishWarps = kFinishThreads / 32;
constexpr int kAddKeysPerThread = 4;
constexpr int kAddKeys = kAddKeysPerThread * kFinishThreads;

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
__device__ __forceinline__ void add_weights(const DecodeParams& p, int b, int g, int chunk, float* weights) {
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
  const int heads = min(p.group, p.block_heads);
  join_head<kF16, D>(p, i / heads, i % heads);
}

template <bool kF16, int D>
cudaError_t launch_finish(const DecodeParams& p, int shares, float* weights, int64_t ld_w_batch, int64_t ld_w_head,
                          cudaStream_t stream) {
  const int heads = p.group < p.block_heads ? p.group : p.block_heads;
  const int64_t joins = p.unit_tiles == kUnitTiles ? static_cast<int64_t>(shares) * heads : 0;
  const int64_t chunks = weights ? ((static_cast<int64_t>(p.c.max_pages) << p.c.page_shift) + kAddKeys - 1) / kAddKeys : 0;
  const int64_t adds = chunks * p.c.heads * p.c.batch, ctas = adds + joins;
  if (ctas > 0x7fffffff) return cudaErrorNotSupported;
  if (ctas == 0) return cudaSuccess;
  return launch_after(decode_finish_kernel<kF16, D>, dim3(static_cast<unsigned>(ctas)), kFinishThreads, 0, stream, p,
                      static_cast<int>(adds), static_cast<int>(chunks), weights, ld_w_batch, ld_w_head);
}

cudaError_t launch_finish(const DecodeParams& p, bool f16, int D, int shares, float* weights, int64_t ld_w_batch,
                          int64_t ld_w_head, cudaStream_t stream) {
  if (D == 128)
    return f16 ? launch_finish<true, 128>(p, shares, weights, ld_w_batch, ld_w_head, stream)
               : launch_finish<false, 128>(p, shares, weights, ld_w_batch, ld_w_head, stream);
  return f16 ? launch_finish<true, 64>(p, shares, weights, ld_w_batch, ld_w_head, stream)
             : launch_finish<false, 64>(p, shares, weights, ld_w_batch, ld_w_head, stream);
}

}  // namespace

namespace decode {

bool make_plan(int H, const os_paged_cache& c, int ctas, int tile_keys, int item_weight, bool weights, Plan* out) {
  const int sms = device_sms();
  if (sms < 1) return false;
  const int group = H / c.heads;
  Plan pl;
  pl.block_heads = heads_of_block(group);
  pl.head_blocks = (group + pl.block_heads - 1) / pl.block_heads;
  pl.score_heads = pl.head_blocks > 1 ? pl.block_heads : (group + 3) / 4 * 4;
  const int64_t capacity = static_cast<int64_t>(c.max_pages) * c.page_size;
  const int64_t items = static_cast<int64_t>(c.batch) * c.heads * pl.head_blocks;
  pl.shares = sms * ctas;
  pl.whole = capacity <= kWholeKeys || (capacity <= kWholeKeysMany && items >= pl.shares);
  pl.unit_tiles = pl.whole ? kWholeKeysMany / tile_keys : kUnitTiles;
  pl.item_weight = pl.whole ? 0 : item_weight;
  // no more than there are places in the row of items, if every sequence fills its pages
  const int64_t unit = static_cast<int64_t>(tile_keys) * pl.unit_tiles;
  const int64_t places = items * ((capacity + unit - 1) / unit + pl.item_weight);
  if (pl.shares > places) pl.shares = static_cast<int>(places);
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

DecodeParams decode_params(const Plan& pl, const PagedCache& c, const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head,
                           int H, float scale, uint16_t* o, float* lse, void* workspace, unsigned int* err) {
  char* ws = static_cast<char*>(workspace);
  DecodeParams p = {};
  p.c = c;
  p.q = q;
  p.ld_q_batch = ld_q_batch;
  p.ld_q_head = ld_q_head;
  p.H = H;
  p.group = H / c.heads;
  p.head_blocks = pl.head_blocks;
  p.block_heads = pl.block_heads;
  p.unit_tiles = pl.unit_tiles;
  p.item_weight = pl.item_weight;
  p.score_heads = pl.score_heads;
  p.scale2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  p.o = o;
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_ml);
  p.meta = reinterpret_cast<int4*>(ws + pl.meta);
  p.err = err;
  return p;
}

cudaError_t launch_join(const DecodeParams& p, bool f16, int D, int shares, cudaStream_t stream) {
  return launch_finish(p, f16, D, shares, nullptr, 0, 0, stream);
}

}  // namespace decode

int64_t decode_paged_workspace_bytes(int H, const os_paged_cache& cache, bool weights) {
  Plan pl;
  return make_plan(H, cache, kCtasPerSm, kTileKeys, 0, weights, &pl) ? pl.bytes : -1;
}

cudaError_t launch_decode_paged(const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head, int H,
                                const os_paged_cache& cache, float scale, uint16_t* o, float* lse,
                                float* weights, int64_t ld_w_batch, int64_t ld_w_head,
                                void* workspace, unsigned int* err, cudaStream_t stream) {
  Plan pl;
  if (!make_plan(H, cache, kCtasPerSm, kTileKeys, 0, weights != nullptr, &pl)) return cudaErrorInvalidDevice;
  DecodeParams p = decode_params(pl, paged_cache(cache), q, ld_q_batch, ld_q_head, H, scale, o, lse, workspace, err);
  if (weights) {
    char* ws = static_cast<char*>(workspace);
    p.lse2 = reinterpret_cast<float*>(ws + pl.lse2);
    p.item_meta = reinterpret_cast<int2*>(ws + pl.item_meta);
    p.scores = reinterpret_cast<float*>(ws + pl.scores);
  }
  const bool f16 = cache.dtype == OS_DTYPE_F16;
  const cudaError_t e = launch_kernel<kPlain>(p, f16, cache.head_dim, pl.shares, stream);
  return e != cudaSuccess ? e : launch_finish(p, f16, cache.head_dim, pl.shares, weights, ld_w_batch, ld_w_head, stream);
}

}  // namespace oss
