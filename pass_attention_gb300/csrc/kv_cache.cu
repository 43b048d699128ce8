// The paged key-value cache: appending new tokens, and eviction.
//
// Append is a copy (4 D heads bytes read and written per token), bound by HBM
// for whole prompts and by latency for one token a sequence.
//
// Eviction keeps n = min(len, budget) tokens of each (sequence, key head): the
// last `recent`, and of the older ones those of the largest summed weight. The
// selection finds the smallest kept weight by radix: fp32 weights become
// integer keys of the same order, and a histogram of the leading digits of
// the keys that match the digits found so far gives the next digit. Only
// integers are counted, so atomics leave no order in the result. One more
// sweep writes the kept positions in ascending order; of the keys equal to the
// last one kept, the lowest positions are taken.

#include <cstdint>

#include "device_common.cuh"
#include "oss_internal.h"
#include "paged.h"

namespace oss {
namespace {

__device__ __forceinline__ void bad_index(unsigned int* err, unsigned int site) {
  report_error(err, kKernelPaged | (site << 8));
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------

constexpr int kAppendThreads = 256;

// One 16-byte chunk of K and of V per thread; a token's chunks are contiguous
// over the threads.
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, int64_t ld_token,
                 int64_t ld_head, int64_t tokens, const int32_t* __restrict__ cu, PagedCache c,
                 uint16_t* k_pages, uint16_t* v_pages, int chunks_per_head, unsigned int* err) {
  const int per_token = c.heads * chunks_per_head;
  const int64_t total = tokens * per_token;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kAppendThreads) {
    const int64_t token = i / per_token;
    const int within = static_cast<int>(i - token * per_token);
    const int head = within / chunks_per_head;
    const int chunk = within - head * chunks_per_head;
    int seq = static_cast<int>(token);
    int64_t behind = 1;  // new tokens of the sequence from this one on
    if (cu) {
      seq = sequence_of(token, cu, c.batch);
      if (seq < 0) continue;  // a row of no sequence
      behind = cu[seq + 1] - token;
    }
    const int64_t pos = c.kv_len[seq] - behind;
    if (pos < 0 || (pos >> c.page_shift) >= c.max_pages) {
      bad_index(err, kSiteBadPosition);
      continue;
    }
    const int page = c.table[static_cast<int64_t>(seq) * c.ld_table + (pos >> c.page_shift)];
    if (!page_ok(page, c.num_pages)) {
      bad_index(err, kSiteBadPage);
      continue;
    }
    const int slot = static_cast<int>(pos) & ((1 << c.page_shift) - 1);
    const int64_t from = token * ld_token + head * ld_head + chunk * 8;
    const int64_t to = pool_offset(page, head, slot, c.ld_page, c.ld_head, c.ld_slot) + chunk * 8;
    *reinterpret_cast<uint4*>(k_pages + to) = *reinterpret_cast<const uint4*>(k + from);
    *reinterpret_cast<uint4*>(v_pages + to) = *reinterpret_cast<const uint4*>(v + from);
  }
}

// ---------------------------------------------------------------------------
// evict
// ---------------------------------------------------------------------------

constexpr int kSelectThreads = 1024;
constexpr int kDigitBits = 8;
constexpr int kBins = 1 << kDigitBits;

struct EvictParams {
  PagedCache c;
  const float* weights;
  int64_t ld_w_batch, ld_w_head;
  const int32_t* new_table;
  int64_t ld_new_table;
  int32_t new_max_pages, budget, recent;
  int32_t* kept;
  int32_t* new_len;
  float* new_weights;
};

__device__ __forceinline__ uint32_t weight_key(float w) { return weight_key_bits(__float_as_uint(w)); }

// Inclusive scan over the block's threads; *total gets the block's sum.
__device__ uint32_t block_scan(uint32_t x, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int w = 0; w < kSelectThreads / 32; ++w) {
    const uint32_t s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return x + before;
}

// One CTA per (key head, sequence).
__global__ void __launch_bounds__(kSelectThreads)
evict_select_kernel(EvictParams p) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sums[kSelectThreads / 32];
  __shared__ uint32_t found_digit, found_rank;
  const int head = blockIdx.x, seq = blockIdx.y;
  const int len = paged_length(p.c.kv_len[seq], p.c.max_pages, p.c.page_shift);
  const int keep = min(len, p.budget);
  const int recent = min(p.recent, keep);
  const int older = len - recent;
  const int choose = keep - recent;  // <= older
  const int64_t row = static_cast<int64_t>(seq) * p.c.heads + head;
  const float* w = p.weights + static_cast<int64_t>(seq) * p.ld_w_batch + static_cast<int64_t>(head) * p.ld_w_head;
  int32_t* kept = p.kept + row * p.budget;
  const int room = p.new_max_pages << p.c.page_shift;
  float* nw = p.new_weights + row * room;
  if (head == 0 && threadIdx.x == 0) p.new_len[seq] = keep;

  // the smallest kept key, and how many keys equal to it are kept
  uint32_t last = 0, ties = 0xffffffffu;
  if (choose < older) {
    uint32_t rank = choose;  // keys still to place at or below the digits found
    for (int shift = 32 - kDigitBits; shift >= 0 && choose > 0; shift -= kDigitBits) {
      for (int i = threadIdx.x; i < kBins; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      const uint64_t mask = ~((uint64_t(1) << (shift + kDigitBits)) - 1);
      for (int i = threadIdx.x; i < older; i += kSelectThreads) {
        const uint32_t key = weight_key(w[i]);
        if ((key & mask) == last) atomicAdd(&hist[(key >> shift) & (kBins - 1)], 1u);
      }
      __syncthreads();
      // thread i < kBins: keys in the bins above kBins - 1 - i, that bin included
      const uint32_t mine = threadIdx.x < kBins ? hist[kBins - 1 - threadIdx.x] : 0u;
      uint32_t total;
      const uint32_t upto = block_scan(mine, warp_sums, &total);
      if (threadIdx.x < kBins && upto >= rank && upto - mine < rank) {
        found_digit = kBins - 1 - threadIdx.x;
        found_rank = rank - (upto - mine);
      }
      __syncthreads();
      last |= found_digit << shift;
      rank = found_rank;
      __syncthreads();
    }
    ties = rank;
    if (choose == 0) {
      last = 0xffffffffu;
      ties = 0;
    }
  }
  // kept positions in ascending order
  uint32_t above = 0, equal = 0;  // keys before this tile
  for (int base = 0; base < older; base += kSelectThreads) {
    const int i = base + threadIdx.x;
    const uint32_t key = i < older ? weight_key(w[i]) : 0u;
    const bool gt = i < older && (key > last || ties == 0xffffffffu);
    const bool eq = i < older && key == last && !gt;
    uint32_t total;
    const uint32_t upto = block_scan((gt ? 1u : 0u) | (eq ? 0x10000u : 0u), warp_sums, &total);
    const uint32_t gt_before = above + (upto & 0xffffu) - (gt ? 1u : 0u);
    const uint32_t eq_before = equal + (upto >> 16) - (eq ? 1u : 0u);
    if (gt || (eq && eq_before < ties)) {
      const uint32_t at = gt_before + min(eq_before, ties);
      kept[at] = i;
      nw[at] = w[i];
    }
    above += total & 0xffffu;
    equal += total >> 16;
  }
  for (int i = threadIdx.x; i < recent; i += kSelectThreads) {
    kept[choose + i] = older + i;
    nw[choose + i] = w[older + i];
  }
  for (int i = keep + threadIdx.x; i < p.budget; i += kSelectThreads) kept[i] = -1;
  for (int i = keep + threadIdx.x; i < room; i += kSelectThreads) nw[i] = 0.f;
}

constexpr int kMoveThreads = 128;
constexpr int kMoveRows = 64;  // rows a CTA moves

// One CTA per (rows, key head, sequence); a group of D / 8 threads takes a row.
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(EvictParams p, uint16_t* k_pages, uint16_t* v_pages, int chunks_per_head,
                  unsigned int* err) {
  const int head = blockIdx.y, seq = blockIdx.z;
  const int64_t row = static_cast<int64_t>(seq) * p.c.heads + head;
  const int32_t* kept = p.kept + row * p.budget;
  const int rows = min(p.budget, p.new_max_pages << p.c.page_shift);
  const int per_pass = kMoveThreads / chunks_per_head;
  const int chunk = threadIdx.x % chunks_per_head;
  const int first = blockIdx.x * kMoveRows;
  const int slot_mask = (1 << p.c.page_shift) - 1;
  for (int r = first + threadIdx.x / chunks_per_head; r < min(first + kMoveRows, rows); r += per_pass) {
    const int pos = kept[r];
    if (pos < 0) break;
    const int from = p.c.table[static_cast<int64_t>(seq) * p.c.ld_table + (pos >> p.c.page_shift)];
    const int to = p.new_table[static_cast<int64_t>(seq) * p.ld_new_table + (r >> p.c.page_shift)];
    if (!page_ok(from, p.c.num_pages) || !page_ok(to, p.c.num_pages)) {
      bad_index(err, kSiteBadPage);
      continue;
    }
    const int64_t a = pool_offset(from, head, pos & slot_mask, p.c.ld_page, p.c.ld_head, p.c.ld_slot) + chunk * 8;
    const int64_t b = pool_offset(to, head, r & slot_mask, p.c.ld_page, p.c.ld_head, p.c.ld_slot) + chunk * 8;
    const uint4 kk = *reinterpret_cast<const uint4*>(k_pages + a);
    const uint4 vv = *reinterpret_cast<const uint4*>(v_pages + a);
    *reinterpret_cast<uint4*>(k_pages + b) = kk;
    *reinterpret_cast<uint4*>(v_pages + b) = vv;
  }
}

PagedCache device_cache(const os_paged_cache& c) {
  int shift = 0;
  while ((1 << shift) < c.page_size) ++shift;
  return PagedCache{static_cast<const uint16_t*>(c.k_pages), static_cast<const uint16_t*>(c.v_pages),
                    c.ld_page, c.ld_head, c.ld_slot, c.page_table, c.ld_table, c.kv_len,
                    c.num_pages, shift, c.max_pages, c.heads, c.batch};
}

}  // namespace

PagedCache paged_cache(const os_paged_cache& c) { return device_cache(c); }

cudaError_t launch_kv_append(const uint16_t* k, const uint16_t* v, int64_t ld_token, int64_t ld_head,
                             int64_t tokens, const int32_t* cu, const os_paged_cache& cache,
                             unsigned int* err, cudaStream_t stream) {
  const int chunks = cache.head_dim / 8;
  const int64_t total = tokens * cache.heads * chunks;
  int64_t blocks = (total + kAppendThreads - 1) / kAppendThreads;
  if (blocks > 152 * 64) blocks = 152 * 64;
  kv_append_kernel<<<static_cast<unsigned>(blocks), kAppendThreads, 0, stream>>>(
      k, v, ld_token, ld_head, tokens, cu, device_cache(cache),
      static_cast<uint16_t*>(cache.k_pages), static_cast<uint16_t*>(cache.v_pages), chunks, err);
  return cudaGetLastError();
}

cudaError_t launch_kv_evict(const os_paged_cache& cache, const float* weights, int64_t ld_w_batch,
                            int64_t ld_w_head, const int32_t* new_table, int64_t ld_new_table,
                            int32_t new_max_pages, int32_t budget, int32_t recent, int32_t* kept,
                            int32_t* new_len, float* new_weights, unsigned int* err,
                            cudaStream_t stream) {
  const EvictParams p{device_cache(cache), weights, ld_w_batch, ld_w_head, new_table, ld_new_table,
                      new_max_pages, budget, recent, kept, new_len, new_weights};
  evict_select_kernel<<<dim3(cache.heads, cache.batch), kSelectThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 grid((budget + kMoveRows - 1) / kMoveRows, cache.heads, cache.batch);
  evict_move_kernel<<<grid, kMoveThreads, 0, stream>>>(p, static_cast<uint16_t*>(cache.k_pages),
                                                       static_cast<uint16_t*>(cache.v_pages),
                                                       cache.head_dim / 8, err);
  return cudaGetLastError();
}

}  // namespace oss
