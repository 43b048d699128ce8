// The paged key-value cache: appending new tokens, and eviction.
//
// Append is a copy (4 D heads bytes read and written per token), bound by HBM
// for whole prompts (37 k tokens, 8 heads of 128: 47.6 us, 0.96 of the copy peak)
// and by latency for one token a sequence (64 sequences: 3.5 us).
//
// Eviction keeps n = min(len, budget) tokens of each (sequence, key head): the
// last `recent`, and of the older ones those of the largest summed weight. Two
// kernels, both bound by HBM:
//
// * select. The smallest kept weight is found by radix: fp32 weights become
//   integer keys of the same order, and a histogram of a digit (11, 11, 10 bits)
//   of the keys that agree with the digits found so far gives the next digit.
//   A thread-block cluster takes a row: its CTAs hold the weights of a slice in
//   shared memory (one read), and each adds up all CTAs' histograms through
//   distributed shared memory, so every digit costs one cluster barrier: first 64
//   sums of 32 bins each, then the 32 bins that hold the digit (all 2048 bins from
//   eight CTAs took 2 us a digit). Only integers are counted, so the atomics leave
//   no order in the result. One more sweep writes the kept positions in ascending
//   order; of the keys equal to the last one kept, the lowest positions are taken.
// * move. Kept rows are copied page to page, four rows of a thread in flight.
//
// 2 x 8 rows of up to 131072 weights cut to 16384: 69 us, of them 42 the copy (at
// the copy peak) and most of the rest the selection, a chain of about ten meetings
// of a cluster's CTAs; 8 x 8 rows of up to 8192 cut to 2048: 37 us, 23 of them the
// copy.

#include <atomic>
#include <cstdint>

#include "device_common.cuh"
#include "launch.cuh"
#include "oss_internal.h"
#include "paged.h"
#include "softmax_common.cuh"

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
kv_append_kernel(const uint16_t* k, const uint16_t* v, int64_t ld_token, int64_t ld_head, int64_t tokens, const int32_t* cu,
                 PagedCache c, uint16_t* k_pages, uint16_t* v_pages, int chunks_per_head, unsigned int* err) {
  let_next_kernel_start();
  wait_for_previous_kernel();
  // offsets that do not fit the rows: tokens that kv_len counts are not written
  if (cu)
    for (int b = blockIdx.x * kAppendThreads + threadIdx.x; b < c.batch; b += gridDim.x * kAppendThreads)
      if (row_range(cu[b], cu[b + 1], static_cast<int32_t>(tokens)).clamped) bad_index(err, kSiteBadOffsets);
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
    const int32_t len = c.kv_len[seq];
    if (!cu && len == 0) continue;  // an empty place of the batch
    const int64_t pos = len - behind;
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
    const uint4 key = *reinterpret_cast<const uint4*>(k + from), value = *reinterpret_cast<const uint4*>(v + from);
    *reinterpret_cast<uint4*>(k_pages + to) = key;
    *reinterpret_cast<uint4*>(v_pages + to) = value;
  }
}

// ---------------------------------------------------------------------------
// evict
// ---------------------------------------------------------------------------

constexpr int kSelectThreads = 1024;
constexpr int kDigits = 3;
constexpr int kBins = 2048;
constexpr int kCoarse = 64;  // sums of 32 bins
constexpr int kMaxCluster = 8;
constexpr int kMaxSliceKeys = 48 * 1024;  // 192 KB of weights in shared memory
constexpr int kLeastSlice = 4096;

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

// Inclusive scan over a warp.
__device__ __forceinline__ uint32_t warp_scan(uint32_t x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  return x;
}

// Inclusive scan over the block's threads; *total gets the block's sum.
__device__ uint32_t block_scan(uint32_t x, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_scan(x);
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  // every warp scans the warps' sums
  const uint32_t w = warp_scan(warp_sums[lane]);
  *total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return x + (warp > 0 ? before : 0u);
}

__device__ __forceinline__ uint2 ld_peer2(const uint32_t* slot, uint32_t rank) {
  uint32_t remote;
  uint2 x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(slot)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(remote) : "memory");
  return x;
}

__device__ __forceinline__ uint32_t ld_peer(const uint32_t* slot, uint32_t rank) {
  uint32_t remote, x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(slot)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(remote) : "memory");
  return x;
}

// One cluster per (key head, sequence). kCached: a CTA's slice of the keys lies in
// shared memory; otherwise every sweep reads the weights again.
template <bool kCached>
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(EvictParams p) {
  extern __shared__ uint32_t slice_bits[];  // the weights of this CTA's slice, as they are
  __shared__ uint32_t hist[kDigits][kBins];
  __shared__ __align__(8) uint32_t coarse[kDigits][kCoarse];
  __shared__ uint32_t warp_sums[kSelectThreads / 32];
  __shared__ uint32_t found_digit, found_rank;
  __shared__ __align__(8) uint32_t slice_counts[2];
  let_next_kernel_start();
  const uint32_t C = cluster_size(), rank = cluster_rank();
  const int head = blockIdx.x / C, seq = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  const int in_cluster = static_cast<int>(rank) * kSelectThreads + tid, all_threads = static_cast<int>(C) * kSelectThreads;
  if (head == 0 && in_cluster == 0) p.new_len[seq] = keep;

  // the rows' parts that need no selection
  auto write_rest = [&]() {
    for (int i = in_cluster; i < recent; i += all_threads) {
      kept[choose + i] = older + i;
      nw[choose + i] = w[older + i];
    }
    for (int i = keep + in_cluster; i < p.budget; i += all_threads) kept[i] = -1;
    for (int i = keep + in_cluster; i < room; i += all_threads) nw[i] = 0.f;
  };
  if (choose == 0 || choose == older) {  // the same for the whole cluster
    write_rest();
    for (int i = in_cluster; i < choose; i += all_threads) {
      kept[i] = i;
      nw[i] = w[i];
    }
    return;
  }

  const int slice = (older + static_cast<int>(C) - 1) / static_cast<int>(C);
  const int first = min(older, static_cast<int>(rank) * slice);
  const int n = min(older - first, slice);
  auto bits_at = [&](int i) -> uint32_t { return kCached ? slice_bits[i] : __float_as_uint(w[first + i]); };
  if constexpr (kCached) {
    // (asynchronous: every key of a thread is on its way at once)
#pragma unroll 4
    for (int i = tid; i < n; i += kSelectThreads)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(slice_bits + i)), "l"(w + first + i) : "memory");
  }
  for (int i = tid; i < kDigits * kBins; i += kSelectThreads) (&hist[0][0])[i] = 0;
  if constexpr (kCached) asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // the smallest kept key, and how many keys equal to it are kept
  uint32_t last = 0, ties = choose;
#pragma unroll
  for (int d = 0; d < kDigits; ++d) {
    const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0);
    const int bits = d == 2 ? 10 : 11;
#pragma unroll 4
    for (int i = tid; i < n; i += kSelectThreads) {
      const uint32_t key = weight_key_bits(bits_at(i));
      if (d == 0 || (key >> (shift + bits)) == (last >> (shift + bits)))
        atomicAdd(&hist[d][(key >> shift) & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    // a warp: two sums of 32 bins
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t c = __reduce_add_sync(0xffffffffu, hist[d][(2 * warp + i) * 32 + lane]);
      if (lane == 0) coarse[d][2 * warp + i] = c;
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) {
      // over all slices, from the top: lane l has sums 63 - 2 l and 62 - 2 l
      uint2 peer[kMaxCluster];
      uint32_t lo = 0, hi = 0;
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r)
        peer[r] = r < C ? ld_peer2(&coarse[d][kCoarse - 2 - 2 * lane], r) : make_uint2(0u, 0u);
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r) {
        lo += peer[r].x;
        hi += peer[r].y;
      }
      const uint32_t upto = warp_scan(hi + lo);
      const uint32_t at = __ffs(__ballot_sync(0xffffffffu, upto >= ties)) - 1;  // the lane whose sums reach it
      uint32_t above = __shfl_sync(0xffffffffu, upto - hi - lo, at);           // keys in higher bins
      const uint32_t first_sum = __shfl_sync(0xffffffffu, hi, at);
      uint32_t sum_of = kCoarse - 1 - 2 * at;
      if (above + first_sum < ties) {
        above += first_sum;
        --sum_of;
      }
      // its 32 bins, lane l: bin 31 - l
      uint32_t bin[kMaxCluster], count = 0;
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r)
        bin[r] = r < C ? ld_peer(&hist[d][sum_of * 32 + 31 - lane], r) : 0u;
#pragma unroll
      for (uint32_t r = 0; r < kMaxCluster; ++r) count += bin[r];
      const uint32_t within = warp_scan(count);
      const uint32_t l = __ffs(__ballot_sync(0xffffffffu, above + within >= ties)) - 1;
      if (lane == l) {
        found_digit = sum_of * 32 + 31 - lane;
        const uint32_t rank_in = ties - above - (within - count);
        found_rank = rank_in < count ? rank_in : 0;
      }
    }
    __syncthreads();
    last |= found_digit << shift;
    ties = found_rank;
    if (ties == 0) {
      // the whole bin is kept: every key from its first on (last is not 0 here: the
      // least key, -infinity's, is 0x007fffff, so the first digit is 3 or more). Going
      // on instead: 8 x 8 rows of up to 8192 37.3 against 37.0 us, 2 x 8 of 131072
      // 68.7 against 68.4.
      --last;
      break;
    }
  }

  // a thread's run of keys: contiguous, of odd length (no bank conflicts)
  const int run = ((n + kSelectThreads - 1) / kSelectThreads) | 1;
  const int r0 = min(n, tid * run), r1 = min(n, r0 + run);
  uint32_t gt = 0, eq = 0;
  for (int i = r0; i < r1; ++i) {
    const uint32_t key = weight_key_bits(bits_at(i));
    gt += key > last;
    eq += key == last;
  }
  // both counts in one scan: a cached slice has fewer than 2^16 keys
  uint32_t all_gt, all_eq, gt_at, eq_at;
  if constexpr (kCached) {
    uint32_t all;
    const uint32_t upto = block_scan(gt | (eq << 16), warp_sums, &all);
    gt_at = (upto & 0xffffu) - gt;
    eq_at = (upto >> 16) - eq;
    all_gt = all & 0xffffu;
    all_eq = all >> 16;
  } else {
    gt_at = block_scan(gt, warp_sums, &all_gt) - gt;
    eq_at = block_scan(eq, warp_sums, &all_eq) - eq;
  }
  if (tid == 0) {
    slice_counts[0] = all_gt;
    slice_counts[1] = all_eq;
  }
  __syncwarp();
  cluster_sync_all();
  {
    uint2 peer[kMaxCluster];
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; ++r) peer[r] = r < rank ? ld_peer2(slice_counts, r) : make_uint2(0u, 0u);
#pragma unroll
    for (uint32_t r = 0; r < kMaxCluster; ++r) {
      gt_at += peer[r].x;
      eq_at += peer[r].y;
    }
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // no store before this last barrier: its and the earlier ones' releases would wait
  // for them (77 against 70 us for 2 x 8 rows of 131072)
  write_rest();
  for (int i = r0; i < r1; ++i) {
    const uint32_t bits = bits_at(i), key = weight_key_bits(bits);
    if (key > last || (key == last && eq_at < ties)) {
      const uint32_t at = gt_at + min(eq_at, ties);
      kept[at] = first + i;
      nw[at] = __uint_as_float(bits);
    }
    gt_at += key > last;
    eq_at += key == last;
  }
  // a CTA's counts may be read until the others have passed here
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kMoveThreads = 256;
constexpr int kMoveBatch = 4;  // rows of a thread in flight

// One CTA per (rows, key head, sequence); a group of D / 8 threads takes a row.
template <int kChunks>
__global__ void __launch_bounds__(kMoveThreads)
evict_move_kernel(EvictParams p, uint16_t* k_pages, uint16_t* v_pages, unsigned int* err) {
  constexpr int kGroups = kMoveThreads / kChunks;
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int head = blockIdx.y, seq = blockIdx.z;
  const int32_t* kept = p.kept + (static_cast<int64_t>(seq) * p.c.heads + head) * p.budget;
  const int chunk = threadIdx.x % kChunks;
  const int r0 = blockIdx.x * (kGroups * kMoveBatch) + threadIdx.x / kChunks;
  const int slot_mask = (1 << p.c.page_shift) - 1;
  const int32_t* table = p.c.table + static_cast<int64_t>(seq) * p.c.ld_table;
  const int32_t* new_table = p.new_table + static_cast<int64_t>(seq) * p.ld_new_table;
  int64_t from[kMoveBatch], to[kMoveBatch];
  uint4 kk[kMoveBatch], vv[kMoveBatch];
#pragma unroll
  for (int u = 0; u < kMoveBatch; ++u) {
    const int r = r0 + u * kGroups;
    to[u] = -1;
    const int pos = r < p.budget ? kept[r] : -1;
    if (pos < 0) continue;
    const int src = table[pos >> p.c.page_shift], dst = new_table[r >> p.c.page_shift];
    if (!page_ok(src, p.c.num_pages) || !page_ok(dst, p.c.num_pages)) {
      bad_index(err, kSiteBadPage);
      continue;
    }
    from[u] = pool_offset(src, head, pos & slot_mask, p.c.ld_page, p.c.ld_head, p.c.ld_slot) + chunk * 8;
    to[u] = pool_offset(dst, head, r & slot_mask, p.c.ld_page, p.c.ld_head, p.c.ld_slot) + chunk * 8;
  }
#pragma unroll
  for (int u = 0; u < kMoveBatch; ++u) {
    if (to[u] < 0) continue;
    kk[u] = *reinterpret_cast<const uint4*>(k_pages + from[u]);
    vv[u] = *reinterpret_cast<const uint4*>(v_pages + from[u]);
  }
#pragma unroll
  for (int u = 0; u < kMoveBatch; ++u) {
    if (to[u] < 0) continue;
    *reinterpret_cast<uint4*>(k_pages + to[u]) = kk[u];
    *reinterpret_cast<uint4*>(v_pages + to[u]) = vv[u];
  }
}

constexpr int kMaxDevices = 64;

// Launch of the selection by clusters of C CTAs with `smem` bytes each. (Not
// overlapped with the kernel before it: clusters that were placed between that
// one's last CTAs took 6 us longer for 2 x 8 rows of 131072.)
template <bool kCached>
cudaLaunchConfig_t select_config(const EvictParams& p, int C, int smem, cudaStream_t stream, cudaLaunchAttribute (&attr)[1]) {
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.c.heads * C, p.c.batch);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// The kernel's shared-memory limit, raised once per device.
cudaError_t raise_select_smem(int dev) {
  static std::atomic<bool> done[kMaxDevices];
  if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kMaxSliceKeys * 4);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  return e;
}

// Clusters of C CTAs that the device holds at one time with a full slice each
// (one CTA an SM); asked once per device and C.
int resident_clusters(const EvictParams& p, int dev, int C) {
  static std::atomic<int> known[kMaxDevices][kMaxCluster + 1];
  if (dev < 0 || dev >= kMaxDevices) return 0;
  int n = known[dev][C].load(std::memory_order_relaxed);
  if (n > 0) return n;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = select_config<true>(p, C, kMaxSliceKeys * 4, nullptr, attr);
  if (cudaOccupancyMaxActiveClusters(&n, evict_select_kernel<true>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  known[dev][C].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace

PagedCache paged_cache(const os_paged_cache& c) {
  int shift = 0;
  while ((1 << shift) < c.page_size) ++shift;
  return PagedCache{static_cast<const uint16_t*>(c.k_pages), static_cast<const uint16_t*>(c.v_pages),
                    c.ld_page, c.ld_head, c.ld_slot, c.page_table, c.ld_table, c.kv_len,
                    c.num_pages, shift, c.max_pages, c.heads, c.batch};
}

cudaError_t launch_kv_append(const uint16_t* k, const uint16_t* v, int64_t ld_token, int64_t ld_head,
                             int64_t tokens, const int32_t* cu, const os_paged_cache& cache,
                             unsigned int* err, cudaStream_t stream) {
  const int chunks = cache.head_dim / 8;
  const int64_t total = tokens * cache.heads * chunks;
  int64_t blocks = (total + kAppendThreads - 1) / kAppendThreads;
  const int sms = device_sms();
  if (sms < 1) return cudaErrorInvalidDevice;
  if (blocks > sms * 64) blocks = sms * 64;
  return launch_after(kv_append_kernel, dim3(static_cast<unsigned>(blocks)), kAppendThreads, 0, stream, k, v, ld_token,
                      ld_head, tokens, cu, paged_cache(cache), static_cast<uint16_t*>(cache.k_pages),
                      static_cast<uint16_t*>(cache.v_pages), chunks, err);
}

cudaError_t launch_kv_evict(const os_paged_cache& cache, const float* weights, int64_t ld_w_batch,
                            int64_t ld_w_head, const int32_t* new_table, int64_t ld_new_table,
                            int32_t new_max_pages, int32_t budget, int32_t recent, int32_t* kept,
                            int32_t* new_len, float* new_weights, unsigned int* err,
                            cudaStream_t stream) {
  const EvictParams p{paged_cache(cache), weights, ld_w_batch, ld_w_head, new_table, ld_new_table,
                      new_max_pages, budget, recent, kept, new_len, new_weights};
  // CTAs of a row: as many (up to eight) as fit on the GPU for all rows at once while a
  // slice keeps at least kLeastSlice keys, and as many as it takes for a slice
  // to fit shared memory where eight can do that. (16 rows of 131072 keys: clusters of
  // eight do not all fit at once and took 15 us longer than clusters of seven.)
  const int64_t capacity = static_cast<int64_t>(cache.max_pages) * cache.page_size;
  const int64_t rows = static_cast<int64_t>(cache.heads) * cache.batch;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if ((e = raise_select_smem(dev)) != cudaSuccess) return e;
  int C = 1;
  while (C < kMaxCluster && (capacity > static_cast<int64_t>(C) * kMaxSliceKeys ||
                             (capacity >= static_cast<int64_t>(C + 1) * kLeastSlice && rows <= resident_clusters(p, dev, C + 1))))
    ++C;
  const int64_t slice = (capacity + C - 1) / C;
  cudaLaunchAttribute attr[1];
  if (slice <= kMaxSliceKeys) {
    const cudaLaunchConfig_t cfg = select_config<true>(p, C, static_cast<int>(slice) * 4, stream, attr);
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel<true>, p);
  } else {
    const cudaLaunchConfig_t cfg = select_config<false>(p, C, 0, stream, attr);
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel<false>, p);
  }
  if (e != cudaSuccess) return e;
  const int chunks = cache.head_dim / 8, rows_per_cta = kMoveThreads / chunks * kMoveBatch;
  const dim3 grid((budget + rows_per_cta - 1) / rows_per_cta, cache.heads, cache.batch);
  uint16_t *k = static_cast<uint16_t*>(cache.k_pages), *v = static_cast<uint16_t*>(cache.v_pages);
  return chunks == 16 ? launch_after(evict_move_kernel<16>, grid, kMoveThreads, 0, stream, p, k, v, err)
                      : launch_after(evict_move_kernel<8>, grid, kMoveThreads, 0, stream, p, k, v, err);
}

}  // namespace oss
