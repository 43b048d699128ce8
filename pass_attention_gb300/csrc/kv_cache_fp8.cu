// The paged key-value cache in 8 bits: appending new tokens, and reading them back.
//
// A row (a token's key or value in one key head) is D e4m3 values and one
// power-of-two scale 2^e, e the smallest integer >= -127 with max |x| <= 448 * 2^e (448 is
// e4m3's largest value), stored as the byte e + 127 (e8m0; 255 is NaN). Dividing by a
// power of two is exact, so the only rounding is the one to e4m3, and the codes do not
// depend on how a division rounds. A scale that is no power of two would buy
// nothing: e4m3 is a floating format, and its values' relative error is the same
// anywhere between 448 and 2^-6.
//
// Both are copies bound by HBM: 2 D and D + 1 bytes a row on either side.

#include <cstdint>

#include "device_common.cuh"
#include "fp8.cuh"
#include "launch.cuh"
#include "oss_internal.h"
#include "paged.h"

namespace oss {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void bad_index(unsigned int* err, unsigned int site) {
  report_error(err, kKernelPaged | (site << 8));
}

// Offsets that do not fit the rows: tokens that kv_len counts have no row.
__device__ __forceinline__ void check_offsets(const int32_t* cu, int32_t batch, int64_t tokens, unsigned int* err) {
  for (int b = blockIdx.x * kThreads + threadIdx.x; b < batch; b += gridDim.x * kThreads)
    if (row_range(cu[b], cu[b + 1], static_cast<int32_t>(tokens)).clamped) bad_index(err, kSiteBadOffsets);
}

// Page and slot of packed row `token` (cu null: the last token of sequence `token`);
// false for a row without one.
__device__ __forceinline__ bool locate(int32_t token, const int32_t* cu, const PagedCache& c, int* page,
                                       int* slot, unsigned int* err) {
  int seq = token;
  int64_t behind = 1;  // tokens of the sequence from this one on
  if (cu) {
    seq = sequence_of(token, cu, c.batch);
    if (seq < 0) return false;  // a row of no sequence
    behind = cu[seq + 1] - token;
  }
  const int32_t len = c.kv_len[seq];
  if (!cu && len == 0) return false;  // an empty place of the batch
  const int64_t pos = len - behind;
  if (pos < 0 || (pos >> c.page_shift) >= c.max_pages) {
    bad_index(err, kSiteBadPosition);
    return false;
  }
  *page = c.table[static_cast<int64_t>(seq) * c.ld_table + (pos >> c.page_shift)];
  if (!page_ok(*page, c.num_pages)) {
    bad_index(err, kSiteBadPage);
    return false;
  }
  *slot = static_cast<int>(pos) & ((1 << c.page_shift) - 1);
  return true;
}

// The larger of two pairs of 16-bit magnitudes.
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// A thread has 16 values of a row: 8 in each half of it, so that neighbours' loads and
// stores of 16 and 8 bytes lie side by side.
struct Chunk {
  uint4 a, b;
  __device__ __forceinline__ uint32_t word(int i) const {
    return i == 0 ? a.x : i == 1 ? a.y : i == 2 ? a.z : i == 3 ? a.w : i == 4 ? b.x : i == 5 ? b.y : i == 6 ? b.z : b.w;
  }
};

// (half: elements from one half of the row to the other)
__device__ __forceinline__ Chunk load_chunk(const uint16_t* p, int half) {
  return Chunk{*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + half)};
}

// Codes of this thread's 16 values and the scale of the row that kLanes threads hold.
template <bool kF16, int kLanes>
__device__ __forceinline__ uint4 quantise(const Chunk& x, uint32_t lanes, uint32_t* scale) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max_pair(top, x.word(i) & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
#pragma unroll
  for (int off = 1; off < kLanes; off <<= 1) top = max(top, __shfl_xor_sync(lanes, top, off));
  const uint32_t s = fp8_scale_byte(__float_as_uint(widen2<kF16>(top).x));
  *scale = s;
  // a row with NaN or infinity reads as NaN
  if (s == kFp8ScaleNan) return make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
  const float down = __uint_as_float((254u - s) << 23);  // 2^-e
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = widen2<kF16>(x.word(2 * i)), hi = widen2<kF16>(x.word(2 * i + 1));
    w[i] = to_e4m3x2(lo.x * down, lo.y * down) | (to_e4m3x2(hi.x * down, hi.y * down) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a thread works on: kHeads heads of a token, from `head` on, 16 values of each.
template <int kLanes, int kHeads>
struct Piece {
  int32_t token;
  int head, part;
  __device__ __forceinline__ Piece(int64_t i, int heads) {
    const int groups = (heads + kHeads - 1) / kHeads;
    part = static_cast<int>(threadIdx.x % kLanes);
    const uint64_t g = static_cast<uint64_t>(i) / kLanes;
    // (a 64-bit division is a hundred instructions)
    token = static_cast<int32_t>(g >> 32 ? g / groups : static_cast<uint32_t>(g) / static_cast<uint32_t>(groups));
    head = static_cast<int>(g - static_cast<uint64_t>(token) * groups) * kHeads;
  }
  __device__ __forceinline__ static int64_t count(int64_t tokens, int heads) {
    return tokens * ((heads + kHeads - 1) / kHeads) * kLanes;
  }
};

// D / 16 threads a row.
template <bool kF16, int kLanes, int kHeads>
__global__ void __launch_bounds__(kThreads)
kv_append_fp8_kernel(const uint16_t* k, const uint16_t* v, int64_t ld_token, int64_t ld_head,
                     int64_t tokens, const int32_t* cu, PagedCache c, Fp8Pools f, unsigned int* err) {
  using Piece = Piece<kLanes, kHeads>;
  constexpr int kHalf = kLanes * 8;
  let_next_kernel_start();
  wait_for_previous_kernel();
  if (cu) check_offsets(cu, c.batch, tokens, err);
  const uint32_t lanes = ((1u << kLanes) - 1) << (threadIdx.x & 31 & ~(kLanes - 1));  // of this row, in the warp
  const int64_t count = Piece::count(tokens, c.heads);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < count;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const Piece t(i, c.heads);
    const int64_t from = t.token * ld_token + t.head * ld_head + t.part * 8;
    Chunk kx[kHeads], vx[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (t.head + h >= c.heads) continue;
      kx[h] = load_chunk(k + from + h * ld_head, kHalf);
      vx[h] = load_chunk(v + from + h * ld_head, kHalf);
    }
    int page, slot;
    if (!locate(t.token, cu, c, &page, &slot, err)) continue;  // the same for all threads of the row
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (t.head + h >= c.heads) continue;
      uint32_t ks, vs;
      const uint4 kc = quantise<kF16, kLanes>(kx[h], lanes, &ks), vc = quantise<kF16, kLanes>(vx[h], lanes, &vs);
      const int64_t to = pool_offset(page, t.head + h, slot, c.ld_page, c.ld_head, c.ld_slot) + t.part * 8;
      *reinterpret_cast<uint2*>(f.k + to) = make_uint2(kc.x, kc.y);
      *reinterpret_cast<uint2*>(f.k + to + kHalf) = make_uint2(kc.z, kc.w);
      *reinterpret_cast<uint2*>(f.v + to) = make_uint2(vc.x, vc.y);
      *reinterpret_cast<uint2*>(f.v + to + kHalf) = make_uint2(vc.z, vc.w);
      if (t.part == 0) {
        const int64_t at = pool_offset(page, t.head + h, slot, f.ld_page, f.ld_head, 1);
        f.k_scales[at] = static_cast<uint8_t>(ks);
        f.v_scales[at] = static_cast<uint8_t>(vs);
      }
    }
  }
}

// Eight values of a row.
template <bool kF16>
__device__ __forceinline__ uint4 values(uint2 codes, float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = widen2<true>(from_e4m3x2((i < 2 ? codes.x : codes.y) >> (16 * (i & 1))));
    w[i] = pack2<kF16>(x.x * scale, x.y * scale);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool kF16, int kLanes, int kHeads>
__global__ void __launch_bounds__(kThreads)
kv_read_fp8_kernel(PagedCache c, Fp8Pools f, const int32_t* cu, int64_t tokens, uint16_t* k,
                   uint16_t* v, int64_t ld_token, int64_t ld_head, unsigned int* err) {
  using Piece = Piece<kLanes, kHeads>;
  constexpr int kHalf = kLanes * 8;
  let_next_kernel_start();
  wait_for_previous_kernel();
  check_offsets(cu, c.batch, tokens, err);
  const int64_t count = Piece::count(tokens, c.heads);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < count;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const Piece t(i, c.heads);
    int page, slot;
    if (!locate(t.token, cu, c, &page, &slot, err)) continue;
    uint2 kc[kHeads][2], vc[kHeads][2];
    uint32_t ks[kHeads], vs[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (t.head + h >= c.heads) continue;
      const int64_t from = pool_offset(page, t.head + h, slot, c.ld_page, c.ld_head, c.ld_slot) + t.part * 8;
      const int64_t at = pool_offset(page, t.head + h, slot, f.ld_page, f.ld_head, 1);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        kc[h][e] = *reinterpret_cast<const uint2*>(f.k + from + e * kHalf);
        vc[h][e] = *reinterpret_cast<const uint2*>(f.v + from + e * kHalf);
      }
      ks[h] = f.k_scales[at];
      vs[h] = f.v_scales[at];
    }
    const int64_t to = t.token * ld_token + t.head * ld_head + t.part * 8;
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (t.head + h >= c.heads) continue;
      const float ky = fp8_scale_value(ks[h]), vy = fp8_scale_value(vs[h]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        *reinterpret_cast<uint4*>(k + to + h * ld_head + e * kHalf) = values<kF16>(kc[h][e], ky);
        *reinterpret_cast<uint4*>(v + to + h * ld_head + e * kHalf) = values<kF16>(vc[h][e], vy);
      }
    }
  }
}

// Heads of a thread, and CTAs (at most 64 an SM, whose threads go on). With two heads a
// thread looks its token's place up once for both and has two rows on their way: 37 k
// tokens, 8 heads of 128, read in 37.7 us against 40.6 with one head and 38.4 with four, written in
// 39.4 against 43.0 and 41.8 (four take its registers). With rows for less than the GPU's
// threads, one head a thread is as fast (64 rows of 8 heads: 3.3 us).
constexpr int kManyHeads = 2;

bool many_rows(int64_t rows, int lanes, int sms) { return rows * lanes > static_cast<int64_t>(sms) * 2048; }

unsigned copy_blocks(int64_t tokens, int heads, int lanes, bool many, int sms) {
  const int64_t groups = many ? (heads + kManyHeads - 1) / kManyHeads : heads;
  const int64_t n = (tokens * groups * lanes + kThreads - 1) / kThreads, most = static_cast<int64_t>(sms) * 64;
  return static_cast<unsigned>(n < most ? n : most);
}

}  // namespace

Fp8Pools fp8_pools(const os_paged_cache_fp8& c) {
  return Fp8Pools{static_cast<uint8_t*>(c.pages.k_pages), static_cast<uint8_t*>(c.pages.v_pages),
                  static_cast<uint8_t*>(c.k_scales), static_cast<uint8_t*>(c.v_scales), c.ld_scale_page, c.ld_scale_head};
}

cudaError_t launch_kv_append_fp8(const uint16_t* k, const uint16_t* v, int64_t ld_token, int64_t ld_head, int64_t tokens,
                                 const int32_t* cu, const os_paged_cache_fp8& cache, unsigned int* err,
                                 cudaStream_t stream) {
  const int sms = device_sms();
  if (sms < 1) return cudaErrorInvalidDevice;
  const int lanes = cache.pages.head_dim / 16, heads = cache.pages.heads;
  const bool many = many_rows(tokens * heads, lanes, sms), f16 = cache.pages.dtype == OS_DTYPE_F16;
  const dim3 grid(copy_blocks(tokens, heads, lanes, many, sms));
  const PagedCache c = paged_cache(cache.pages);
  const Fp8Pools f = fp8_pools(cache);
  const auto launch = [&](auto* kernel) {
    return launch_after(kernel, grid, kThreads, 0, stream, k, v, ld_token, ld_head, tokens, cu, c, f, err);
  };
  if (many) {
    if (lanes == 8) return f16 ? launch(kv_append_fp8_kernel<true, 8, kManyHeads>) : launch(kv_append_fp8_kernel<false, 8, kManyHeads>);
    return f16 ? launch(kv_append_fp8_kernel<true, 4, kManyHeads>) : launch(kv_append_fp8_kernel<false, 4, kManyHeads>);
  }
  if (lanes == 8) return f16 ? launch(kv_append_fp8_kernel<true, 8, 1>) : launch(kv_append_fp8_kernel<false, 8, 1>);
  return f16 ? launch(kv_append_fp8_kernel<true, 4, 1>) : launch(kv_append_fp8_kernel<false, 4, 1>);
}

cudaError_t launch_kv_read_fp8(const os_paged_cache_fp8& cache, const int32_t* cu, int64_t tokens, uint16_t* k,
                               uint16_t* v, int64_t ld_token, int64_t ld_head, unsigned int* err, cudaStream_t stream) {
  const int sms = device_sms();
  if (sms < 1) return cudaErrorInvalidDevice;
  const int lanes = cache.pages.head_dim / 16, heads = cache.pages.heads;
  const bool many = many_rows(tokens * heads, lanes, sms), f16 = cache.pages.dtype == OS_DTYPE_F16;
  const dim3 grid(copy_blocks(tokens, heads, lanes, many, sms));
  const PagedCache c = paged_cache(cache.pages);
  const Fp8Pools f = fp8_pools(cache);
  const auto launch = [&](auto* kernel) {
    return launch_after(kernel, grid, kThreads, 0, stream, c, f, cu, tokens, k, v, ld_token, ld_head, err);
  };
  if (many) {
    if (lanes == 8) return f16 ? launch(kv_read_fp8_kernel<true, 8, kManyHeads>) : launch(kv_read_fp8_kernel<false, 8, kManyHeads>);
    return f16 ? launch(kv_read_fp8_kernel<true, 4, kManyHeads>) : launch(kv_read_fp8_kernel<false, 4, kManyHeads>);
  }
  if (lanes == 8) return f16 ? launch(kv_read_fp8_kernel<true, 8, 1>) : launch(kv_read_fp8_kernel<false, 8, 1>);
  return f16 ? launch(kv_read_fp8_kernel<true, 4, 1>) : launch(kv_read_fp8_kernel<false, 4, 1>);
}

}  // namespace oss
