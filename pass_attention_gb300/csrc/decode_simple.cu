// Attention of one new token per sequence, in the simplest form: over a cache in 8 bits, and
// over a 16-bit cache behind prefixes that groups of sequences share.
//
// One CTA a query head; its four warps take the keys in turn, lanes over the dims,
// each with its own running maximum, sum and output, which meet at the end.

#include <cstdint>

#include "device_common.cuh"
#include "fp8.cuh"
#include "launch.cuh"
#include "oss_internal.h"
#include "paged.h"

namespace oss {
namespace {

constexpr int kWarps = 4;
constexpr float kLn2 = 0.69314718055994530942f;

struct Params {
  PagedCache c;
  Fp8Pools f;
  PrefixTables prefix;  // groups 0: none
  const uint16_t* q;
  int64_t ld_q_batch, ld_q_head;
  int32_t H;
  float scale2;
  uint16_t* o;
  float* lse;
  unsigned int* err;
};

__device__ __forceinline__ float reference(float m) { return m == neg_inf() ? 0.f : m; }

template <bool kF16, int D, bool kFp8>
__global__ void __launch_bounds__(kWarps * 32) decode_simple_kernel(const Params p) {
  constexpr int kDims = D / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int h = blockIdx.x, b = blockIdx.y, g = h / (p.H / p.c.heads);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d0 = lane * kDims;
  auto widen = [](const uint16_t* x, float (&y)[kDims]) {
#pragma unroll
    for (int i = 0; i < kDims; i += 2) {
      const float2 w = widen2<kF16>(*reinterpret_cast<const uint32_t*>(x + i));
      y[i] = w.x;
      y[i + 1] = w.y;
    }
  };
  auto widen8 = [](const uint8_t* x, float s, float (&y)[kDims]) {
#pragma unroll
    for (int i = 0; i < kDims; i += 2) {
      const float2 w = widen2<true>(from_e4m3x2(*reinterpret_cast<const uint16_t*>(x + i)));
      y[i] = w.x * s;
      y[i + 1] = w.y * s;
    }
  };
  float q[kDims], m = neg_inf(), l = 0.f, acc[kDims];
  widen(p.q + b * p.ld_q_batch + h * p.ld_q_head + d0, q);
#pragma unroll
  for (int i = 0; i < kDims; ++i) acc[i] = 0.f;
  auto walk = [&](const int32_t* table, int32_t len) {
    for (int t = warp; t < len; t += kWarps) {
      const int page = table[t >> p.c.page_shift];
      if (!page_ok(page, p.c.num_pages)) {
        report_error(p.err, kKernelPaged | (kSiteBadPage << 8));
        continue;
      }
      const int slot = t & ((1 << p.c.page_shift) - 1);
      const int64_t at = pool_offset(page, g, slot, p.c.ld_page, p.c.ld_head, p.c.ld_slot) + d0;
      float k[kDims], v[kDims];
      if constexpr (kFp8) {
        const int64_t sc = pool_offset(page, g, slot, p.f.ld_page, p.f.ld_head, 1);
        widen8(p.f.k + at, fp8_scale_value(p.f.k_scales[sc]), k);
        widen8(p.f.v + at, fp8_scale_value(p.f.v_scales[sc]), v);
      } else {
        widen(p.c.k + at, k);
        widen(p.c.v + at, v);
      }
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kDims; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s *= p.scale2;
      const float to = fmaxf(m, s), ref = reference(to), corr = ex2(m - ref), w = ex2(s - ref);
      m = to;
      l = fmaf(l, corr, w);
#pragma unroll
      for (int i = 0; i < kDims; ++i) acc[i] = fmaf(v[i], w, acc[i] * corr);
    }
  };
  if (p.prefix.groups > 0) {
    if (p.prefix.cu && blockIdx.x == 0 && blockIdx.y == 0)
      for (int i = threadIdx.x; i < p.prefix.groups; i += kWarps * 32)
        if (row_range(p.prefix.cu[i], p.prefix.cu[i + 1], p.c.batch).clamped)
          report_error(p.err, kKernelPaged | (kSiteBadOffsets << 8));
    const int32_t group = prefix_group(p.prefix, b);
    if (group >= 0)
      walk(p.prefix.table + group * p.prefix.ld_table,
           paged_length(p.prefix.len[group], p.prefix.max_pages, p.c.page_shift));
  }
  walk(p.c.table + b * p.c.ld_table, paged_length(p.c.kv_len[b], p.c.max_pages, p.c.page_shift));
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < kDims; ++i) so[warp][d0 + i] = acc[i];
  __syncthreads();
  if (threadIdx.x >= D / 2) return;
  float M = neg_inf(), L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sm[i]);
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const float f = ex2(sm[i] - reference(M));
    L = fmaf(sl[i], f, L);
    x = fmaf(so[i][2 * threadIdx.x], f, x);
    y = fmaf(so[i][2 * threadIdx.x + 1], f, y);
  }
  const int64_t row = static_cast<int64_t>(b) * p.H + h;
  const float inv = L != 0.f ? 1.f / L : 0.f;
  reinterpret_cast<uint32_t*>(p.o + row * D)[threadIdx.x] = pack2<kF16>(x * inv, y * inv);
  if (threadIdx.x == 0 && p.lse) p.lse[row] = L != 0.f ? (M + log2f(L)) * kLn2 : neg_inf();
}

template <bool kFp8>
cudaError_t launch(const Params& p, bool f16, int D, cudaStream_t stream) {
  const dim3 grid(p.H, p.c.batch);
  const auto go = [&](auto* kernel) { return launch_after(kernel, grid, kWarps * 32, 0, stream, p); };
  if (f16) return D == 128 ? go(decode_simple_kernel<true, 128, kFp8>) : go(decode_simple_kernel<true, 64, kFp8>);
  return D == 128 ? go(decode_simple_kernel<false, 128, kFp8>) : go(decode_simple_kernel<false, 64, kFp8>);
}

float base2(float scale) { return static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074); }

}  // namespace

int64_t decode_shared_workspace_bytes(int, const os_paged_cache&, int, int) { return 16; }

cudaError_t launch_decode_shared(const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head, int H,
                                 const os_paged_cache& cache, const PrefixTables& prefix, float scale, uint16_t* o,
                                 float* lse, void*, unsigned int* err, const AttnFault&, cudaStream_t stream) {
  const Params p{paged_cache(cache), Fp8Pools{}, prefix, q, ld_q_batch, ld_q_head, H, base2(scale), o, lse, err};
  return launch<false>(p, cache.dtype == OS_DTYPE_F16, cache.head_dim, stream);
}

}  // namespace oss
