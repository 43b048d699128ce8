// Attention of one new token per sequence over a paged key-value cache.
//
// One CTA per (key head, sequence): for each query head of the group, warps
// take the keys in turn, lanes the head dims, and the warps' running (m, l, O)
// are merged in a fixed order. With weights, a second sweep adds exp(s - lse).

#include <cstdint>

#include "device_common.cuh"
#include "oss_internal.h"
#include "paged.h"

namespace oss {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLn2 = 0.69314718055994530942f;

template <bool kF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (kF16) {
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi) : "r"(w));
    return make_float2(lo, hi);
  } else {
    return make_float2(bf16_lo(w), bf16_hi(w));
  }
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

struct DecodeParams {
  PagedCache c;
  const uint16_t* q;
  int64_t ld_q_batch, ld_q_head;
  int32_t H;
  float scale2;  // scale * log2(e)
  uint16_t* o;
  float* lse;
  float* weights;
  int64_t ld_w_batch, ld_w_head;
  unsigned int* err;
};

template <bool kF16, int D>
__global__ void __launch_bounds__(kThreads) decode_paged_kernel(DecodeParams p) {
  constexpr int W = D / 64;  // 32-bit words (pairs of dims) of a row that a lane holds
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int g = blockIdx.x, seq = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = p.H / p.c.heads;
  const int len = paged_length(p.c.kv_len[seq], p.c.max_pages, p.c.page_shift);
  const int32_t* table = p.c.table + static_cast<int64_t>(seq) * p.c.ld_table;
  const int slot_mask = (1 << p.c.page_shift) - 1;
  for (int hh = 0; hh < group; ++hh) {
    const int h = g * group + hh;
    float2 q[W];
    for (int i = 0; i < W; ++i) {
      q[i] = unpack2<kF16>(reinterpret_cast<const uint32_t*>(
          p.q + seq * p.ld_q_batch + h * p.ld_q_head)[lane + 32 * i]);
      q[i].x *= p.scale2;
      q[i].y *= p.scale2;
    }
    auto score = [&](int t, int64_t* at) -> float {
      const int page = table[t >> p.c.page_shift];
      if (!page_ok(page, p.c.num_pages)) {
        report_error(p.err, kKernelPaged | (kSiteBadPage << 8));
        return neg_inf();
      }
      *at = pool_offset(page, g, t & slot_mask, p.c.ld_page, p.c.ld_head, p.c.ld_slot);
      float s = 0.f;
      for (int i = 0; i < W; ++i) {
        const float2 kk = unpack2<kF16>(reinterpret_cast<const uint32_t*>(p.c.k + *at)[lane + 32 * i]);
        s = fmaf(q[i].x, kk.x, fmaf(q[i].y, kk.y, s));
      }
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      return s;
    };
    float m = neg_inf(), l = 0.f;
    float2 o[W];
    for (int i = 0; i < W; ++i) o[i] = make_float2(0.f, 0.f);
    for (int t = warp; t < len; t += kWarps) {
      int64_t at = 0;
      const float s = score(t, &at);
      if (s == neg_inf()) continue;
      const float mn = fmaxf(m, s), corr = ex2(m - mn), w = ex2(s - mn);
      m = mn;
      l = fmaf(l, corr, w);
      for (int i = 0; i < W; ++i) {
        const float2 vv = unpack2<kF16>(reinterpret_cast<const uint32_t*>(p.c.v + at)[lane + 32 * i]);
        o[i].x = fmaf(o[i].x, corr, w * vv.x);
        o[i].y = fmaf(o[i].y, corr, w * vv.y);
      }
    }
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    for (int i = 0; i < W; ++i) {
      so[warp][2 * (lane + 32 * i)] = o[i].x;
      so[warp][2 * (lane + 32 * i) + 1] = o[i].y;
    }
    __syncthreads();
    float M = neg_inf(), L = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    if (M != neg_inf())
      for (int w = 0; w < kWarps; ++w) L += sl[w] * ex2(sm[w] - M);
    const int64_t row = static_cast<int64_t>(seq) * p.H + h;
    const float lse2 = L > 0.f ? M + log2f(L) : neg_inf();
    if (threadIdx.x < D / 2) {
      float2 acc = make_float2(0.f, 0.f);
      if (L > 0.f) {
        for (int w = 0; w < kWarps; ++w) {
          const float f = ex2(sm[w] - M);
          acc.x += f * so[w][2 * threadIdx.x];
          acc.y += f * so[w][2 * threadIdx.x + 1];
        }
        acc.x /= L;
        acc.y /= L;
      }
      reinterpret_cast<uint32_t*>(p.o + row * D)[threadIdx.x] = pack2<kF16>(acc.x, acc.y);
    }
    if (threadIdx.x == 0 && p.lse) p.lse[row] = L > 0.f ? lse2 * kLn2 : neg_inf();
    if (p.weights && L > 0.f) {
      float* wt = p.weights + seq * p.ld_w_batch + g * p.ld_w_head;
      for (int t = warp; t < len; t += kWarps) {
        int64_t at = 0;
        const float s = score(t, &at);
        if (lane == 0) wt[t] += ex2(s - lse2);
      }
    }
    __syncthreads();
  }
}

}  // namespace

int64_t decode_paged_workspace_bytes(int H, const os_paged_cache& cache, bool weights) {
  (void)H; (void)cache; (void)weights;
  return 16;
}

cudaError_t launch_decode_paged(const uint16_t* q, int64_t ld_q_batch, int64_t ld_q_head, int H,
                                const os_paged_cache& cache, float scale, uint16_t* o, float* lse,
                                float* weights, int64_t ld_w_batch, int64_t ld_w_head,
                                void* workspace, unsigned int* err, cudaStream_t stream) {
  (void)workspace;
  const DecodeParams p{paged_cache(cache), q, ld_q_batch, ld_q_head, H,
                       static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074),
                       o, lse, weights, ld_w_batch, ld_w_head, err};
  const dim3 grid(cache.heads, cache.batch);
  const bool f16 = cache.dtype == OS_DTYPE_F16;
  if (cache.head_dim == 128) {
    if (f16) decode_paged_kernel<true, 128><<<grid, kThreads, 0, stream>>>(p);
    else decode_paged_kernel<false, 128><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (f16) decode_paged_kernel<true, 64><<<grid, kThreads, 0, stream>>>(p);
    else decode_paged_kernel<false, 64><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace oss
