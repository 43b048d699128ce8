// Attention forward over packed sequences, grouped key heads.
//
// One warp per (query token, query head); lanes hold the head dims, and the
// online-softmax recurrence runs key by key.

#include <cstdint>

#include "device_common.cuh"
#include "oss_internal.h"
#include "paged.h"

namespace oss {
namespace {

constexpr int kThreads = 256;
constexpr float kLn2 = 0.69314718055994530942f;

struct PackedParams {
  const uint16_t *q, *k, *v;
  int64_t ld_q_token, ld_q_head, ld_kv_token, ld_kv_head;
  uint16_t* o;
  float* lse;
  const int32_t *cu_q, *cu_k;
  int32_t batch, tokens_q, tokens_k, Hq, Hkv;
  float scale2;
  int causal;
  unsigned int* err;
};

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

template <bool kF16, int D>
__global__ void __launch_bounds__(kThreads) attn_packed_kernel(PackedParams p) {
  constexpr int W = D / 64;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.batch; b += kThreads)
      if (row_range(p.cu_q[b], p.cu_q[b + 1], p.tokens_q).clamped ||
          row_range(p.cu_k[b], p.cu_k[b + 1], p.tokens_k).clamped)
        report_error(p.err, kKernelPaged | (kSiteBadOffsets << 8));
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  if (row >= static_cast<int64_t>(p.tokens_q) * p.Hq) return;
  const int64_t token = row / p.Hq;
  const int h = static_cast<int>(row - token * p.Hq);
  const int seq = sequence_of(token, p.cu_q, p.batch);
  if (seq < 0) return;
  const RowRange rq = row_range(p.cu_q[seq], p.cu_q[seq + 1], p.tokens_q);
  const RowRange rk = row_range(p.cu_k[seq], p.cu_k[seq + 1], p.tokens_k);
  const int64_t i = token - rq.start;
  int64_t n = rk.len;
  if (p.causal && i + rk.len - rq.len + 1 < n) n = i + rk.len - rq.len + 1;
  float2 q[W], o[W];
  for (int w = 0; w < W; ++w) {
    q[w] = unpack2<kF16>(reinterpret_cast<const uint32_t*>(p.q + token * p.ld_q_token + h * p.ld_q_head)[lane + 32 * w]);
    q[w].x *= p.scale2;
    q[w].y *= p.scale2;
    o[w] = make_float2(0.f, 0.f);
  }
  const int g = h / (p.Hq / p.Hkv);
  float m = neg_inf(), l = 0.f;
  for (int64_t j = 0; j < n; ++j) {
    const int64_t at = (rk.start + j) * p.ld_kv_token + g * p.ld_kv_head;
    float s = 0.f;
    for (int w = 0; w < W; ++w) {
      const float2 kk = unpack2<kF16>(reinterpret_cast<const uint32_t*>(p.k + at)[lane + 32 * w]);
      s = fmaf(q[w].x, kk.x, fmaf(q[w].y, kk.y, s));
    }
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float mn = fmaxf(m, s), corr = ex2(m - mn), e = ex2(s - mn);
    m = mn;
    l = fmaf(l, corr, e);
    for (int w = 0; w < W; ++w) {
      const float2 vv = unpack2<kF16>(reinterpret_cast<const uint32_t*>(p.v + at)[lane + 32 * w]);
      o[w].x = fmaf(o[w].x, corr, e * vv.x);
      o[w].y = fmaf(o[w].y, corr, e * vv.y);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int w = 0; w < W; ++w) {
    uint32_t r;
    if constexpr (kF16)
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(o[w].y * inv), "f"(o[w].x * inv));
    else
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(o[w].y * inv), "f"(o[w].x * inv));
    reinterpret_cast<uint32_t*>(p.o + row * D)[lane + 32 * w] = r;
  }
  if (lane == 0 && p.lse) p.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : neg_inf();
}

}  // namespace

int64_t attn_packed_workspace_bytes(int batch, int64_t tokens_q, int Hq, int Hkv) {
  (void)batch; (void)tokens_q; (void)Hq; (void)Hkv;
  return 16;
}

cudaError_t launch_attn_packed(const PackedArgs& a, void* workspace, unsigned int* err,
                               const AttnFault& fault, cudaStream_t stream) {
  (void)workspace;
  (void)fault;
  const PackedParams p{a.q, a.k, a.v, a.ld_q_token, a.ld_q_head, a.ld_kv_token, a.ld_kv_head, a.o, a.lse,
                       a.cu_q, a.cu_k, a.batch, static_cast<int32_t>(a.tokens_q), static_cast<int32_t>(a.tokens_k),
                       a.Hq, a.Hkv, static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634074),
                       a.causal, err};
  const unsigned blocks = static_cast<unsigned>((a.tokens_q * a.Hq + 7) / 8);
  if (a.D == 128) {
    if (a.f16) attn_packed_kernel<true, 128><<<blocks, kThreads, 0, stream>>>(p);
    else attn_packed_kernel<false, 128><<<blocks, kThreads, 0, stream>>>(p);
  } else {
    if (a.f16) attn_packed_kernel<true, 64><<<blocks, kThreads, 0, stream>>>(p);
    else attn_packed_kernel<false, 64><<<blocks, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace oss
