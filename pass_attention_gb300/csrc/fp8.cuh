// The 8-bit cache's number format for the kernels: rows of e4m3 values with one
// power-of-two scale, and conversions between them and 16 bits.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "device_common.cuh"
#include "paged.h"

namespace oss {

// Pools of an os_paged_cache_fp8 beside its tables: values with the PagedCache's strides,
// scales [page, head, slot] with unit stride over the slots.
struct Fp8Pools {
  uint8_t *k, *v, *k_scales, *v_scales;
  int64_t ld_page, ld_head;  // of the scales
};

// Two 16-bit values of one word, widened.
template <bool kF16>
__device__ __forceinline__ float2 widen2(uint32_t w) {
  if constexpr (kF16)
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else
    return make_float2(bf16_lo(w), bf16_hi(w));
}

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t w;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(w) : "f"(hi), "f"(lo));
  return w;
}

// Two e4m3 values (the low half of w) as two fp16 ones: exact.
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t w) {
  uint32_t x;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"(static_cast<uint16_t>(w)));
  return x;
}

__device__ __forceinline__ float fp8_scale_value(uint32_t byte) { return __uint_as_float(fp8_scale_bits(byte)); }

}  // namespace oss
