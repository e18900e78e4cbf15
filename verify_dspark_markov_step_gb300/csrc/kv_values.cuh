// kv_values.cuh -- 16- and 8-bit values of rows and caches.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dspark {

__device__ __forceinline__ float half_bits_to_float(uint32_t bits) {
  float f;
  asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.f32.f16 %0, h; }" : "=f"(f) : "r"(bits));
  return f;
}

// Two values to 8 bits, nearest even, clamped to the largest finite value,
// NaN kept; `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint32_t r;
  asm("{ .reg .b16 h; cvt.rn.satfinite.e4m3x2.f32 h, %1, %2; cvt.u32.u16 %0, h; }"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

template <bool kF16>
__device__ __forceinline__ void unpack(uint32_t w, float& a, float& b) {
  if constexpr (kF16) {
    a = half_bits_to_float(w & 0xFFFFu);
    b = half_bits_to_float(w >> 16);
  } else {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  }
}

// Two values to 16 bits, nearest even; `lo` in the low half.
template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (kF16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace dspark
