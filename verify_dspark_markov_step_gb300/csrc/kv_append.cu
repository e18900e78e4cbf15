// kv_append.cu -- the keys and values of new tokens into their pages.
//
// A copy with an address per token: 16 bytes (8 values) of a key or value row
// per thread, read from the tokens' side (which may be a view into a fused
// projection) and written into the page, as they are or divided by the
// head's scale and rounded to 8 bits. Bound by memory for long prompts (each
// value read once and written once), by latency for a decode step.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "paged.h"

namespace dspark {

namespace {

constexpr int kThreads = 256;

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
__device__ __forceinline__ uint32_t quantise_pair(uint32_t w, float scale) {
  float a, b;
  if constexpr (kF16) {
    a = half_bits_to_float(w & 0xFFFFu);
    b = half_bits_to_float(w >> 16);
  } else {
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xFFFF0000u);
  }
  return e4m3_pair(__fdiv_rn(a, scale), __fdiv_rn(b, scale));
}

template <bool kQuantise, bool kF16>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(KvAppendParams P) {
  const int chunks = P.H * P.D / 8;  // 16-byte pieces of a token's keys (or values)
  const int64_t n = static_cast<int64_t>(P.T) * 2 * chunks;
  const int cd = P.D / 8;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int t = static_cast<int>(i / (2 * chunks));
    int c = static_cast<int>(i - static_cast<int64_t>(t) * 2 * chunks);
    const int which = c >= chunks ? 1 : 0;  // keys, then values
    c -= which * chunks;
    const int64_t slot = P.slot_map[t];
    if (slot < 0) continue;
    if (slot >= P.num_slots) {
      report(P.status, DSPARK_ERR_BOUNDS);
      continue;
    }
    const int h = c / cd, d = (c - h * cd) * 8;
    const uint16_t* src = static_cast<const uint16_t*>(P.src[which]) +
                          static_cast<int64_t>(t) * P.src_stride[which] + c * 8;
    const uint4 x = *reinterpret_cast<const uint4*>(src);
    const int64_t at = (slot >> P.page_shift) * P.block_stride[which] + h * P.head_stride[which] +
                       (slot & ((1 << P.page_shift) - 1)) * P.token_stride[which] + d;
    if constexpr (kQuantise) {
      const float s = P.scale[which] ? P.scale[which][h] : 1.f;
      const uint32_t lo = quantise_pair<kF16>(x.x, s) | (quantise_pair<kF16>(x.y, s) << 16);
      const uint32_t hi = quantise_pair<kF16>(x.z, s) | (quantise_pair<kF16>(x.w, s) << 16);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(P.dst[which]) + at) = make_uint2(lo, hi);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.dst[which]) + at) = x;
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream) {
  const int64_t n = static_cast<int64_t>(p.T) * 2 * (p.H * p.D / 8);
  int64_t ctas = (n + kThreads - 1) / kThreads;
  if (ctas > 152 * 64) ctas = 152 * 64;
  const dim3 grid(static_cast<unsigned>(ctas));
  if (p.cache_dtype != DSPARK_E4M3)
    kv_append_kernel<false, false><<<grid, kThreads, 0, stream>>>(p);
  else if (p.dtype == DSPARK_F16)
    kv_append_kernel<true, true><<<grid, kThreads, 0, stream>>>(p);
  else
    kv_append_kernel<true, false><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dspark
