// kv_append.cu -- the keys and values of new tokens into their pages.
//
// A copy with an address per token: a thread owns a 16-byte piece (8 values) of
// the token's keys or values and takes it for several tokens, read from the
// tokens' side (which may be a view into a fused projection) and written into
// the page, as it is or divided by the head's scale and rounded to 8 bits. The
// quotient is the IEEE one, by products with the scale's reciprocal and a
// correction: 8 divisions a piece would cost as much time as the memory. In a
// 16-bit cache with scales, which is rare, it is by division.
//
// Bound by memory for long prompts (each value read once and written once; 16384
// tokens of 8 heads of 128 in bf16: 20.6 us, 6.5 TB/s) and by instruction issue
// beside it where values are rounded to 8 bits (20.5 us, 70% of the slots; 48
// registers for five CTAs an SM: 22.7 without that limit); by latency for a
// decode step (256 tokens 1.9 us), where a thread takes one token instead of
// kBatch, so that few tokens are spread over the GPU.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "paged.h"

namespace dspark {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // tokens per thread, all loaded before the first is stored

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

// A piece by divisions (out of line: hardly ever called).
template <bool kF16>
__device__ __noinline__ uint2 quantise_by_division(uint4 x, float scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[4];
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack<kF16>(w[i], a, b);
    y[i] = e4m3_pair(__fdiv_rn(a, scale), __fdiv_rn(b, scale));
  }
  return make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
}

// The 8 values of a piece over the scale, rounded to 8 bits. With r = rn(1 /
// scale), q = rn(x r) and the residual x - q scale (exact in an FMA),
// rn(q + (x - q scale) r) is the correctly rounded quotient (Markstein's
// theorem, as for temp_div2) wherever nothing over- or underflows. What
// underflows is far below the smallest 8-bit value; overflow, infinities and
// NaN make the quotient and so the piece's sum NaN, and such pieces, and scales
// outside [2^-30, 2^30] (`slow`), take the division itself.
template <bool kF16>
__device__ __forceinline__ uint2 quantise(uint4 x, unsigned long long r2, unsigned long long nt2,
                                          float scale, bool slow) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t y[4];
  unsigned long long sum = 0ull;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack<kF16>(w[i], a, b);
    const unsigned long long z = f2_pack(a, b), q = f2_mul(z, r2);
    const unsigned long long v = f2_fma(f2_fma(q, nt2, z), r2, q);
    sum = i ? f2_add(sum, v) : v;
    f2_unpack(v, a, b);
    y[i] = e4m3_pair(a, b);
  }
  float s0, s1;
  f2_unpack(sum, s0, s1);
  s0 += s1;
  if (slow || s0 != s0) return quantise_by_division<kF16>(x, scale);
  return make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
}

// The 8 values of a piece over the scale, rounded to fp32 and to their own type.
template <bool kF16>
__device__ __forceinline__ uint4 scaled16(uint4 x, float scale) {
  uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack<kF16>(w[i], a, b);
    a = __fdiv_rn(a, scale);
    b = __fdiv_rn(b, scale);
    if constexpr (kF16)
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
    else
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What becomes of a value: its bits, 8 bits of its quotient by the scale, 16.
enum Form { kCopy, kTo8, kTo16 };

// `width` threads share a token, `abreast` tokens are taken at a time.
template <Form kForm, bool kF16, int kPer>
__global__ void __launch_bounds__(kThreads, 5)
kv_append_kernel(KvAppendParams P, int width, int abreast) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int sub = threadIdx.x / width;
  if (sub >= abreast) return;
  const int t0 = blockIdx.x * (abreast * kPer) + sub;
  int64_t slot[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int t = t0 + i * abreast;
    slot[i] = t < P.T ? P.slot_map[t] : -1;
  }
  const int cd = P.D / 8, chunks = P.H * cd;  // pieces of a head, of a token's keys
  for (int p = threadIdx.x - sub * width; p < 2 * chunks; p += width) {
    const int which = p >= chunks ? 1 : 0;  // keys, then values
    const int c = p - which * chunks, h = c / cd;
    const uint16_t* src = static_cast<const uint16_t*>(P.src[which]) + c * 8;
    uint4 x[kPer];  // (not waiting for the slots: rows without one are read for nothing)
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (t0 + i * abreast < P.T)
        x[i] = *reinterpret_cast<const uint4*>(
            src + static_cast<int64_t>(t0 + i * abreast) * P.src_stride[which]);
    const int64_t head = h * P.head_stride[which] + (c - h * cd) * 8;
    float scale = 1.f;
    if (kForm != kCopy && P.scale[which]) scale = P.scale[which][h];
    const bool slow = !temp_div_t_ok(scale);
    const float rcp = __frcp_rn(scale);
    const unsigned long long r2 = f2_pack(rcp, rcp), nt2 = f2_pack(-scale, -scale);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (slot[i] < 0) continue;
      if (slot[i] >= P.num_slots) {
        report(P.status, DSPARK_ERR_BOUNDS);
        continue;
      }
      const int block = static_cast<int>(slot[i] >> P.page_shift);
      const int off = static_cast<int>(slot[i]) & ((1 << P.page_shift) - 1);
      const int64_t at = block * P.block_stride[which] + off * P.token_stride[which] + head;
      if constexpr (kForm == kTo8) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(P.dst[which]) + at) =
            quantise<kF16>(x[i], r2, nt2, scale, slow);
      } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.dst[which]) + at) =
            kForm == kTo16 ? scaled16<kF16>(x[i], scale) : x[i];
      }
    }
  }
}

template <Form kForm, bool kF16, int kPer>
cudaError_t launch(const KvAppendParams& p, int width, int abreast, cudaStream_t stream) {
  const int per = abreast * kPer;
  // (may be set up while the kernel before it ends, and waits for it)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.T + per - 1) / per));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_append_kernel<kForm, kF16, kPer>, p, width, abreast);
}

template <Form kForm, bool kF16>
cudaError_t launch_per(const KvAppendParams& p, cudaStream_t stream) {
  const int pieces = 2 * (p.H * p.D / 8);
  const int width = pieces < kThreads ? pieces : kThreads;
  const int abreast = kThreads / width;
  // up to four CTAs an SM with a token a thread, kBatch tokens a thread beyond
  return p.T <= 152 * 4 * abreast
             ? launch<kForm, kF16, 1>(p, width, abreast, stream)
             : launch<kForm, kF16, kBatch>(p, width, abreast, stream);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream) {
  const bool f16 = p.dtype == DSPARK_F16;
  if (p.cache_dtype == DSPARK_E4M3)
    return f16 ? launch_per<kTo8, true>(p, stream) : launch_per<kTo8, false>(p, stream);
  if (p.scale[0] || p.scale[1])
    return f16 ? launch_per<kTo16, true>(p, stream) : launch_per<kTo16, false>(p, stream);
  return launch_per<kCopy, false>(p, stream);
}

}  // namespace dspark
