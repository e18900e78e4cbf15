// paged_attention.cu -- attention of a step's new tokens over the paged cache.
//
// The plainest form that is right for every case: one CTA per (token, query
// head). Each warp takes every fourth key that the row sees, its lanes split
// the head dimension, and the softmax runs along with one pass over the keys
// (running maximum and sum in fp32); the four warps' partial results are
// joined at the end.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "paged.h"

namespace dspark {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float f16_bits_to_float(uint16_t h) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(h));
  return f;
}
__device__ __forceinline__ uint16_t float_to_f16_bits(float f) {
  uint16_t h;
  asm("cvt.rn.f16.f32 %0, %1;" : "=h"(h) : "f"(f));
  return h;
}
__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
  uint32_t h;
  asm("{ .reg .b16 x; cvt.u16.u32 x, %1; cvt.rn.f16x2.e4m3x2 %0, x; }"
      : "=r"(h)
      : "r"(static_cast<uint32_t>(b)));
  return f16_bits_to_float(static_cast<uint16_t>(h & 0xFFFFu));
}

__device__ __forceinline__ float load_value(const void* p, int dtype, int64_t i) {
  if (dtype == DSPARK_E4M3) return e4m3_to_float(static_cast<const uint8_t*>(p)[i]);
  const uint16_t h = static_cast<const uint16_t*>(p)[i];
  return dtype == DSPARK_F16 ? f16_bits_to_float(h) : bf16_bits_to_float(h);
}

template <int kDim>
__global__ void __launch_bounds__(32 * kWarps) paged_attention_kernel(PagedAttentionParams P) {
  constexpr int kPer = kDim / 32;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][kDim];
  const int t = blockIdx.x, hq = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the request of this token: the first whose range holds it
  int b = -1, q0 = 0, q1 = 0;
  for (int i = 0; i < P.B; ++i) {
    const int a = P.query_start[i], e = P.query_start[i + 1];
    if (a < 0 || e < a || e > P.T) {
      if (threadIdx.x == 0) report(P.status, DSPARK_ERR_BOUNDS);
      continue;
    }
    if (b < 0 && t >= a && t < e) {
      b = i;
      q0 = a;
      q1 = e;
    }
  }
  if (b < 0) return;
  const int slot = P.rsi[b];
  int64_t len = P.seq_lens[b];
  const int64_t most = static_cast<int64_t>(P.M) << P.page_shift;
  if (slot < 0) {
    len = 0;
  } else if (slot >= P.S || len < 0 || len > most) {
    if (threadIdx.x == 0) report(P.status, DSPARK_ERR_BOUNDS);
    len = 0;
  }
  const int64_t pos = len - (q1 - q0) + (t - q0);
  int64_t j0 = 0, j1 = len;
  if (P.causal && pos + 1 < j1) j1 = pos + 1;
  if (P.window > 0 && pos - P.window + 1 > j0) j0 = pos - P.window + 1;
  const int h = hq / (P.Hq / P.kv.kv_heads);
  float q[kPer], o[kPer];
  for (int i = 0; i < kPer; ++i) {
    q[i] = load_value(P.q, P.dtype, static_cast<int64_t>(t) * P.q_stride + hq * kDim + lane + 32 * i);
    o[i] = 0.f;
  }
  const float sk = P.scale * (P.kv.k_scale ? P.kv.k_scale[h] : 1.f);
  float m = -INFINITY, l = 0.f;
  for (int64_t j = j0 + warp; j < j1; j += kWarps) {
    const int id = P.block_table[static_cast<int64_t>(slot) * P.M + (j >> P.page_shift)];
    const bool have = id >= 0 && id < P.kv.num_blocks;
    if (!have && lane == 0) report(P.status, DSPARK_ERR_BOUNDS);
    const int64_t off = j & ((1 << P.page_shift) - 1);
    const int64_t ka = id * P.kv.k_block_stride + h * P.kv.k_head_stride + off * P.kv.k_token_stride;
    const int64_t va = id * P.kv.v_block_stride + h * P.kv.v_head_stride + off * P.kv.v_token_stride;
    float x = 0.f;
    for (int i = 0; i < kPer; ++i)
      if (have) x = fmaf(q[i], load_value(P.kv.k, P.kv.dtype, ka + lane + 32 * i), x);
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, s);
    x *= sk;
    const float mn = fmaxf(m, x);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float keep = expf(m - base), p = expf(x - base);
    l = l * keep + p;
    for (int i = 0; i < kPer; ++i)
      o[i] = fmaf(p, have ? load_value(P.kv.v, P.kv.dtype, va + lane + 32 * i) : 0.f, o[i] * keep);
    m = mn;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int i = 0; i < kPer; ++i) s_o[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float mt = -INFINITY, lt = 0.f;
  for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, s_m[w]);
  const float base = mt == -INFINITY ? 0.f : mt;
  for (int w = 0; w < kWarps; ++w) lt += s_l[w] * expf(s_m[w] - base);
  const float vs = P.kv.v_scale ? P.kv.v_scale[h] : 1.f;
  const int64_t row = static_cast<int64_t>(t) * P.Hq + hq;
  for (int d = threadIdx.x; d < kDim; d += 32 * kWarps) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += s_o[w][d] * expf(s_m[w] - base);
    v = j1 > j0 ? v / lt * vs : 0.f;
    static_cast<uint16_t*>(P.out)[row * kDim + d] =
        P.dtype == DSPARK_F16 ? float_to_f16_bits(v) : float_to_bf16_bits(v);
  }
  if (P.lse && threadIdx.x == 0) P.lse[row] = j1 > j0 ? base + logf(lt) : -INFINITY;
}

}  // namespace

size_t paged_attention_workspace_bytes(int B, int Hq, int Hkv, int D) {
  (void)B;
  (void)Hq;
  (void)Hkv;
  (void)D;
  return 256;
}

cudaError_t launch_paged_attention(const PagedAttentionParams& p, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.T), static_cast<unsigned>(p.Hq));
  if (p.kv.head_dim == 64)
    paged_attention_kernel<64><<<grid, 32 * kWarps, 0, stream>>>(p);
  else
    paged_attention_kernel<128><<<grid, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dspark
