// qk_rope.cu -- the norm of each query and key head and the rotation by the token's
// position, in one pass over the rows; with keys and values written into their
// pages, or without a cache.
//
// Mathematics. A head's row x of D values: y = x w / sqrt(mean x^2 + eps), then the
// pair (a, b) of frequency i becomes m (a cos t - b sin t, b cos t + a sin t), where
// t = position * 2 pi * turns_i / 2^64. turns_i is a 64-bit integer, so position *
// turns_i modulo 2^64 is the angle modulo a whole turn, exactly, at any position: no
// table over the positions, and no loss where a 32-bit angle has lost its fraction.
// The upper 32 bits give the nearest quarter turn and a rest of at most pi / 4, for
// which the series of sine and cosine to the ninth and eighth power are exact to
// 2^-25. All of this is fp32; a value is rounded once, to the type it is stored in.
//
// Layout. D / 16 lanes (up to a power of two) share a head's row, 16 values each:
// the two 16-byte pieces that hold both halves of eight pairs, so a pair never
// leaves its lane and the norm's sum is all that lanes exchange. The heads of a
// token follow each other in one or more warps ("parts": enough to fill the GPU with
// few tokens), and the eight sines and cosines of a lane serve all of them.
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kv_values.cuh"
#include "paged.h"

namespace dspark {

namespace {

constexpr int kThreads = 256;

// What becomes of keys and values: rows, the cache's pages as they are, in 8
// bits by their scales, in 16 bits by their scales.
enum Form { kRows, kCopy, kTo8, kTo16 };

// Cosine and sine of f / 2^32 turns.
__device__ __forceinline__ void cos_sin(uint32_t f, float& c, float& s) {
  const uint32_t quarter = (f + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(f - (quarter << 30))) *
                  1.46291807926715968e-9f;  // 2 pi / 2^32
  const float z = x * x;
  float sn = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  sn = fmaf(z, sn, 1.f / 120.f);
  sn = fmaf(z, sn, -1.f / 6.f);
  sn = fmaf(z * x, sn, x);
  float cs = fmaf(z, 1.f / 40320.f, -1.f / 720.f);
  cs = fmaf(z, cs, 1.f / 24.f);
  cs = fmaf(z, cs, -0.5f);
  cs = fmaf(z, cs, 1.f);
  c = quarter & 1u ? sn : cs;
  s = quarter & 1u ? cs : sn;
  if ((quarter + 1u) & 2u) c = -c;
  if (quarter & 2u) s = -s;
}

// 8 values over the scale, in 8 bits: the IEEE quotient rounded once more.
__device__ __noinline__ uint2 to8_by_division(float4 x, float4 y, float scale) {
  const uint32_t a = e4m3_pair(__fdiv_rn(x.x, scale), __fdiv_rn(x.y, scale));
  const uint32_t b = e4m3_pair(__fdiv_rn(x.z, scale), __fdiv_rn(x.w, scale));
  const uint32_t c = e4m3_pair(__fdiv_rn(y.x, scale), __fdiv_rn(y.y, scale));
  const uint32_t d = e4m3_pair(__fdiv_rn(y.z, scale), __fdiv_rn(y.w, scale));
  return make_uint2(a | (b << 16), c | (d << 16));
}

// The same by the scale's reciprocal and a correction (Markstein's theorem, as for
// temp_div2): exact where nothing over- or underflows. What underflows is far below
// the smallest 8-bit value; overflow, infinities and NaN make the quotients' sum
// NaN and take the division, and so do scales outside [2^-30, 2^30] (`slow`).
__device__ __forceinline__ uint2 to8(const float (&v)[8], float rcp, float scale, bool slow) {
  const unsigned long long r2 = f2_pack(rcp, rcp), nt2 = f2_pack(-scale, -scale);
  uint32_t y[4];
  unsigned long long sum = 0ull;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned long long z = f2_pack(v[2 * i], v[2 * i + 1]), q = f2_mul(z, r2);
    const unsigned long long x = f2_fma(f2_fma(q, nt2, z), r2, q);
    sum = i ? f2_add(sum, x) : x;
    float a, b;
    f2_unpack(x, a, b);
    y[i] = e4m3_pair(a, b);
  }
  float s0, s1;
  f2_unpack(sum, s0, s1);
  s0 += s1;
  if (slow || s0 != s0)
    return to8_by_division(make_float4(v[0], v[1], v[2], v[3]), make_float4(v[4], v[5], v[6], v[7]),
                           scale);
  return make_uint2(y[0] | (y[1] << 16), y[2] | (y[3] << 16));
}

template <bool kF16>
__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]) {
  unpack<kF16>(w.x, v[0], v[1]);
  unpack<kF16>(w.y, v[2], v[3]);
  unpack<kF16>(w.z, v[4], v[5]);
  unpack<kF16>(w.w, v[6], v[7]);
}

template <bool kF16>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack16<kF16>(v[0], v[1]), pack16<kF16>(v[2], v[3]), pack16<kF16>(v[4], v[5]),
                    pack16<kF16>(v[6], v[7]));
}

// `width` lanes a head (a power of two), `parts` warps a token, `per` rounds of 32 /
// width heads a warp. kSplit: pairs are (i, i + rotary / 2), else (2 i, 2 i + 1).
template <Form kForm, bool kF16, bool kSplit>
__global__ void __launch_bounds__(kThreads, 3)
qk_rope_kernel(QkRopeParams P, int width, int parts, int per) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int t = static_cast<int>(warp / parts);
  if (t >= P.T) return;
  const int part = static_cast<int>(warp - static_cast<int64_t>(t) * parts);
  const int l = lane & (width - 1), abreast = 32 / width;
  const int R = P.rotary;
  const bool mine = 16 * l < P.D, turns = 16 * l < R;
  // the first values of this lane's two pieces
  const int c0 = kSplit ? (turns ? 8 * l : 16 * l) : 16 * l;
  const int c1 = kSplit && turns ? c0 + R / 2 : c0 + 8;
  const int heads = kForm == kRows ? P.Hq + P.H : P.Hq + 2 * P.H;
  int n = part * per * abreast + lane / width;  // head row of the token: queries, keys, values
  const int end = min(heads, (part + 1) * per * abreast);

  auto source = [&](int r, int& what, int& h) -> const uint16_t* {
    what = r < P.Hq ? 0 : r < P.Hq + P.H ? 1 : 2;
    h = what == 0 ? r : what == 1 ? r - P.Hq : r - P.Hq - P.H;
    return static_cast<const uint16_t*>(P.src[what]) + t * P.src_stride[what] +
           static_cast<int64_t>(h) * P.D;
  };
  uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
  int what, h;
  if (mine && n < end) {  // (not waiting for the position)
    const uint16_t* src = source(n, what, h);
    a = *reinterpret_cast<const uint4*>(src + c0);
    b = *reinterpret_cast<const uint4*>(src + c1);
  }
  const int64_t position = P.positions[t];
  int64_t slot = -1;
  if (kForm != kRows) {
    slot = P.slot_map[t];
    if (slot >= P.num_slots) {
      if (part == 0 && lane == 0 && position >= 0) report(P.status, DSPARK_ERR_BOUNDS);
      slot = -1;
    }
  }
  if (position < 0) return;
  float cs[8], sn[8];
  if (turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t at = static_cast<uint64_t>(position) * P.turns[8 * l + i];
      cos_sin(static_cast<uint32_t>(at >> 32), cs[i], sn[i]);
      cs[i] *= P.factor;
      sn[i] *= P.factor;
    }
  }
  // (the loop is uniform in a warp, whose lanes exchange sums)
  for (int r0 = part * per * abreast; r0 < end; r0 += abreast, n += abreast) {
    uint4 an = make_uint4(0u, 0u, 0u, 0u), bn = an;
    const int next = n + abreast;
    if (mine && next < end) {
      int w1, h1;
      const uint16_t* src = source(next, w1, h1);
      an = *reinterpret_cast<const uint4*>(src + c0);
      bn = *reinterpret_cast<const uint4*>(src + c1);
    }
    const bool live = mine && n < end;
    source(n, what, h);
    float x[8], y[8];
    unpack8<kF16>(a, x);
    unpack8<kF16>(b, y);
    const void* weight = what == 0 ? P.weight[0] : what == 1 ? P.weight[1] : nullptr;
    if (P.weight[0] || P.weight[1]) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], fmaf(y[i], y[i], sum));
      for (int o = width >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      if (live && weight) {
        const uint16_t* w = static_cast<const uint16_t*>(weight);
        const float scale = rsqrtf(sum * P.inv_d + P.eps);
        float w0[8], w1[8];
        unpack8<kF16>(*reinterpret_cast<const uint4*>(w + c0), w0);
        unpack8<kF16>(*reinterpret_cast<const uint4*>(w + c1), w1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= scale * w0[i];
          y[i] *= scale * w1[i];
        }
      }
    }
    if (turns && what != 2) {
      auto turn = [&](float& p, float& q, int i) {
        const float u = p * cs[i] - q * sn[i];
        q = q * cs[i] + p * sn[i];
        p = u;
      };
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (kSplit)
          turn(x[i], y[i], i);
        else if (i < 4)
          turn(x[2 * i], x[2 * i + 1], i);
        else
          turn(y[2 * i - 8], y[2 * i - 7], i);
      }
    }
    if (live) {
      if (what == 0 || kForm == kRows) {
        uint16_t* dst = static_cast<uint16_t*>(P.dst[what]) + t * P.dst_stride[what] +
                        static_cast<int64_t>(h) * P.D;
        *reinterpret_cast<uint4*>(dst + c0) = pack8<kF16>(x);
        *reinterpret_cast<uint4*>(dst + c1) = pack8<kF16>(y);
      } else if (slot >= 0) {
        const int block = static_cast<int>(slot >> P.page_shift);
        const int off = static_cast<int>(slot) & ((1 << P.page_shift) - 1);
        const int64_t at = block * P.block_stride[what - 1] + off * P.dst_stride[what] +
                           h * P.head_stride[what - 1];
        float scale = 1.f;
        if (kForm != kCopy && P.scale[what - 1]) scale = P.scale[what - 1][h];
        if constexpr (kForm == kTo8) {
          const bool slow = !temp_div_t_ok(scale);
          const float rcp = __frcp_rn(scale);
          uint8_t* dst = static_cast<uint8_t*>(P.dst[what]) + at;
          *reinterpret_cast<uint2*>(dst + c0) = to8(x, rcp, scale, slow);
          *reinterpret_cast<uint2*>(dst + c1) = to8(y, rcp, scale, slow);
        } else {
          uint16_t* dst = static_cast<uint16_t*>(P.dst[what]) + at;
          if constexpr (kForm == kTo16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              x[i] = __fdiv_rn(x[i], scale);
              y[i] = __fdiv_rn(y[i], scale);
            }
          }
          *reinterpret_cast<uint4*>(dst + c0) = pack8<kF16>(x);
          *reinterpret_cast<uint4*>(dst + c1) = pack8<kF16>(y);
        }
      }
    }
    a = an;
    b = bn;
  }
}

template <Form kForm, bool kF16, bool kSplit>
cudaError_t launch(const QkRopeParams& p, cudaStream_t stream) {
  int width = 1;
  while (16 * width < p.D) width *= 2;
  const int heads = kForm == kRows ? p.Hq + p.H : p.Hq + 2 * p.H;
  const int abreast = 32 / width, rounds = (heads + abreast - 1) / abreast;
  // a token's rounds over as many warps as it takes to give every SM 24
  constexpr int kWarps = 152 * 24;
  int parts = (kWarps + p.T - 1) / p.T;
  if (parts > rounds) parts = rounds;
  const int per = (rounds + parts - 1) / parts;
  parts = (rounds + per - 1) / per;
  const int64_t warps = static_cast<int64_t>(p.T) * parts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  // (may be set up while the kernel before it ends, and waits for it)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_rope_kernel<kForm, kF16, kSplit>, p, width, parts, per);
}

template <Form kForm>
cudaError_t launch_form(const QkRopeParams& p, cudaStream_t stream) {
  if (p.dtype == DSPARK_F16)
    return p.interleaved ? launch<kForm, true, false>(p, stream)
                         : launch<kForm, true, true>(p, stream);
  return p.interleaved ? launch<kForm, false, false>(p, stream)
                       : launch<kForm, false, true>(p, stream);
}

}  // namespace

cudaError_t launch_qk_rope(const QkRopeParams& p, cudaStream_t stream) {
  if (!p.slot_map) return launch_form<kRows>(p, stream);
  if (p.cache_dtype == DSPARK_E4M3) return launch_form<kTo8>(p, stream);
  if (p.scale[0] || p.scale[1]) return launch_form<kTo16>(p, stream);
  return launch_form<kCopy>(p, stream);
}

}  // namespace dspark
