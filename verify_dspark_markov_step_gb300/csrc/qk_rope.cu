// qk_rope.cu -- the norm of each query and key head and the rotation by the token's
// position, in one pass over the rows; with keys and values written into their
// pages, or without a cache.
//
// Mathematics. A head's row x of D values: y = x w / sqrt(mean x^2 + eps), then the
// pair (a, b) of frequency i becomes m (a cos t - b sin t, b cos t + a sin t), where
// t = position * 2 pi * turns_i / 2^64. turns_i is a 64-bit integer, so position *
// turns_i modulo 2^64 is that angle modulo a whole turn, exactly: no table over the
// positions, and no loss where a 32-bit angle has lost its fraction. (turns_i itself is
// rounded: position * 2^-65 turns.)
// The upper 32 bits give the nearest quarter turn and a rest of at most pi / 4, for
// which the series of sine and cosine to the ninth and eighth power are exact to
// 2^-25. All of this is fp32; a value is rounded once, to the type it is stored in.
//
// Layout. D / 16 lanes (up to a power of two) share a head's row, 16 values each: two
// 16-byte pieces, each of which neighbouring lanes have side by side, with both halves
// of eight pairs, so a pair never leaves its lane and the norm's sum is all that lanes
// exchange. A warp takes a few heads at a time of one kind of row (queries, keys,
// values); a token's sines and cosines are shared out over the warp, passed on in shared
// memory and folded with the weights, and serve all of its rounds. Rows come through a
// ring in shared memory, three rounds ahead (cp.async; every lane reads what it has
// loaded itself, so nothing is waited for but its own copies), and leave by wide stores;
// arithmetic is in packed pairs.
//
// Bound and measured. Prompts: memory; 16384 tokens, 32/8 heads of 128 in fp16, rows to
// rows: 51.5 us, 6.5 TB/s (96% of a copy; with rows one round ahead in registers 68);
// 64/8 heads with norms into a bf16 cache 102 us, 6.6 TB/s, into an e4m3 cache 103.5 us,
// 6.2 TB/s, instruction issue beside it (with kinds of rows mixed in a warp 115), into a
// bf16 cache with scales 113 us, 5.9 TB/s (16 divisions a lane; its long-batch kernels spill
// 4 to 16 bytes); in place 1 to 2% slower than into other rows. With few heads the angles,
// twice a token whatever its heads (queries and keys are in different CTAs), and the start
// of a warp: 8/1 heads 25 us where the bytes take 12. A decode step: latency; 256 tokens 3.9
// to 4.3 us, one 2.3.
// (Five CTAs an SM; six spill registers: 256 tokens 5.2 us, 1500 13.7 for 12.5.)
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kv_values.cuh"
#include "paged.h"

namespace dspark {

namespace {

constexpr int kThreads = 128, kCtas = 5;  // of an SM
// From so many tokens on a warp takes the rounds of several, and a round has place for
// several tokens' heads, which spares starts (16384 tokens, single and several: 16/2 heads
// of 128 43.5 and 37.5 us, 2/2 33.9 and 16.6, one of 64 30.6 and 9.6, 64/8 of 128 104.0 and
// 102.3); with fewer they only make warps longer (8192 tokens, 16/2: 23.3 both; 4000: 12.9
// and 16.3; 1500 of 64/8 11.7 and 15.2). That holds for many heads. With few of them the
// crossing lies lower, as 8191 (single) and 8192 (several) show: 1/1 heads of 64 16.7 and
// 6.3 us, 2/2 of 128 17.8 and 12.0, 8/1 21.4 and 18.2, 16/2 24.8 and 22.6, 64/8 54.1 and
// 52.6. What decides is how many of a round's lanes a token leaves free and the rounds in
// all; the rule does not look at them.
constexpr int kManyTokens = 8192;
constexpr int kStages = 4;  // rounds of rows on their way to a lane, and the one it works on

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

// Pairs (x[i], y[i]) of a lane's two pieces: of their i-th values, or of neighbours.
template <bool kF16, bool kSplit>
__device__ __forceinline__ void take(uint4 a, uint4 b, float (&x)[8], float (&y)[8]) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (kSplit) {
      if (i < 4)
        unpack<kF16>(w[i], x[2 * i], x[2 * i + 1]);
      else
        unpack<kF16>(w[i], y[2 * i - 8], y[2 * i - 7]);
    } else {
      unpack<kF16>(w[i], x[i], y[i]);
    }
  }
}
template <bool kF16, bool kSplit>
__device__ __forceinline__ void give(const float (&x)[8], const float (&y)[8], uint4& a, uint4& b) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (kSplit)
      w[i] = i < 4 ? pack16<kF16>(x[2 * (i & 3)], x[2 * (i & 3) + 1])
                   : pack16<kF16>(y[2 * (i & 3)], y[2 * (i & 3) + 1]);
    else
      w[i] = pack16<kF16>(x[i], y[i]);
  }
  a = make_uint4(w[0], w[1], w[2], w[3]);
  b = make_uint4(w[4], w[5], w[6], w[7]);
}
// Pairs of neighbours as they lie in the two pieces.
__device__ __forceinline__ void unweave(float (&x)[8], float (&y)[8]) {
  float v[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = x[i];
    v[2 * i + 1] = y[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = v[i];
    y[i] = v[8 + i];
  }
}

__device__ __forceinline__ void copy_async(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(to))),
               "l"(from)
               : "memory");
}

// How a launch's warps share the rows of a kind (queries, keys, values): 32 / width
// heads a round, `width` lanes each (a power of two). A round is of one token, or of
// several where their heads (up to a power of two: `share`) leave place; a warp takes a
// part of a token's rounds, or all of one or several tokens'.
struct Kind {
  int share;       // heads of a round that are of one token
  int rounds;      // of a token (of a round's tokens)
  int parts, per;  // warps that share a token's rounds, rounds of each
  int tokens;      // consecutive tokens (rounds' tokens) a warp takes
  int groups;      // tokens (rounds' tokens) in all
  unsigned first;  // CTA
};
struct Split {
  int width;
  Kind of[3];
};

// Where a lane's rows lie: the first values of its two pieces, of which neighbouring
// lanes' are side by side, and whether they are rotated.
template <bool kSplit>
struct Lane {
  int l, g;     // within the head, head of the round
  int c0, c1;
  bool mine, turn0, turn1;
  __device__ __forceinline__ Lane(const QkRopeParams& P, int width) {
    const int lane = threadIdx.x & 31, R = P.rotary;
    l = lane & (width - 1);
    g = lane / width;
    mine = 16 * l < P.D;
    if (kSplit) {  // the halves of eight pairs, or what is left of the row
      const bool pairs = 16 * l < R;
      c0 = pairs ? 8 * l : R / 2 + 8 * l;
      c1 = c0 + (pairs ? R : P.D - R) / 2;
      turn0 = turn1 = pairs;
    } else {       // neighbours lie within a piece
      c0 = 8 * l;
      c1 = c0 + P.D / 2;
      turn0 = c0 < R;
      turn1 = c1 < R;
    }
  }
};

// x' = x ca + y nsa, y' = y cb + x sb for a lane's eight pairs (x, y), two at a time:
// cosine and sine, the factor on them, the weights of a norm.
struct Coefficients {
  unsigned long long ca[4], nsa[4], cb[4], sb[4];
};

// `table` [32 / share][8 width], of this warp; `position` is the lane's token's, `first`
// the turns of the first two pairs that the lane works out.
template <bool kF16, bool kSplit, bool kNorm>
__device__ __forceinline__ void coefficients(const QkRopeParams& P, const Lane<kSplit>& L,
                                             int width, int share, int64_t position,
                                             const uint64_t (&first)[2], const void* weight,
                                             float2* table, Coefficients& k) {
  // the lanes of a token's heads share the work: all pairs' angles
  const int lanes = share * width, q = (threadIdx.x & 31) & (lanes - 1), pairs = 8 * width;
  table += (L.g / share) * pairs;
  __syncwarp();  // (the last token's have been read)
#pragma unroll 1
  for (int f0 = q; f0 < pairs; f0 += 2 * lanes) {  // (two at a time)
    float c[2], s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int f = f0 + u * lanes;
      const bool turns = 2 * f < P.rotary;
      const uint64_t a_turn = f0 == q ? first[u] : turns ? P.turns[f] : 0;
      const uint64_t at = static_cast<uint64_t>(position) * a_turn;
      cos_sin(static_cast<uint32_t>(at >> 32), c[u], s[u]);
      if (turns) {
        c[u] *= P.factor;
        s[u] *= P.factor;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (f0 + u * lanes < pairs) table[f0 + u * lanes] = make_float2(c[u], s[u]);
  }
  __syncwarp();
  float wx[8], wy[8];  // of the pairs' first and second values
#pragma unroll
  for (int i = 0; i < 8; ++i) wx[i] = wy[i] = 1.f;
  if (kNorm && weight && L.mine) {
    const uint16_t* w = static_cast<const uint16_t*>(weight);
    take<kF16, kSplit>(*reinterpret_cast<const uint4*>(w + L.c0),
                       *reinterpret_cast<const uint4*>(w + L.c1), wx, wy);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // pairs 2 i and 2 i + 1 of this lane: of its halves, or four of each piece
    const int f = kSplit ? 8 * L.l + 2 * i : (i < 2 ? L.c0 / 2 + 2 * i : L.c1 / 2 + 2 * i - 4);
    const float4 cs = *reinterpret_cast<const float4*>(table + min(f, pairs - 2));
    const unsigned long long c = f2_pack(cs.x, cs.z), s = f2_pack(cs.y, cs.w);
    const unsigned long long ns = f2_pack(-cs.y, -cs.w);
    const unsigned long long x = f2_pack(wx[2 * i], wx[2 * i + 1]);
    const unsigned long long y = f2_pack(wy[2 * i], wy[2 * i + 1]);
    k.ca[i] = kNorm ? f2_mul(c, x) : c;
    k.cb[i] = kNorm ? f2_mul(c, y) : c;
    k.nsa[i] = kNorm ? f2_mul(ns, y) : ns;
    k.sb[i] = kNorm ? f2_mul(s, x) : s;
  }
}

// The pairs of a row rotated and, with a norm, weighed and normalised: that comes
// last, so that the lanes' exchange runs beside the rotation.
template <bool kSplit, bool kNorm>
__device__ __forceinline__ void turn(const QkRopeParams& P, const Lane<kSplit>& L, int width,
                                     bool normed, const Coefficients& k, float (&x)[8],
                                     float (&y)[8]) {
  unsigned long long p[4], q[4], n2 = 0ull;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    p[i] = f2_pack(x[2 * i], x[2 * i + 1]);
    q[i] = f2_pack(y[2 * i], y[2 * i + 1]);
  }
  if (kNorm && normed) {
    unsigned long long sum2 = f2_mul(p[0], p[0]), sum3 = f2_mul(q[0], q[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      sum2 = f2_fma(p[i], p[i], sum2);
      sum3 = f2_fma(q[i], q[i], sum3);
    }
    float s0, s1;
    f2_unpack(f2_add(sum2, sum3), s0, s1);
    s0 += s1;
    for (int o = width >> 1; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xFFFFFFFFu, s0, o);
    const float norm = rsqrtf(fmaf(s0, P.inv_d, P.eps));
    n2 = f2_pack(norm, norm);
  }
  // (values that are not rotated apart: a sine of 0 would make NaN of an infinite
  // neighbour)
  constexpr int kPart = kSplit ? 4 : 2;
#pragma unroll
  for (int i0 = 0; i0 < 4; i0 += kPart) {
    if (i0 == 0 ? L.turn0 : L.turn1) {
#pragma unroll
      for (int i = i0; i < i0 + kPart; ++i) {
        const unsigned long long u = f2_fma(p[i], k.ca[i], f2_mul(q[i], k.nsa[i]));
        q[i] = f2_fma(q[i], k.cb[i], f2_mul(p[i], k.sb[i]));
        p[i] = u;
      }
    } else if (kNorm) {
#pragma unroll
      for (int i = i0; i < i0 + kPart; ++i) {
        p[i] = f2_mul(p[i], k.ca[i]);
        q[i] = f2_mul(q[i], k.cb[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kNorm && normed) {
      p[i] = f2_mul(p[i], n2);
      q[i] = f2_mul(q[i], n2);
    }
    f2_unpack(p[i], x[2 * i], x[2 * i + 1]);
    f2_unpack(q[i], y[2 * i], y[2 * i + 1]);
  }
}

// One warp's rounds of one kind of row; of one token unless kMulti.
template <int kWhat, Form kForm, bool kF16, bool kSplit, bool kNorm, bool kMulti>
__device__ __forceinline__ void rounds(const QkRopeParams& P, int width, const Kind& of,
                                       uint4 (&ring)[kStages][2][kThreads], float2* table) {
  constexpr bool kTurns = kWhat < 2, kPages = kForm != kRows && kWhat > 0;
  constexpr int kBytes = kPages && kForm == kTo8 ? 1 : 2;
  const int64_t warp = static_cast<int64_t>(blockIdx.x - of.first) * (kThreads / 32) +
                       (threadIdx.x >> 5);
  const int64_t group = warp / of.parts * of.tokens;
  if (group >= of.groups) return;
  int r = static_cast<int>(warp % of.parts) * of.per;
  const int n = of.parts > 1 ? min(of.per, of.rounds - r)
                             : static_cast<int>(min(static_cast<int64_t>(of.tokens),
                                                    of.groups - group)) * of.rounds;
  const Lane<kSplit> L(P, width);
  const int abreast = 32 / width, heads = kWhat == 0 ? P.Hq : P.H;
  const int tokens = abreast / of.share;            // of a round
  int t = static_cast<int>(group) * tokens + L.g / of.share;  // this lane's token
  const int g = L.g & (of.share - 1);               // its head of a round

  // Rows into this lane's own places of the ring, so that nobody else waits.
  const int across = L.c1 - L.c0, step = abreast * P.D;
  int load_t = t, load_r = r, left = n;
  auto row_of = [&](int token, int round) {
    return static_cast<const uint16_t*>(P.src[kWhat]) + token * P.src_stride[kWhat] +
           (static_cast<int64_t>(round) * step + g * P.D + L.c0);
  };
  const uint16_t* src = row_of(load_t, load_r);
  int64_t position = t < P.T ? P.positions[t] : -1, slot = -1;
  if (kPages && t < P.T) slot = P.slot_map[t];
  // what the first coefficients need, on its way beside the position
  const void* weight = kTurns ? P.weight[kTurns ? kWhat : 0] : nullptr;
  uint64_t turns[2] = {0, 0};
  if (kTurns) {
    const int lanes = of.share * width, q = (threadIdx.x & 31) & (lanes - 1);
    if (2 * q < P.rotary) turns[0] = P.turns[q];
    if (2 * (q + lanes) < P.rotary) turns[1] = P.turns[q + lanes];
  }
  auto load = [&](unsigned stage) {
    if (left > 0) {
      if (L.mine && load_t < P.T && load_r * abreast + g < heads) {
        copy_async(&ring[stage][0][threadIdx.x], src);
        copy_async(&ring[stage][1][threadIdx.x], src + across);
      }
      --left;
      src += step;
      if (++load_r == of.rounds && kMulti) {
        load_r = 0;
        load_t += tokens;
        src = row_of(load_t, 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (kTurns && !L.mine) {  // lanes past the row add nothing to its norm
#pragma unroll
    for (int i = 0; i < kStages; ++i)
      ring[i][0][threadIdx.x] = ring[i][1][threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(i);  // (not waiting for the position)
  Coefficients k;
  uint8_t* dst = nullptr;  // of this lane's first piece of the round
  const int64_t next = kPages ? abreast * P.head_stride[kWhat > 0 ? kWhat - 1 : 0] * kBytes
                              : static_cast<int64_t>(step) * kBytes;
  bool live = false;       // the token has a place for its rows
  auto begin = [&]() {     // a token
    live = L.mine && position >= 0;
    const int64_t h = static_cast<int64_t>(r) * abreast + g;
    if (kPages) {
      if (slot >= P.num_slots) {
        if (kWhat == 1 && live) report(P.status, DSPARK_ERR_BOUNDS);
        slot = -1;
      }
      live &= slot >= 0;
      const int off = static_cast<int>(slot) & ((1 << P.page_shift) - 1);
      dst = static_cast<uint8_t*>(P.dst[kWhat]) +
            ((slot >> P.page_shift) * P.block_stride[kWhat > 0 ? kWhat - 1 : 0] +
             off * P.dst_stride[kWhat] + h * P.head_stride[kWhat > 0 ? kWhat - 1 : 0] + L.c0) *
                kBytes;
    } else {
      dst = static_cast<uint8_t*>(P.dst[kWhat]) +
            (t * P.dst_stride[kWhat] + h * P.D + L.c0) * kBytes;
    }
    if (kTurns)
      coefficients<kF16, kSplit, kNorm>(P, L, width, of.share, position, turns, weight, table, k);
  };
  begin();
  if (!kMulti && __all_sync(0xFFFFFFFFu, !live)) {  // no place for any
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
#pragma unroll(kMulti ? 1 : kStages)
  for (int i = 0; i < n; ++i) {  // (uniform in a warp, whose lanes exchange sums)
    if (kMulti && r == 0) {
      if (i > 0) begin();
      // of the next token, if it is this warp's
      t += tokens;
      position = -1;
      if (t < P.T && n - i > of.rounds) {
        position = P.positions[t];
        if (kPages) slot = P.slot_map[t];
      }
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    const unsigned stage = static_cast<unsigned>(i) % kStages;
    uint4 a = ring[stage][0][threadIdx.x], b = ring[stage][1][threadIdx.x];
    load((stage + kStages - 1) % kStages);  // into the place that the round before has read
    const int h = r * abreast + g;
    const bool store = live && h < heads;
    float scale = 1.f;
    if (kPages && kForm != kCopy && store && P.scale[kWhat - 1]) scale = P.scale[kWhat - 1][h];
    float x[8], y[8];
    if (kTurns || (kPages && kForm != kCopy)) take<kF16, kSplit>(a, b, x, y);
    if (kTurns) turn<kSplit, kNorm>(P, L, width, weight != nullptr, k, x, y);
    if (kPages && kForm == kTo8) {
      const bool slow = !temp_div_t_ok(scale);
      const float rcp = __frcp_rn(scale);
      if (!kSplit) unweave(x, y);
      if (store) {
        *reinterpret_cast<uint2*>(dst) = to8(x, rcp, scale, slow);
        *reinterpret_cast<uint2*>(dst + across) = to8(y, rcp, scale, slow);
      }
    } else {
      if (kPages && kForm == kTo16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = __fdiv_rn(x[e], scale);
          y[e] = __fdiv_rn(y[e], scale);
        }
      }
      if (kTurns || (kPages && kForm == kTo16)) give<kF16, kSplit>(x, y, a, b);
      if (store) {
        *reinterpret_cast<uint4*>(dst) = a;
        *reinterpret_cast<uint4*>(dst + 2 * across) = b;
      }
    }
    dst += next;
    if (++r == of.rounds && kMulti) r = 0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// kSplit: pairs are (i, i + rotary / 2), else (2 i, 2 i + 1). kNorm: queries or keys
// have a norm. kMulti: several tokens a warp. The CTAs' kinds of rows are apart, so that
// one's warps end together.
template <Form kForm, bool kF16, bool kSplit, bool kNorm, bool kMulti>
__global__ void __launch_bounds__(kThreads, kCtas)
qk_rope_kernel(const __grid_constant__ QkRopeParams P, const __grid_constant__ Split split) {
  __shared__ uint4 ring[kStages][2][kThreads];
  __shared__ __align__(16) float2 angles[kThreads / 32][256];  // 8 for each lane
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float2* table = angles[threadIdx.x >> 5];
  if (blockIdx.x < split.of[1].first)
    rounds<0, kForm, kF16, kSplit, kNorm, kMulti>(P, split.width, split.of[0], ring, table);
  else if (kForm == kRows || blockIdx.x < split.of[2].first)
    rounds<1, kForm, kF16, kSplit, kNorm, kMulti>(P, split.width, split.of[1], ring, table);
  else if constexpr (kForm != kRows)
    rounds<2, kForm, kF16, kSplit, false, kMulti>(P, split.width, split.of[2], ring, table);
}

template <Form kForm, bool kF16, bool kSplit, bool kNorm, bool kMulti>
cudaError_t launch(const QkRopeParams& p, cudaStream_t stream) {
  int sms = 0;
  const cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  Split split;
  split.width = 1;
  while (16 * split.width < p.D) split.width *= 2;
  const int abreast = 32 / split.width;
  // Warps that are resident at a time (as many rounds a warp as there are for each of
  // them), and the most rounds a warp takes of more than one token.
  constexpr int kMost = 6, kPerCta = kThreads / 32;
  const int resident = sms * kCtas * kPerCta;
  const int heads[3] = {p.Hq, p.H, kForm == kRows ? 0 : p.H};
  int64_t total = 0;
  for (int what = 0; what < 3; ++what) {
    Kind& of = split.of[what];
    of.share = kMulti ? 1 : abreast;
    while (of.share < heads[what] && of.share < abreast) of.share *= 2;
    of.rounds = (heads[what] + abreast - 1) / abreast;
    const int tokens = abreast / of.share;
    of.groups = of.rounds ? (p.T + tokens - 1) / tokens : 0;
    total += static_cast<int64_t>(of.groups) * of.rounds;
  }
  const int64_t per = (total + resident - 1) / resident;
  unsigned ctas = 0;
  for (Kind& of : split.of) {
    of.parts = of.tokens = 1;
    of.per = of.rounds;
    if (per < of.rounds) {
      of.parts = (of.rounds + static_cast<int>(per) - 1) / static_cast<int>(per);
      of.per = (of.rounds + of.parts - 1) / of.parts;
      of.parts = (of.rounds + of.per - 1) / of.per;
    } else if (kMulti && of.rounds > 0 && of.rounds < kMost) {
      of.tokens = static_cast<int>(per < kMost ? per : kMost) / of.rounds;
    }
    const int64_t warps =
        (static_cast<int64_t>(of.groups) + of.tokens - 1) / of.tokens * of.parts;
    of.first = ctas;
    ctas += static_cast<unsigned>((warps + kPerCta - 1) / kPerCta);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  // (may be set up while the kernel before it ends, and waits for it)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, qk_rope_kernel<kForm, kF16, kSplit, kNorm, kMulti>, p, split);
}

template <Form kForm, bool kNorm, bool kMulti>
cudaError_t launch_norm(const QkRopeParams& p, cudaStream_t stream) {
  if (p.dtype == DSPARK_F16)
    return p.interleaved ? launch<kForm, true, false, kNorm, kMulti>(p, stream)
                         : launch<kForm, true, true, kNorm, kMulti>(p, stream);
  return p.interleaved ? launch<kForm, false, false, kNorm, kMulti>(p, stream)
                       : launch<kForm, false, true, kNorm, kMulti>(p, stream);
}

template <Form kForm>
cudaError_t launch_form(const QkRopeParams& p, cudaStream_t stream) {
  const bool multi = p.T >= kManyTokens;
  const bool norm = p.weight[0] || p.weight[1];
  if (multi)
    return norm ? launch_norm<kForm, true, true>(p, stream)
                : launch_norm<kForm, false, true>(p, stream);
  return norm ? launch_norm<kForm, true, false>(p, stream)
              : launch_norm<kForm, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_qk_rope(const QkRopeParams& p, cudaStream_t stream) {
  if (!p.slot_map) return launch_form<kRows>(p, stream);
  if (p.cache_dtype == DSPARK_E4M3) return launch_form<kTo8>(p, stream);
  if (p.scale[0] || p.scale[1]) return launch_form<kTo16>(p, stream);
  return launch_form<kCopy>(p, stream);
}

}  // namespace dspark
