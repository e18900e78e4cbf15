// paged_attention.cu -- attention of a step's new tokens over the paged cache,
// on the 5th-generation tensor cores: one persistent launch, and a small one
// that joins the requests whose keys were split over CTAs.
//
// Mathematics. For a query row, softmax(x) V over its visible keys in one pass
// over tiles of 128 keys: with a reference r (a running maximum of the scaled
// scores, in powers of two), p_j = 2^(x_j - r), l = sum p_j and O = sum p_j v_j
// are kept; when the maximum grows, O and l are multiplied by
// 2^(r_old - r_new). r is only moved when the maximum has grown by more than
// 2^8 (p then stays below 2^8, exact in any of the types), so that O, which
// lives in tensor memory, is hardly ever touched by the softmax. Scores, l and
// O are fp32; the p_j are rounded to the MMA's 16-bit type (bf16 keeps its
// range; fp16 gets 2^7 on top, so that a p 2^-31 below the maximum is still
// nonzero), which costs as much accuracy as the output's own rounding. x_j - r is
// one FMA of the unscaled score and the rounded r; where r is so large that its
// rounding shows, the row's reference is first taken off its scores, which is
// exact near the maximum (p keeps its bound whatever the scores' size).
//
// Rows. The query heads of a key head read the same keys, so a tile's 128 rows
// are (token, head of the group) pairs: floor(128 / group) tokens. A unit of
// work is two such row tiles of one request and key head ("pair": each of the
// two softmax warpgroups owns a row tile, and every key tile is used twice), or
// a single one ("single": the two warpgroups take key tiles in turn, and their
// results are joined at the end). Two single units of neighbouring key heads have
// the same lengths and masks; where a run has both whole, they are done side by
// side ("twin": a warpgroup each, nothing to join, one end for two units: 177
// requests of one token over 279 keys, 8 heads of 64, fp16: 49 us for 64). In all
// three the tensor core works on one warpgroup's scores while the other's are being
// exponentiated.
//
// Split. Lengths live on the device and are ragged. Every CTA sums up the costs
// of all units (key tiles and a constant) and takes a run of equal cost, so a long
// request is spread over many CTAs and short ones share a CTA, without the host
// and without atomics. A unit that a run's ends cut is written as partial
// (O, r, l) per CTA and joined by paged_join_kernel in a fixed order; where even
// runs gain less than that costs, a CTA takes the units that start in its run to
// their ends and nothing is joined.
//
// Warps: 0-3 and 4-7 softmax (thread = row = lane of tensor memory), 9 issues
// the MMAs (the warpgroups' in turn, which keeps one's softmax beside the other's
// products; what the issuer spends on waits and commits the tensor core idles, so
// an item has one wait and one commit, and the softmax warps give back the tiles
// that committed MMAs have read), 8 and 10 are the TMA producers (keys and values
// go through one ring in the order of their use; each issues half of a tile's
// boxes), 11 the scout: it walks the units ahead of the others, loads their query
// rows (a ring of two row tiles) and publishes what the others need to know of
// them. With an 8-bit cache 8 loads alone, 10 and 13-15 convert e4m3 tiles to fp16
// in shared memory (the 8-bit values are exact in fp16; an 8-bit MMA would want
// the queries and p in 8 bits too), and the softmax warps bring the query rows to
// fp16 by a power of two per row. Pages: a 128-key tile is 128 / page_size TMA
// boxes.
//
// What a row does not see must not reach it: masked scores are replaced (not
// added to), value rows past the request's last token are zeroed in shared
// memory, and in tiles that some row sees only in part a non-finite value of a
// key that is not seen by all moves that tile's P V off the tensor core (where
// 0 * NaN would spread) onto a slow exact path.
//
// Bound and measured (GB300). Few new tokens: memory; 32 requests x 8 tokens over
// 22k, 64/8 heads of 128, bf16: 431 to 440 us, 6.75 TB/s or more (a copy makes
// 6.70); 4 x 8 tokens 70 us, one token (32/8 heads) 28.7 us, of which 8 us pass
// before the first scores (plan, first page, first tile) and 4 in the join.
// Prompts: the tensor cores; 4096 tokens over 12288: 1.30 ms among other work, 1.48
// PFLOP/s (1.22 ms by itself on a cool card), the tensor pipe active 68%. An 8-bit
// cache: shared memory, through which a tile passes three times here (raw,
// converted, operands): about 1800 clocks a tile of K and V at 128 bytes a clock,
// 1870 taken; 256 x 4 tokens over 2-6k, 32/4 heads: 268 us.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "paged.h"
#include "tc_ptx.cuh"

namespace dspark {

namespace {

constexpr int kRows = 128;   // rows of a tile (UMMA M, lanes of tensor memory)
constexpr int kKeys = 128;   // keys of a tile
constexpr int kMaxStages = 10;
constexpr int kMaxRaw = 8;
constexpr int kMaxCtas = 160;
constexpr int kMinTiles = 2;  // key tiles a CTA takes at least
// What a unit costs besides its key tiles, in tiles (its query rows, the first
// scores, masks and the result overlap with little): the runs are of equal cost.
constexpr int kUnitTiles = 3;
// Where the table can only hold units of at most this many key tiles, none is split
// over CTAs and the join is not launched: each part costs a CTA a segment, and the
// join 4 to 12 us (32 requests x 8 tokens over 1400: 41 us whole, 50 split; one
// token over 600: 13 and 17). With units for few of the SMs long ones gain more from
// more SMs (one token over 1400: 20 and 18).
constexpr int kWholeTiles = 12, kWholeTilesFewUnits = 8;
// Else the plan decides by the lengths: units stay whole where the longest run of
// whole units is at most this many tiles longer than an even split's (8, and 2 for
// each unit an SM up to two: with more units a CTA has more parts). Measured, split
// and whole, units of 256 rows, bf16, heads of 128: 112 units of 8 tiles 40.0 and
// 22.5 us, of 24 tiles 64.3 and 48.7; 56 of 12 tiles 30.3 and 27.8, of 24 tiles
// 41.2 and 46.4; 8 of 8 tiles 19.3 and 20.8; 480 of 12 tiles 106 and 104, of 24
// tiles 170 and 178. Units of 8 rows, fp16 heads of 64 and an 8-bit cache change
// sides within two tiles of these.
constexpr int kSplitGain = 8, kSplitGainUnits = 2;
constexpr int kMaxRun = 0x3FFFFFFF;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kGrow = 8.0f;  // the reference moves when the maximum passes it by 2^8
// A reference beyond this (in powers of two) is taken off the scores before they
// are scaled: a rounded 2^29 is off by enough to bring a p past fp16's range, or
// to zero. Done behind the branch that every tile has for a maximum that moves: one
// of its own in every tile took 1344 us for 1311 (4096 tokens over 12288).
constexpr float kFar = 1024.f;

template <int D, bool kQuant>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTileBytes = kHalves * kRows * 128;  // 128 x D in 16 bits
  static constexpr int kRawBytes = kKeys * D;               // 128 x D in 8 bits
  // (3 + 3 stages beside an 8-bit cache: 4 + 2 took 302 us for 277, 3 + 4 280)
  static constexpr int kStages = kQuant ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);
  static constexpr int kRaw = kQuant ? (D == 128 ? 3 : 6) : 0;
  static constexpr int kThreads = kQuant ? 512 : 384;
  // Registers a thread after the split: 2 x 216 + 72 = the launch's 3 x 168, or
  // 2 x 184 + 2 x 72 = 4 x 128. 216 hold the 128 scores of a row; beside the
  // converters they are taken 64 at a time.
  static constexpr int kSoftmaxRegs = kQuant ? 184 : 216;
  static constexpr int kOtherRegs = 72;
  // shared memory, offsets from a 1024-byte aligned base
  static constexpr int q = 0;
  static constexpr int kv = q + 2 * kTileBytes;
  static constexpr int raw = kv + kStages * kTileBytes;
  static constexpr int misc = raw + kRaw * kRawBytes;
  static constexpr int kBytes = misc + 2048 + 1024;
  static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
};

struct Request {
  int q0, n, slot, len;
};

// A run of key tiles of one unit.
struct Seg {
  Request r;
  int h;
  int t0, t1;   // tokens of the unit within the request
  int j0, j1;   // key tiles
  int after;    // CTAs after this one that work on the unit
  bool pair, opens, closes;  // two row tiles; starts / ends with the unit
  bool twin;    // the whole units of key heads h and h + 1
  bool end;     // no segment, the walk is over
  __device__ int tiles() const { return j1 - j0; }
  __device__ bool two() const { return pair || twin; }  // a row tile each
  // items (key tiles) of warpgroup w and the k-th one's tile
  __device__ int items(int w) const { return two() ? tiles() : (tiles() + 1 - w) / 2; }
  __device__ int tile(int w, int k) const { return two() ? j0 + k : j0 + 2 * k + w; }
  // The tiles in the order of their loading (a twin's heads in turn): how many,
  // which one is item k of warpgroup w, the i-th one's key tile and head.
  __device__ int loads() const { return twin ? 2 * tiles() : tiles(); }
  __device__ int load_of(int w, int k) const { return pair ? k : 2 * k + w; }
  __device__ int load_tile(int i) const { return j0 + (twin ? i >> 1 : i); }
  __device__ int load_head(int i) const { return twin ? h + (i & 1) : h; }
  __device__ int ahead() const { return pair ? 1 : 2; }  // key tiles loaded before the first values
  // place of the i-th tile's keys / values among all loads of the segment
  __device__ int k_place(int i) const {
    const int a = ahead();
    return i < a ? i : 2 * i - a + 1;
  }
  __device__ int v_place(int i) const { return i + min(loads(), ahead() + i); }
};

struct Misc {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  uint64_t raw_full[kMaxRaw], raw_empty[kMaxRaw];
  uint64_t q_full[2], q_ready[2], q_empty[2];
  uint64_t s_full[2], p_ready[2], o_full[2], scanned[2];
  uint64_t merge[2], merged, drain;
  Seg seg[2];  // of the segment whose first row tile is in the slot
  uint32_t tmem;
  int fail;
  uint32_t total;    // tiles that the producer has loaded, once it is done
  uint32_t filling;  // tiles of the MMA's ring whose stage is being filled, or was
  int bad[2];      // the last tile whose values were found non-finite, per warpgroup
  int skip_pv[2];  // the last item whose P V the warpgroup did itself
  int start_b;
  int per;         // places of a run
  int end, limit;  // as in Walk
  Request start_r;
  int start_h;
  long long start_rem;
  unsigned long long warp_sum[16];
  unsigned int warp_units[16], warp_lo[16], warp_hi[16];  // units, their least and largest cost
  union {
    float2 x[kRows];  // joined unit: r, l of the second warpgroup, then f0, f1
    // 8-bit cache: of the query rows in a slot; all read before the first items
    // end, and so before x is written
    float row_scale[2][kRows];
  };
};
static_assert(sizeof(Misc) <= 2048, "Misc fits its place");

// One CTA's tail unit that others continue: what the join needs.
struct JoinDesc {
  int parts;   // 0: nothing to join
  int token0;  // first query row (token) of the unit
  int tokens;  // its tokens
  int h;
};

struct Ws {
  size_t desc, stats, o, total;
  __host__ __device__ explicit Ws(int D) {
    desc = 0;
    stats = desc + kMaxCtas * sizeof(JoinDesc);
    o = stats + size_t(kMaxCtas) * 2 * 2 * kRows * sizeof(float2);
    total = o + size_t(kMaxCtas) * 2 * 2 * kRows * D * sizeof(float);
  }
};

// ---- tensor memory ---------------------------------------------------------------
#define DSPARK_R8(r, i) \
  "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), \
      "=r"(r[i + 6]), "=r"(r[i + 7])
#define DSPARK_V8(r, i) \
  "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), \
      "r"(r[i + 6]), "r"(r[i + 7])
// Each lane of the warp reads (writes) 32 consecutive 32-bit columns of its lane.
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : DSPARK_R8(r, 0), DSPARK_R8(r, 8), DSPARK_R8(r, 16), DSPARK_R8(r, 24)
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
      DSPARK_V8(r, 0), DSPARK_V8(r, 8), DSPARK_V8(r, 16), DSPARK_V8(r, 24)
      : "memory");
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t a) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <int kCount>
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)),
               "n"(kCount)
               : "memory");
}

__device__ __forceinline__ bool elect_one() {  // one lane of a converged warp
  uint32_t p;
  asm volatile("{ .reg .pred q; elect.sync _|q, 0xFFFFFFFF; selp.u32 %0, 1, 0, q; }" : "=r"(p));
  return p != 0;
}

// D[tmem] (+)= A * B^T, kind::f16, A from shared (ss) or tensor (ts) memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Instruction descriptor: fp32 accumulator, both operands bf16 or fp16, A
// K-major, B K-major or (b_mn) MN-major.
__device__ constexpr uint32_t idesc_of(bool bf16, bool b_mn, int N) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}
// Descriptor of the values as the MN-major operand (N = head dimension, K =
// keys): 128-byte swizzled rows of 64 values; the next 64 values of N one half
// tile on (leading offset), the next 8 keys 1024 bytes on (stride offset).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((kKeys * 128) >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            int w, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar)),
      "l"(policy)
      : "memory");
}

// ---- small conversions -----------------------------------------------------------
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void unpack_f16(uint32_t w, float& lo, float& hi) {
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b; }"
      : "=f"(lo), "=f"(hi)
      : "r"(w));
}
__device__ __forceinline__ void unpack_bf16(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xFFFF0000u);
}
// Two e4m3 values (low 16 bits of w, or high) as two fp16, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{ .reg .b16 h; cvt.u16.u32 h, %1; cvt.rn.f16x2.e4m3x2 %0, h; }" : "=r"(r) : "r"(w));
  return r;
}

// Lane j of a quad holds four 16-byte parts y[4 i ..] of its own row; afterwards
// it holds part j of the quad's rows i = 0 .. 3 (two exchanges, as a 4 x 4
// matrix of parts is transposed).
__device__ __forceinline__ void quad_transpose16(uint32_t (&y)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d <= 2; d <<= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & d) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t& lo = y[4 * i + e];
        uint32_t& hi = y[4 * (i + d) + e];
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? lo : hi, d);
        if (up)
          lo = got;
        else
          hi = got;
      }
    }
  }
}

__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t phase) {  // no waiting
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(phase)
      : "memory");
  return ok != 0;
}

// A wait that gives up after kWaitLimitNs or when another warp has.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t phase, volatile int* fail,
                                        int32_t* status) {
  if (mbar_try_wait(bar, phase)) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (;;) {
    for (int i = 0; i < 8; ++i)
      if (mbar_try_wait_sleep(bar, phase, 2000u)) return true;
    if (*fail) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      report(status, DSPARK_ERR_TIMEOUT);
      *fail = 1;
      return false;
    }
  }
}

// The same for a whole warp, with one answer.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t phase, volatile int* fail,
                                          int32_t* status) {
  return __all_sync(0xFFFFFFFFu, wait_on(bar, phase, fail, status));
}

// A converter warp's wait for the n-th tile; false after the last, too.
__device__ __forceinline__ bool wait_raw(uint64_t* bar, uint32_t phase, Misc* m, uint32_t n,
                                         int32_t* status) {
  volatile int* fail = &m->fail;
  bool there = mbar_try_wait(bar, phase);
  if (!there) {
    const unsigned long long t0 = globaltimer_ns();
    while (!(there = mbar_try_wait_sleep(bar, phase, 500u))) {
      if (n >= *const_cast<volatile uint32_t*>(&m->total) || *fail) break;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        report(status, DSPARK_ERR_TIMEOUT);
        *fail = 1;
        break;
      }
    }
  }
  return __all_sync(0xFFFFFFFFu, there);
}

// Two barriers at once (their latencies overlap when both are through), and a
// third one that is only looked at: `c_through` says whether to, and comes back
// as whether it was through.
__device__ __forceinline__ bool wait_warp2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb,
                                           uint64_t* c, uint32_t pc, bool& c_through,
                                           volatile int* fail, int32_t* status) {
  const bool ra = mbar_try_wait(a, pa), rb = mbar_try_wait(b, pb);
  const bool rc = c_through && mbar_test_wait(c, pc);
  c_through = __all_sync(0xFFFFFFFFu, rc);
  if (__all_sync(0xFFFFFFFFu, ra && rb)) return true;
  return wait_warp(a, pa, fail, status) && wait_warp(b, pb, fail, status);
}

// A softmax warp's wait for tile n of a ring of kStages. A barrier only tells the
// parity of its phase, and this waiter has not seen every one before (as the MMA
// warp and the producers have), so the wait begins when the tile's stage is being
// filled, from when on the parity is unambiguous.
template <int kStages>
__device__ __forceinline__ bool wait_tile(Misc* m, uint32_t n, int32_t* status) {
  volatile int* fail = &m->fail;
  bool ok = true;
  if (static_cast<int>(*const_cast<volatile uint32_t*>(&m->filling) - n) <= 0) {
    const unsigned long long t0 = globaltimer_ns();
    do {
      __nanosleep(20);
      if (*fail) ok = false;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        report(status, DSPARK_ERR_TIMEOUT);
        *fail = 1;
        ok = false;
      }
    } while (ok && static_cast<int>(*const_cast<volatile uint32_t*>(&m->filling) - n) <= 0);
  }
  ok = ok && wait_on(&m->kv_full[n % kStages], (n / kStages) & 1, fail, status);
  return __all_sync(0xFFFFFFFFu, ok);
}

// ---- the units of work -------------------------------------------------------------
__device__ __forceinline__ Request load_request(const PagedAttentionParams& P, int b, bool tell) {
  Request r;
  const int a = P.query_start[b], e = P.query_start[b + 1];
  r.slot = P.rsi[b];
  r.len = P.seq_lens[b];
  r.q0 = a;
  r.n = e - a;
  bool bad = false;
  if (a < 0 || e < a || e > P.T) {
    r.n = 0;
    bad = true;
  }
  if (r.slot < 0) {
    r.len = 0;
  } else if (r.slot >= P.S || r.len < 0 ||
             static_cast<int64_t>(r.len) > (static_cast<int64_t>(P.M) << P.page_shift)) {
    r.len = 0;
    bad = true;
  }
  if (bad && tell) report(P.status, DSPARK_ERR_BOUNDS);
  return r;
}

// Key range [lo, hi) that tokens t0 .. t1 - 1 of a request can see.
__device__ __forceinline__ void key_range(const PagedAttentionParams& P, int n, int len, int t0,
                                          int t1, int& lo, int& hi) {
  const int at = len - n;
  hi = P.causal ? min(len, at + t1) : len;
  lo = P.window > 0 ? max(0, at + t0 - P.window + 1) : 0;
  if (hi <= lo) lo = hi = 0;
}

// Key tiles of a unit; a unit whose rows see nothing still has one (empty) tile.
__device__ __forceinline__ void unit_tiles(const PagedAttentionParams& P, const Request& r, int tp,
                                           int u, int& jb, int& je) {
  int lo, hi;
  key_range(P, r.n, r.len, u * 2 * tp, min(r.n, (u + 1) * 2 * tp), lo, hi);
  jb = lo / kKeys;
  je = max(jb + 1, (hi + kKeys - 1) / kKeys);
}

// The segments of this CTA in order. Positions count the units' costs from the
// run's start: the first kUnitTiles places of a unit stand for no tile. Units that
// start before `end` are this CTA's, up to `limit`.
struct Walk {
  const PagedAttentionParams& P;
  int tp, b, h, u, jb, je;
  int v;  // place within the unit
  int pos, end, limit, per;
  Request r;
  __device__ Walk(const PagedAttentionParams& P_, const Misc* m, int tp_)
      : P(P_), tp(tp_), b(m->start_b), h(0), u(0), pos(0), end(m->end), limit(m->limit),
        per(m->per) {
    if (pos >= end) return;
    r = m->start_r;
    h = m->start_h;
    long long rem = m->start_rem;
    for (;; ++u) {
      unit_tiles(P, r, tp, u, jb, je);
      if (rem < cost()) break;
      rem -= cost();
    }
    v = static_cast<int>(rem);
    if (limit > end && v != 0) {  // the CTA before takes the unit to its end
      pos += cost() - v;
      advance();
    }
  }
  __device__ int cost() const { return je - jb + kUnitTiles; }
  // To the next unit, if the run goes on.
  __device__ void advance() {
    if (pos >= end) return;
    if (++u * 2 * tp >= r.n) {
      u = 0;
      if (++h == P.kv.kv_heads) {
        h = 0;
        do {
          r = load_request(P, ++b, false);
        } while (r.n == 0);
      }
    }
    unit_tiles(P, r, tp, u, jb, je);
    v = 0;
  }
  __device__ bool next(Seg& s) {
    while (pos < end) {
      const int left = cost() - v;
      const int take = min(left, limit - pos);
      s.j0 = jb + max(0, v - kUnitTiles);
      s.j1 = jb + max(0, v + take - kUnitTiles);
      const bool some = s.j1 > s.j0;
      s.twin = false;
      if (some) {
        s.r = r;
        s.h = h;
        s.t0 = u * 2 * tp;
        s.t1 = min(r.n, s.t0 + 2 * tp);
        s.pair = s.t1 - s.t0 > tp;
        s.opens = s.j0 == jb;
        s.closes = s.j1 == je;
        s.after = static_cast<unsigned int>(pos + left - 1) / static_cast<unsigned int>(per);
        s.end = false;
        // the next unit is the next head's, of the same cost: all of it in this run?
        s.twin = s.opens && s.closes && r.n <= tp && h + 1 < P.kv.kv_heads &&
               pos + left < end && pos + left + cost() <= limit;
      }
      pos += take;
      v += take;
      if (s.twin) {
        pos += cost();
        ++h;
      }
      if (take == left) advance();
      if (some) return true;
    }
    return false;
  }
};

// Where this CTA's run starts: the key tiles of every request summed up (one
// request per thread, long prompts by whole warps), `pre` as scratch.
template <int kThreads>
__device__ void make_plan(const PagedAttentionParams& P, Misc* m, unsigned long long* pre, int tp) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = P.B;
  unsigned long long sum = 0;
  unsigned int n_units = 0, least = 0xFFFFFFFFu, largest = 0;  // of units' costs
  auto count = [&](const Request& o, int u) -> unsigned int {
    int jb, je;
    unit_tiles(P, o, tp, u, jb, je);
    const unsigned int c = je - jb + kUnitTiles;
    least = min(least, c);
    largest = max(largest, c);
    return c;
  };
  // each thread takes `each` consecutive requests, so that a scan of the
  // threads' sums gives the prefix
  const int each = (B + kThreads - 1) / kThreads;
  Request r;
  for (int i = 0; i < each; ++i) {
    const int b = tid * each + i;
    r.n = 0;
    if (b < B) r = load_request(P, b, blockIdx.x == 0);
    const int units = (r.n + 2 * tp - 1) / (2 * tp);
    unsigned long long cost = 0;
    const bool big = units > 4;
    n_units += min(units, 1 << 16);
    if (!big)
      for (int u = 0; u < units; ++u) cost += count(r, u);
    unsigned int todo = __ballot_sync(0xFFFFFFFFu, big);
    while (todo) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      Request o;
      o.n = __shfl_sync(0xFFFFFFFFu, r.n, src);
      o.len = __shfl_sync(0xFFFFFFFFu, r.len, src);
      const int ou = (o.n + 2 * tp - 1) / (2 * tp);
      unsigned long long c = 0;
      for (int u = lane; u < ou; u += 32) c += count(o, u);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) c += __shfl_xor_sync(0xFFFFFFFFu, c, s);
      if (lane == src) cost = c;
    }
    cost *= P.kv.kv_heads;
    sum += cost;
    if (b < B) pre[b] = sum;  // within the thread
  }
  unsigned long long v = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  n_units = __reduce_add_sync(0xFFFFFFFFu, n_units);
  least = __reduce_min_sync(0xFFFFFFFFu, least);
  largest = __reduce_max_sync(0xFFFFFFFFu, largest);
  if (lane == 31) {
    m->warp_sum[warp] = v;
    m->warp_units[warp] = n_units;
    m->warp_lo[warp] = least;
    m->warp_hi[warp] = largest;
  }
  __syncthreads();
  unsigned long long base = v - sum, total = 0;
  const int used = (B + 32 * each - 1) / (32 * each);  // warps that have requests
  for (int w = 0; w < used; ++w) {
    if (w < warp) base += m->warp_sum[w];
    total += m->warp_sum[w];
  }
  unsigned long long per =
      total >> 31 ? (total + gridDim.x - 1) / gridDim.x
                  : (static_cast<unsigned int>(total) + gridDim.x - 1) / gridDim.x;
  per = min(max(per, static_cast<unsigned long long>(kMinTiles)),
            static_cast<unsigned long long>(kMaxRun));
  const unsigned long long pos = per * blockIdx.x;
  if (tid == kThreads - 32) {  // (a warp that mostly has no request's start to find)
    // a run of whole units starts at most ceil(per / least) of them, and ends less
    // than one past its end
    unsigned int units = 0;
    least = 0xFFFFFFFFu, largest = 0;
    for (int w = 0; w < used; ++w) {
      units += m->warp_units[w];
      least = min(least, m->warp_lo[w]);
      largest = max(largest, m->warp_hi[w]);
    }
    units = min(units, 2 * gridDim.x) * P.kv.kv_heads;
    units = min(units, 2 * gridDim.x);
    // (32 bits: a run too long for them gains nothing from whole units)
    const unsigned int run = static_cast<unsigned int>(per);
    bool whole = P.whole;
    if (per < 0x1000000u && largest < 0x1000000u) {
      const unsigned long long most =
          static_cast<unsigned long long>((run + least - 1) / least) * largest;
      const unsigned int past =  // the longest run beyond an even one
          most - run < largest ? static_cast<unsigned int>(most - run) : largest;
      whole |= past * gridDim.x <= kSplitGain * gridDim.x + kSplitGainUnits * units;
    }
    m->per = static_cast<int>(per);
    m->end = total <= pos ? 0 : static_cast<int>(min(per, total - pos));
    m->limit = whole ? 0x7FFFFFFF : m->end;
  }
  for (int i = 0; i < each; ++i) {
    const int b = tid * each + i;
    if (b >= B) break;
    const unsigned long long lo = base + (i ? pre[b - 1] : 0), hi = base + pre[b];
    if (lo <= pos && pos < hi) {
      m->start_b = b;
      m->start_r = each == 1 ? r : load_request(P, b, false);
      const unsigned long long cost = (hi - lo) / P.kv.kv_heads;  // of a head
      const unsigned long long h =
          (hi - lo) >> 32 ? (pos - lo) / cost
                          : static_cast<unsigned int>(pos - lo) / static_cast<unsigned int>(cost);
      m->start_h = static_cast<int>(h);
      m->start_rem = static_cast<long long>(pos - lo - h * cost);
    }
  }
}

// ---- the kernel ----------------------------------------------------------------------
// kF16: the MMA's type is fp16 (fp16 rows, or an 8-bit cache), else bf16. kScaled:
// a 16-bit cache with key scales (apart, since the scale's sign in the issuer's
// descriptor and its size in the softmax are 1 to 2% of a short request's time).
template <int D, bool kF16, bool kQuant, bool kScaled>
__global__ void __launch_bounds__(Cfg<D, kQuant>::kThreads, 1)
paged_attention_kernel(const __grid_constant__ CUtensorMap tmap_q,
                       const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, PagedAttentionParams P) {
  using C = Cfg<D, kQuant>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  Misc* m = reinterpret_cast<Misc*>(smem + C::misc);
  volatile int* fail = &m->fail;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = P.Hq / P.kv.kv_heads;
  const int tp = kRows / G;  // tokens of a row tile
  const Ws ws(D);
  unsigned char* wsp = static_cast<unsigned char*>(P.workspace);

  // the launch after this one may be set up; the one before it ends further down
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 8) {  // a lane per index
    if (lane < C::kStages) {
      mbar_init(&m->kv_full[lane], kQuant ? 4 : 2);
      mbar_init(&m->kv_empty[lane], 2);
    }
    if (lane < C::kRaw) {
      mbar_init(&m->raw_full[lane], 1);
      mbar_init(&m->raw_empty[lane], 4);
    }
    if (lane < 2) {
      mbar_init(&m->q_full[lane], 1);
      mbar_init(&m->q_ready[lane], 4);
      mbar_init(&m->q_empty[lane], 8);  // the softmax warps
      mbar_init(&m->s_full[lane], 1);
      mbar_init(&m->p_ready[lane], 4);
      mbar_init(&m->o_full[lane], 1);
      mbar_init(&m->merge[lane], 4);
      mbar_init(&m->scanned[lane], 4);
      m->bad[lane] = m->skip_pv[lane] = -1;
    }
    if (lane == 0) {
      mbar_init(&m->merged, 8);
      mbar_init(&m->drain, 1);
      m->filling = 0;
      m->total = 0xFFFFFFFFu;
      m->fail = 0;
    }
    fence_mbar_init();
  }
  if (tid == 0) {
    tc::prefetch_tensormap(&tmap_q);
    tc::prefetch_tensormap(&tmap_k);
    tc::prefetch_tensormap(&tmap_v);
  }
  if (warp == 9) {
    tc::tmem_alloc(&m->tmem, 512);
    tc::tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  make_plan<C::kThreads>(P, m, reinterpret_cast<unsigned long long*>(smem + C::kv), tp);
  fence_proxy_async_smem();  // the plan's scratch is TMA's from here on
  tc::fence_before_thread_sync();
  __syncthreads();
  tc::fence_after_thread_sync();
  const uint32_t tmem = m->tmem;
  if (warp < 8) {
    // ---- softmax ------------------------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    const int w = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_t = tmem + lanes + w * kKeys;         // scores, then p
    const uint32_t o_t = tmem + lanes + 256 + w * 128;     // O
    constexpr float kOff = kF16 ? 7.0f : 0.0f;
    constexpr int kCols = kQuant ? 64 : 128;  // scores held at a time
    uint32_t n_q = 0, n_seg = 0, n_item = 0, n_scan = 0, n_merge = 0;
    uint32_t base = 0;  // tiles loaded before this segment
    bool tail_split = false;
    // (a product with the scores of what is masked, which are -inf, has to stay
    // -inf: the scale is not below the least positive number, whose products with
    // finite scores are 2^-21 at most)
    auto bounded = [](float x) { return fminf(fmaxf(x, 0x1p-149f), 3e38f); };
    const float sl0 = kQuant || kScaled ? fabsf(P.scale) * kLog2e : bounded(fabsf(P.scale) * kLog2e);
    const int tok = row / G;  // token within the row tile
    bool ok = true;
    for (;;) {
      if (!(ok = wait_warp(&m->q_full[n_q & 1], (n_q >> 1) & 1, fail, P.status))) break;
      Seg s = m->seg[n_q & 1];
      if (s.end) break;
      const uint32_t n_q1 = n_q + 1;
      if (s.two() && !(ok = wait_warp(&m->q_full[n_q1 & 1], (n_q1 >> 1) & 1, fail, P.status))) break;
      if (s.twin) s.h += w;  // this warpgroup's head
      // (the scales' signs are the queries', here or in the product: a masked
      // score is -inf and the largest score the largest exponent)
      const float k_scale = (kQuant || kScaled) && P.kv.k_scale ? P.kv.k_scale[s.h] : 1.f;
      float sl = kQuant || kScaled ? sl0 * fabsf(k_scale) : sl0;
      const int items = s.items(w);
      // one thread of the warpgroup gives back what its MMAs have read: a tile
      // once, or twice where the other warpgroup has no use for it
      const bool giver = (warp & 3) == 0 && lane == 0;
      // the query rows and the segment's description, of which every warp has its
      // copy by now, after this warpgroup's last scores
      auto give_queries = [&]() {
        if (lane == 0) {
          mbar_arrive(&m->q_empty[n_q & 1]);
          if (s.two()) mbar_arrive(&m->q_empty[n_q1 & 1]);
        }
      };
      if (items == 0) {
        __syncwarp();
        give_queries();
      }
      auto give_tile = [&](uint32_t n) {
        if (s.pair)
          mbar_arrive(&m->kv_empty[n % C::kStages]);
        else
          mbar_arrive_n<2>(&m->kv_empty[n % C::kStages]);
      };
      const bool split = !(s.opens && s.closes);
      const int first = s.t0 + (s.pair ? w * tp : 0);       // first token of the row tile
      const int ntok = min(tp, s.t1 - first);
      const int nrow = ntok * G;
      const bool live = row < nrow;
      const bool warp_live = (warp & 3) * 32 < nrow;
      int lo, hi;
      key_range(P, s.r.n, s.r.len, first + tok, first + tok + 1, lo, hi);
      if (!live) lo = hi = 0;
      // keys seen by every row of the tile
      int all_lo, all_hi, unused;
      key_range(P, s.r.n, s.r.len, first, first + 1, unused, all_hi);
      key_range(P, s.r.n, s.r.len, first + ntok - 1, first + ntok, all_lo, unused);
      if constexpr (kQuant) {
        // The row tile to fp16, in place, each row's largest value brought to 2^14
        // by a power of two: exact but for values 2^-28 below it. D / 8
        // neighbouring lanes hold a row.
        const uint32_t mine = n_q + (s.two() ? w : 0);
        float* scales = m->row_scale[mine & 1];
        if (s.two() || w == 0) {
          unsigned char* q_s = smem + C::q + (mine & 1) * C::kTileBytes;
          // (two rounds at once spill: 276 us for 272 with 256 x 4 tokens over 2-6k)
#pragma unroll 1
          for (int i = row; i < nrow * (D / 8); i += kRows) {
            const int rr = i / (D / 8), c = i % (D / 8);
            uint4* at = reinterpret_cast<uint4*>(q_s + (c >> 3) * (kRows * 128) + rr * 128 +
                                                 (((c & 7) ^ (rr & 7)) << 4));
            const uint4 x = *at;
            uint32_t xw[4] = {x.x, x.y, x.z, x.w};
            float v[8];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              if (P.dtype == DSPARK_F16)
                unpack_f16(xw[y], v[2 * y], v[2 * y + 1]);
              else
                unpack_bf16(xw[y], v[2 * y], v[2 * y + 1]);
            }
            uint32_t big = 0;
#pragma unroll
            for (int y = 0; y < 8; ++y) big = max(big, __float_as_uint(v[y]) & 0x7FFFFFFFu);
            const unsigned int who = ((1u << (D / 8)) - 1u) << (lane & ~(D / 8 - 1));
#pragma unroll
            for (int o = D / 16; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(who, big, o));
            const int ex = big == 0u ? 14 : max(static_cast<int>(big >> 23) - 127, -112);
            const float up =
                copysignf(__uint_as_float(static_cast<uint32_t>(14 - ex + 127) << 23), k_scale);
#pragma unroll
            for (int y = 0; y < 4; ++y) xw[y] = pack_f16(v[2 * y] * up, v[2 * y + 1] * up);
            if (c == 0) scales[rr] = __uint_as_float(static_cast<uint32_t>(ex - 14 + 127) << 23);
            *at = make_uint4(xw[0], xw[1], xw[2], xw[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&m->q_ready[mine & 1]);
        }
        // (A warpgroup without items has given the slot back: nothing keeps its next
        // phases from passing, so it neither waits for the rows nor reads their scales.)
        if (items > 0) {
          if (!(ok = wait_warp(&m->q_ready[mine & 1], (mine >> 1) & 1, fail, P.status))) break;
          if (live) sl *= scales[row];
        }
      }
      if (kQuant || kScaled) sl = bounded(sl);
      float r = -INFINITY, l = 0.f;  // reference (a score, not scaled), sum
      for (int k = 0; k < items; ++k, ++n_item) {
        const int key0 = s.tile(w, k) * kKeys;
        if (!(ok = wait_warp(&m->s_full[w], n_item & 1, fail, P.status))) break;
        tc::fence_after_thread_sync();
        if (giver) {  // these scores are there: the keys, and the values before
          give_tile(base + s.k_place(s.load_of(w, k)));
          if (!kQuant && k > 0) give_tile(base + s.v_place(s.load_of(w, k - 1)));
        }
        if (k == items - 1) give_queries();
        __syncwarp();
        bool scan = false, tail = false;
        const bool masked = key0 < all_lo || key0 + kKeys > all_hi;
        if (masked) {
          // keys past the request's end in this tile, and others that some row
          // does not see
          tail = key0 + kKeys > s.r.len;
          scan = key0 < all_lo || min(key0 + kKeys, s.r.len) > all_hi;
        }
        if (warp_live) {
          // (all 128 scores at once where the registers hold them, else 64 at a
          // time, read twice)
          uint32_t x[kCols];
          auto load = [&](int c0) {
#pragma unroll
            for (int c = 0; c < kCols; c += 32) tmem_ld32(s_t + c0 + c, x + c);
            tc::tmem_wait_ld();
            if (masked) {
              const int clo = lo - key0 - c0, chi = hi - key0 - c0;
#pragma unroll
              for (int g = 0; g < kCols; g += 32) {  // bit c: the row sees key g + c
                const int a = min(max(clo - g, 0), 32), z = min(max(chi - g, 0), 32);
                const uint32_t below = z == 32 ? 0xFFFFFFFFu : (1u << z) - 1u;
                const uint32_t sees = a == 32 ? 0u : below >> a << a;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!(sees >> c & 1u)) x[g + c] = 0xFF800000u;
              }
            }
          };
          float mx = -INFINITY;
#pragma unroll 1
          for (int c0 = 0; c0 < kKeys; c0 += kCols) {
            load(c0);
            float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
            for (int c = 0; c < kCols; c += 4) {
              mx0 = fmaxf(mx0, fmaxf(__uint_as_float(x[c]), __uint_as_float(x[c + 1])));
              mx1 = fmaxf(mx1, fmaxf(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])));
            }
            mx = fmaxf(mx, fmaxf(mx0, mx1));
          }
          const float grown = (mx - r) * sl;  // infinite the first time
          const bool move = grown > kGrow;
          if (move) r = mx;
          const float ref = r == -INFINITY ? 0.f : r * sl;
          float neg = kOff - ref;
          const bool far = live && fabsf(ref) > kFar;
          if (__any_sync(0xFFFFFFFFu, far || (move && k > 0))) {
            if (k > 0) {
              const float keep = move ? ex2_approx(-grown) : 1.f;
              l *= keep;
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(o_t + c, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tmem_st32(o_t + c, o);
              }
            }
            if (__any_sync(0xFFFFFFFFu, far)) {
              if (far) neg = kOff;
              const float off = far ? -r : 0.f;
              const unsigned long long off2 = f2_pack(off, off);
              auto take_off = [&](uint32_t* y, int n) {
#pragma unroll
                for (int c = 0; c < n; c += 2) {
                  float a, b;
                  f2_unpack(f2_add(f2_pack(__uint_as_float(y[c]), __uint_as_float(y[c + 1])), off2),
                            a, b);
                  y[c] = __float_as_uint(a);
                  y[c + 1] = __float_as_uint(b);
                }
              };
              if constexpr (kCols == kKeys) {
                take_off(x, kKeys);
              } else {  // where they are read again (what is masked will be again)
#pragma unroll 1
                for (int c = 0; c < kKeys; c += 32) {
                  uint32_t y[32];
                  tmem_ld32(s_t + c, y);
                  tc::tmem_wait_ld();
                  take_off(y, 32);
                  tmem_st32(s_t + c, y);
                }
                tmem_wait_st();
              }
            }
          }
          const unsigned long long sl2 = f2_pack(sl, sl), neg2 = f2_pack(neg, neg);
          unsigned long long sum = 0ull, sum1 = 0ull;
#pragma unroll 1
          for (int c0 = 0; c0 < kKeys; c0 += kCols) {
            if (kCols < kKeys) load(c0);
#pragma unroll
            for (int c = 0; c < kCols; c += 4) {
              if (c == 64) tmem_st32(s_t, x);
              float a, b, e, f;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sl2, neg2),
                        a, b);
              f2_unpack(f2_fma(f2_pack(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sl2,
                               neg2), e, f);
              a = ex2_approx(a);
              b = ex2_approx(b);
              e = ex2_approx(e);
              f = ex2_approx(f);
              sum = f2_add(sum, f2_pack(a, b));
              sum1 = f2_add(sum1, f2_pack(e, f));
              x[c / 2] = kF16 ? pack_f16(a, b) : pack_bf16(a, b);
              x[c / 2 + 1] = kF16 ? pack_f16(e, f) : pack_bf16(e, f);
            }
            // p takes the place of scores that have been read: columns c0 / 2 ..
            tmem_st32(s_t + (c0 + kCols) / 2 - 32, x + kCols / 2 - 32);
          }
          float a, b;
          f2_unpack(f2_add(sum, sum1), a, b);
          l += a + b;
          tmem_wait_st();
        }
        if (tail || scan) {
          // the tile's values: rows past the end become zero; a non-finite one
          // that some row does not see takes P V off the tensor core
          const uint32_t vi = base + s.v_place(s.load_of(w, k));
          unsigned char* v_s = smem + C::kv + (vi % C::kStages) * C::kTileBytes;
          if (!(ok = wait_tile<C::kStages>(m, vi, P.status))) break;
          const int key = key0 + row;
          if (key >= s.r.len) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
              *reinterpret_cast<uint4*>(v_s + (c >> 3) * (kKeys * 128) + row * 128 +
                                        (((c ^ row) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          } else if (scan && (key >= all_hi || key < all_lo)) {
            constexpr uint32_t kInf = kF16 ? 0x7C00u : 0x7F80u;
            bool bad = false;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const uint4 v = *reinterpret_cast<const uint4*>(
                  v_s + (c >> 3) * (kKeys * 128) + row * 128 + (((c ^ row) & 7) << 4));
              const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                bad |= (vw[e] & kInf) == kInf || ((vw[e] >> 16) & kInf) == kInf;
            }
            if (bad) m->bad[w] = static_cast<int>(n_item);
          }
          fence_proxy_async_smem();
          if (scan) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->scanned[w]);
            if (!(ok = wait_warp(&m->scanned[w], n_scan & 1, fail, P.status))) break;
            ++n_scan;
            if (*reinterpret_cast<volatile int*>(&m->bad[w]) == static_cast<int>(n_item)) {
              // O += P V of this tile by hand, over the keys each row sees
              if (warp_live) {
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                  uint32_t o[32];
                  if (k > 0) {
                    tmem_ld32(o_t + c0, o);
                    tc::tmem_wait_ld();
                  } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0u;
                  }
#pragma unroll 1
                  for (int c = 0; c < kKeys; ++c) {
                    const uint32_t pw = tmem_ld1(s_t + (c >> 1));
                    tc::tmem_wait_ld();
                    float p0, p1;
                    if (kF16)
                      unpack_f16(pw, p0, p1);
                    else
                      unpack_bf16(pw, p0, p1);
                    const float p = (c & 1) ? p1 : p0;
                    const bool sees = key0 + c >= lo && key0 + c < hi;
                    const unsigned char* vr =
                        v_s + (c0 >> 6) * (kKeys * 128) + c * 128;
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4) {
                      const uint4 v = *reinterpret_cast<const uint4*>(
                          vr + (((((c0 >> 3) & 7) + q4) ^ (c & 7)) << 4));
                      const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                      for (int e = 0; e < 4; ++e) {
                        float v0, v1;
                        if (kF16)
                          unpack_f16(vw[e], v0, v1);
                        else
                          unpack_bf16(vw[e], v0, v1);
                        uint32_t& o0 = o[8 * q4 + 2 * e];
                        uint32_t& o1 = o[8 * q4 + 2 * e + 1];
                        if (sees) {
                          o0 = __float_as_uint(fmaf(p, v0, __uint_as_float(o0)));
                          o1 = __float_as_uint(fmaf(p, v1, __uint_as_float(o1)));
                        }
                      }
                    }
                  }
                  tmem_st32(o_t + c0, o);
                }
                tmem_wait_st();
              }
              if (lane == 0) m->skip_pv[w] = static_cast<int>(n_item);
            }
          }
        }
        tc::fence_before_thread_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->p_ready[w]);
      }
      if (!ok) break;
      if (items > 0) {
        if (!(ok = wait_warp(&m->o_full[w], n_seg & 1, fail, P.status))) break;
        tc::fence_after_thread_sync();
        ++n_seg;
        if (!kQuant && giver) give_tile(base + s.v_place(s.load_of(w, items - 1)));
      }
      base += 2 * s.loads();
      n_q += s.two() ? 2 : 1;
      // ---- the segment's result -----------------------------------------------------
      // A joined segment's is f0 O_0 + f1 O_1: the first warpgroup works out the
      // factors, and each writes half of the columns.
      const bool joined = !s.two() && s.items(1) > 0;
      if (!s.two() && w == 1 && !joined) continue;
      float f0 = 1.f, f1 = 0.f;
      if (joined && w == 1) {
        m->x[row] = make_float2(r, l);
        tc::fence_before_thread_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->merge[1]);
        if (!(ok = wait_warp(&m->merge[0], n_merge & 1, fail, P.status))) break;
        tc::fence_after_thread_sync();
        const float2 f = m->x[row];
        f0 = f.x;
        f1 = f.y;
      } else {
        float keep1 = 0.f;
        if (joined) {
          if (!(ok = wait_warp(&m->merge[1], n_merge & 1, fail, P.status))) break;
          tc::fence_after_thread_sync();
          const float2 x1 = m->x[row];
          const float rn = fmaxf(r, x1.x);  // (scores of one row and head: the same scale)
          if (rn != -INFINITY) {
            f0 = ex2_approx((r - rn) * sl);
            keep1 = ex2_approx((x1.x - rn) * sl);
          }
          l = l * f0 + x1.y * keep1;
          r = rn;
        }
        const float f = l == 0.f ? 0.f
                        : split  ? 1.f
                                 : (P.kv.v_scale ? P.kv.v_scale[s.h] : 1.f) / l;
        f0 *= f;
        f1 = keep1 * f;
        if (joined) {
          m->x[row] = make_float2(f0, f1);
          tc::fence_before_thread_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&m->merge[0]);
        }
      }
      if (warp_live) {
        const bool none = f0 == 0.f && f1 == 0.f;  // nothing seen: O may hold anything
        const int64_t trow = static_cast<int64_t>(s.r.q0 + first + tok) * P.Hq + s.h * G +
                             (row - tok * G);
        const int64_t prow = ((static_cast<int64_t>(blockIdx.x) * 2 + (s.opens ? 1 : 0)) * 2 +
                              (s.pair ? w : 0)) * kRows + row;
        // a piece is 64 bytes of a row: 32 output values, or 16 of a partial O.
        // A lane's own row would cost a store a line each; the four lanes of a
        // quad trade 16-byte parts and write 64 bytes of each other's rows.
        unsigned char* mine = split ? wsp + ws.o + prow * D * 4
                                    : static_cast<unsigned char*>(P.out) + trow * D * 2;
        if (!live) mine = nullptr;
        unsigned char* to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          to[i] = reinterpret_cast<unsigned char*>(__shfl_sync(
                      0xFFFFFFFFu, reinterpret_cast<unsigned long long>(mine), (lane & ~3) + i));
        const uint32_t o_own = tmem + lanes + 256 + (joined ? 0 : w * 128);
        const int c0 = joined && w == 1 ? D / 2 : 0, c1 = joined && w == 0 ? D / 2 : D;
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_own + c, o);
          if (joined) {
            uint32_t o1[32];
            tmem_ld32(o_own + 128 + c, o1);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 + __uint_as_float(o1[e]) * f1);
          } else {
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f0);
          }
          if (none) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll 1
          for (int q = 0; q < (split ? 2 : 1); ++q) {
            uint32_t y[16];
            if (split) {
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = q ? o[16 + e] : o[e];
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float a = __uint_as_float(o[2 * e]), b = __uint_as_float(o[2 * e + 1]);
                y[e] = P.dtype == DSPARK_F16 ? pack_f16(a, b) : pack_bf16(a, b);
              }
            }
            quad_transpose16(y);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (to[i])
                *reinterpret_cast<uint4*>(to[i] + (split ? (c + 16 * q) * 4 : c * 2) +
                                          (lane & 3) * 16) =
                    make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
          }
        }
        if (live && !(joined && w == 1)) {
          if (split) {
            reinterpret_cast<float2*>(wsp + ws.stats)[prow] = make_float2(r * sl, l);
          } else if (P.lse) {
            P.lse[trow] = l == 0.f ? -INFINITY : (r * sl - kOff + lg2_approx(l)) * kLn2;
          }
        }
      }
      if (joined) {  // neither goes on while the other reads its O
        tc::fence_before_thread_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->merged);
        if (!(ok = wait_warp(&m->merged, n_merge & 1, fail, P.status))) break;
        ++n_merge;
      }
      if (split && s.opens) {
        tail_split = true;
        if (tid == 0) {
          JoinDesc d;
          d.parts = s.after + 1;
          d.token0 = s.r.q0 + s.t0;
          d.tokens = s.t1 - s.t0;
          d.h = s.h;
          reinterpret_cast<JoinDesc*>(wsp + ws.desc)[blockIdx.x] = d;
        }
      }
    }
    if (tid == 0 && !P.whole && (!tail_split || !ok))
      reinterpret_cast<JoinDesc*>(wsp + ws.desc)[blockIdx.x].parts = 0;
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
    if (warp == 8 || (!kQuant && warp == 10)) {
      // ---- TMA producers: keys and values of the segments' tiles, page by page -------
      const uint64_t pol = policy_evict_normal();
      constexpr uint32_t kRing = kQuant ? C::kRaw : C::kStages;
      constexpr int kBytes = kQuant ? C::kRawBytes : C::kTileBytes;
      uint64_t* full = kQuant ? m->raw_full : m->kv_full;
      uint64_t* empty = kQuant ? m->raw_empty : m->kv_empty;
      unsigned char* ring = smem + (kQuant ? C::raw : C::kv);
      const int page = 1 << P.page_shift;
      const int box = page < kKeys ? page : kKeys;  // tokens of a TMA box
      const int boxes = kKeys / box;                // boxes of a tile's 128 bytes of width
      // this warp's boxes: every second one, one to a lane (8-bit: all)
      const int pi = kQuant ? 0 : warp == 10;
      const int bi = kQuant ? lane : 2 * lane + pi;
      const int nb = boxes * (kQuant ? 1 : C::kHalves);
      const int mine = kQuant ? nb : (nb + 1 - pi) / 2;
      const int bc = bi / boxes, bk = (bi - bc * boxes) * box;  // half of the row, first key
      uint32_t base = 0;                            // tiles loaded before this segment
      bool ok = true;
      Walk walk(P, m, tp);
      Seg s;
      while (ok && walk.next(s)) {
        int lo, hi;
        key_range(P, s.r.n, s.r.len, s.t0, s.t1, lo, hi);
        const int64_t row0 = static_cast<int64_t>(s.r.slot < 0 ? 0 : s.r.slot) * P.M;
        // this lane's page of tile j; num_blocks (which TMA reads as zeros) where
        // there is nothing to see
        auto page_of = [&](int j) -> int {
          const int key = j * kKeys + bk;
          if (bi >= nb || key >= hi || key + box <= lo) return P.kv.num_blocks;
          const int id = P.block_table[row0 + (key >> P.page_shift)];
          if (id >= 0 && id < P.kv.num_blocks) return id;
          report(P.status, DSPARK_ERR_BOUNDS);
          return P.kv.num_blocks;
        };
        auto load = [&](const CUtensorMap* map, int i, int id, int place) -> bool {
          const uint32_t n = base + place, st = n % kRing, ph = (n / kRing) & 1;
          if (!wait_warp(&empty[st], ph ^ 1, fail, P.status)) return false;
          if (lane == 0) {
            if (!kQuant && pi == 0) *const_cast<volatile uint32_t*>(&m->filling) = n + 1;
            if (mine > 0)
              mbar_arrive_expect_tx(&full[st], mine * box * (kQuant ? D : 128));
            else
              mbar_arrive(&full[st]);
          }
          __syncwarp();
          if (bi < nb) {
            const int y = (s.load_tile(i) * kKeys + bk) & (page - 1);
            unsigned char* dst = ring + st * kBytes + bk * (kQuant ? D : 128);
            tma_load_4d(dst + bc * (kKeys * 128), map, bc * 64, y, s.load_head(i), id, &full[st],
                        pol);
          }
          return true;
        };
        // the pages of a tile are looked up a tile before it is due
        const int nt = s.loads(), a = s.ahead();  // keys `a` tiles ahead of the values
        int id_next = page_of(s.j0), id_v0 = 0, id_v1 = 0;  // of the tiles one and two before
        for (int i = 0; i < nt + a && ok; ++i) {
          const int id_k = id_next;
          if (i + 1 < nt) id_next = page_of(s.load_tile(i + 1));
          if (i >= a) ok = load(&tmap_v, i - a, a == 2 ? id_v1 : id_v0, s.v_place(i - a));
          if (ok && i < nt) ok = load(&tmap_k, i, id_k, s.k_place(i));
          id_v1 = id_v0;
          id_v0 = id_k;
        }
        base += 2 * nt;
      }
      if (kQuant && lane == 0) *const_cast<volatile uint32_t*>(&m->total) = base;
    } else if (warp == 11) {
      // ---- scout: segments and their query rows ---------------------------------------
      uint32_t n_q = 0;
      bool ok = true;
      Walk walk(P, m, tp);
      Seg s;
      for (;;) {
        const bool more = walk.next(s);
        s.end = !more;
        const int fills = more && s.two() ? 2 : 1;
        for (int f = 0; f < fills && ok; ++f, ++n_q) {
          const uint32_t sl = n_q & 1;
          if (!(ok = wait_warp(&m->q_empty[sl], ((n_q >> 1) & 1) ^ 1, fail, P.status))) break;
          if (f == 0 && lane == 0) m->seg[sl] = s;
          const int tok0 = s.r.q0 + s.t0 + (s.pair ? f * tp : 0);
          const int head = s.h + (s.twin ? f : 0);
          if (lane == 0) {
            if (more) {
              mbar_arrive_expect_tx(&m->q_full[sl], C::kHalves * 128 * G * tp);
#pragma unroll
              for (int c = 0; c < C::kHalves; ++c)
                tc::tma_load_3d(smem + C::q + sl * C::kTileBytes + c * (kRows * 128), &tmap_q,
                                c * 64, head * G, tok0, &m->q_full[sl], policy_evict_normal());
            } else {
              mbar_arrive(&m->q_full[sl]);
            }
          }
        }
        if (!more || !ok) break;
      }
    } else if (warp == 9) {
      // ---- MMA issuer ------------------------------------------------------------------
      // The whole warp runs the loop, so that descriptors stay in uniform
      // registers; one elected lane issues.
      constexpr uint32_t id_pv = idesc_of(!kF16, true, D);
      // (a negative scale is a negated A; the rows beside an 8-bit cache come with
      // their head's sign)
      const uint32_t id_qk = idesc_of(!kF16, false, kKeys) | (P.scale < 0.f ? 1u << 13 : 0u);
      // (a vote, so that the descriptor stays in a uniform register)
      auto id_of = [&](int h) {  // (kScaled)
        return id_qk ^ (__any_sync(0xFFFFFFFFu, P.kv.k_scale[h] < 0.f) ? 1u << 13 : 0u);
      };
      const bool leader = elect_one();
      const uint64_t q_desc = tc::sw128_kmajor_desc(smem_addr(smem + C::q));
      const uint64_t k_desc = tc::sw128_kmajor_desc(smem_addr(smem + C::kv));
      const uint64_t v_desc = sw128_mnmajor_desc(smem_addr(smem + C::kv));
      uint32_t base = 0, n_q = 0, n_item0 = 0, n_item1 = 0;
      bool ok = true;
      while (ok) {
        if (!wait_warp(&m->q_full[n_q & 1], (n_q >> 1) & 1, fail, P.status)) break;
        const Seg s = m->seg[n_q & 1];
        if (s.end) break;
        const uint32_t n_q1 = n_q + 1;
        uint64_t* there = kQuant ? m->q_ready : m->q_full;
        if (kQuant && !wait_warp(&there[n_q & 1], (n_q >> 1) & 1, fail, P.status)) break;
        if (s.two() && !wait_warp(&there[n_q1 & 1], (n_q1 >> 1) & 1, fail, P.status)) break;
        tc::fence_after_thread_sync();
        const int nt = s.loads(), ni = s.pair ? 2 * nt : nt;
        uint32_t id0 = id_qk, id1 = id_qk;
        if constexpr (kScaled) {
          id0 = id_of(s.h);
          id1 = s.twin ? id_of(s.h + 1) : id0;
        }
        auto keys_of = [&](int i) { return base + s.k_place(s.pair ? i >> 1 : i); };
        auto scores = [&](int i, uint32_t ki) {  // S_w = Q K^T of item i
          const int w = i & 1;
          const uint32_t sl = (n_q + (s.two() ? w : 0)) & 1;
          const uint64_t qd = q_desc + static_cast<uint32_t>((sl * C::kTileBytes) >> 4);
          const uint64_t kd =
              k_desc + static_cast<uint32_t>(((ki % C::kStages) * C::kTileBytes) >> 4);
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            const uint32_t off = ((c >> 2) * (kRows * 128) + (c & 3) * 32) >> 4;
            mma_ss(tmem + w * kKeys, qd + off, kd + off, kScaled && w ? id1 : id0, c != 0);
          }
          tc::mma_commit(&m->s_full[w]);
        };
        for (int i = 0; i < 2 && i < ni; ++i) {
          const uint32_t ki = keys_of(i);
          if (!(ok = wait_warp(&m->kv_full[ki % C::kStages], (ki / C::kStages) & 1, fail,
                               P.status)))
            break;
          tc::fence_after_thread_sync();
          if (leader) scores(i, ki);
          __syncwarp();
        }
        for (int i = 0; i < ni && ok; ++i) {  // O_w += P_w V of item i, S_w of item i + 2
          const int w = i & 1;
          const uint32_t vi = base + s.v_place(s.pair ? i >> 1 : i);
          const uint32_t n = w ? n_item1 : n_item0;
          const bool more = i + 2 < ni;
          const uint32_t ki = keys_of(more ? i + 2 : i);
          // values, probabilities; the next keys, if they are there already (behind
          // the converters of an 8-bit cache they hardly ever are)
          bool keys = more && !kQuant;
          if (!(ok = wait_warp2(&m->kv_full[vi % C::kStages], (vi / C::kStages) & 1,
                                &m->p_ready[w], n & 1, &m->kv_full[ki % C::kStages],
                                (ki / C::kStages) & 1, keys, fail, P.status)))
            break;
          tc::fence_after_thread_sync();
          const bool skip = *reinterpret_cast<volatile int*>(&m->skip_pv[w]) == static_cast<int>(n);
          const uint64_t vd =
              v_desc + static_cast<uint32_t>(((vi % C::kStages) * C::kTileBytes) >> 4);
          const uint32_t o_d = tmem + 256 + w * 128, p_d = tmem + w * kKeys;
          if (leader) {
            if (!skip) {
#pragma unroll
              for (int c = 0; c < kKeys / 16; ++c)
                mma_ts(o_d, p_d + c * 8, vd + ((c * 2048) >> 4), id_pv, i >= 2 || c != 0);
            }
            if constexpr (kQuant) {  // few stages: values are given back at once
              tc::mma_commit(&m->kv_empty[vi % C::kStages]);
              if (!s.pair) tc::mma_commit(&m->kv_empty[vi % C::kStages]);
            }
            if (!more) tc::mma_commit(&m->o_full[w]);
            if (keys) scores(i + 2, ki);
          }
          __syncwarp();
          if (more && !keys) {
            if (!(ok = wait_warp(&m->kv_full[ki % C::kStages], (ki / C::kStages) & 1, fail,
                                 P.status)))
              break;
            tc::fence_after_thread_sync();
            if (leader) scores(i + 2, ki);
            __syncwarp();
          }
          n_item0 += w == 0;
          n_item1 += w == 1;
        }
        base += 2 * nt;
        n_q += s.two() ? 2 : 1;
      }
      if (leader) {
        tc::mma_commit(&m->drain);
        (void)mbar_wait(&m->drain, 0, P.status);
      }
    } else if (kQuant && (warp == 10 || warp >= 13)) {
      // ---- e4m3 tiles to fp16, in the MMA's layout ---------------------------------------
      if constexpr (kQuant) {
        const int ct = warp == 10 ? lane : tid - 12 * 32;  // 0..127: a key each
        constexpr int kChunks = D / 16;
        for (uint32_t n = 0;; ++n) {
          const uint32_t rs = n % C::kRaw, st = n % C::kStages;
          if (!wait_raw(&m->raw_full[rs], (n / C::kRaw) & 1, m, n, P.status)) break;
          const unsigned char* src = smem + C::raw + rs * C::kRawBytes + ct * D;
          uint4 x[kChunks];
          // TMA swizzled the 16-byte pieces of a row by the row: 8 rows of 128
          // bytes, or of 64 bytes two to a 128-byte line
          const int sw = D == 128 ? ct & 7 : (ct >> 1) & 3;
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            x[c] = *reinterpret_cast<const uint4*>(src + ((c ^ sw) << 4));
          __syncwarp();
          if (lane == 0) mbar_arrive(&m->raw_empty[rs]);
          if (!wait_warp(&m->kv_empty[st], ((n / C::kStages) & 1) ^ 1, fail,
                       P.status))
            break;
          if (ct == 0) *const_cast<volatile uint32_t*>(&m->filling) = n + 1;
          unsigned char* dst = smem + C::kv + st * C::kTileBytes + ct * 128;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const uint32_t xw[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int ch = 2 * c + e;  // 16-byte piece of the fp16 row
              *reinterpret_cast<uint4*>(dst + (ch >> 3) * (kKeys * 128) +
                                        (((ch & 7) ^ (ct & 7)) << 4)) =
                  make_uint4(e4m3x2_to_f16x2(xw[2 * e] & 0xFFFFu), e4m3x2_to_f16x2(xw[2 * e] >> 16),
                             e4m3x2_to_f16x2(xw[2 * e + 1] & 0xFFFFu),
                             e4m3x2_to_f16x2(xw[2 * e + 1] >> 16));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&m->kv_full[st]);
        }
      }
    }
  }
  tc::fence_before_thread_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_thread_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  // Every copy was waited for by the MMAs that read it; after a failed wait some
  // may still be on their way: they land before the CTA exits.
  if (tid == 0 && *fail) {
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) __nanosleep(1000);
  }
}

// Joins the partial results of the units that more than one CTA worked on: the
// unit that CTA blockIdx.x opened, from its tail part and the head parts of
// the CTAs after it, in that order. A warp per row; its lanes split the row, and
// eight parts are loaded at a time, beside the statistics that weigh them (one
// part after the other, 19 parts of a long request took 7 us of latency).
template <int D>
__global__ void __launch_bounds__(256) paged_join_kernel(PagedAttentionParams P, int off) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Ws ws(D);
  const unsigned char* wsp = static_cast<const unsigned char*>(P.workspace);
  const int c = blockIdx.x;
  const JoinDesc d = reinterpret_cast<const JoinDesc*>(wsp + ws.desc)[c];
  if (d.parts == 0) return;
  const int G = P.Hq / P.kv.kv_heads, tp = kRows / G;
  const int lane = threadIdx.x & 31;
  const float2* stats = reinterpret_cast<const float2*>(wsp + ws.stats);
  const float* po = reinterpret_cast<const float*>(wsp + ws.o);
  constexpr int kPer = D / 32, kBatch = 8;
  const float vs = P.kv.v_scale ? P.kv.v_scale[d.h] : 1.f;
  const int rows = d.tokens * G;
  for (int i = blockIdx.y * 8 + (threadIdx.x >> 5); i < rows; i += gridDim.y * 8) {
    const int tok = i / G, g = i - tok * G;
    const int place = (tok / tp) * kRows + (tok % tp) * G + g;  // row tile, row
    auto at = [&](int p) -> int64_t {
      return (static_cast<int64_t>(c + p) * 2 + (p == 0 ? 1 : 0)) * 2 * kRows + place;
    };
    float r = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = 0.f;
    for (int p0 = 0; p0 < d.parts; p0 += kBatch) {
      float2 x = make_float2(-INFINITY, 0.f);
      if (lane < kBatch && p0 + lane < d.parts) x = stats[at(p0 + lane)];
      float v[kBatch][kPer];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int e = 0; e < kPer; e += 2) {
          float2 y = make_float2(0.f, 0.f);
          if (p0 + b < d.parts)
            y = *reinterpret_cast<const float2*>(po + at(p0 + b) * D + lane * kPer + e);
          v[b][e] = y.x;
          v[b][e + 1] = y.y;
        }
      float m = x.x;
#pragma unroll
      for (int s = kBatch / 2; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, s));
      const float rn = fmaxf(r, __shfl_sync(0xFFFFFFFFu, m, 0));
      const float rb = rn == -INFINITY ? 0.f : rn;
      const float old = ex2_approx(r - rb);
      r = rn;
      l *= old;
#pragma unroll
      for (int e = 0; e < kPer; ++e) o[e] *= old;
      const float keep = ex2_approx(x.x - rb), mass = x.y * keep;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        l += __shfl_sync(0xFFFFFFFFu, mass, b);
        const float k = __shfl_sync(0xFFFFFFFFu, keep, b);
#pragma unroll
        for (int e = 0; e < kPer; ++e) o[e] = fmaf(v[b][e], k, o[e]);
      }
    }
    const bool none = l == 0.f;
    const float inv = none ? 0.f : vs / l;
    const int64_t row = static_cast<int64_t>(d.token0 + tok) * P.Hq + d.h * G + g;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(P.out) + row * D +
                                                lane * kPer);
#pragma unroll
    for (int e = 0; e < kPer; e += 2) {
      const float a = none ? 0.f : o[e] * inv, b = none ? 0.f : o[e + 1] * inv;
      out[e / 2] = P.dtype == DSPARK_F16 ? pack_f16(a, b) : pack_bf16(a, b);
    }
    if (P.lse && lane == 0) P.lse[row] = none ? -INFINITY : (r - off + lg2_approx(l)) * kLn2;
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<EncodeTiledFn>(fn);
}

// [num_blocks, kv_heads, page_size, head_dim] with the cache's strides; a box
// is 64 values (8-bit: a whole row) of up to 128 tokens of one page and head.
bool make_map(CUtensorMap* map, void* base, const dspark_paged_kv& kv, int64_t block, int64_t head,
              int64_t token) {
  static const EncodeTiledFn encode = encode_fn();  // the driver's entry point
  if (!encode) return false;
  const bool quant = kv.dtype == DSPARK_E4M3;
  const cuuint64_t es = quant ? 1 : 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kv.head_dim),
                              static_cast<cuuint64_t>(kv.page_size),
                              static_cast<cuuint64_t>(kv.kv_heads),
                              static_cast<cuuint64_t>(kv.num_blocks)};
  // (the stride of an axis of one is not used)
  const cuuint64_t strides[3] = {token * es, (kv.kv_heads > 1 ? head : token) * es,
                                 (kv.num_blocks > 1 ? block : token) * es};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(quant ? kv.head_dim : 64),
                             static_cast<cuuint32_t>(kv.page_size < kKeys ? kv.page_size : kKeys),
                             1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUtensorMapDataType type = quant ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : kv.dtype == DSPARK_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                            : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle swizzle = quant && kv.head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                                : CU_TENSOR_MAP_SWIZZLE_128B;
  return encode(map, type, 4, base, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// [T, q_heads, head_dim] with the tokens' stride; a box is 64 values of the
// query heads of a key head, of as many tokens as a row tile holds.
bool make_q_map(CUtensorMap* map, const PagedAttentionParams& p) {
  static const EncodeTiledFn encode = encode_fn();
  if (!encode) return false;
  const int G = p.Hq / p.kv.kv_heads, D = p.kv.head_dim;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p.Hq),
                              static_cast<cuuint64_t>(p.T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2,
                                 static_cast<cuuint64_t>(p.q_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(kRows / G)};
  const cuuint32_t one[3] = {1, 1, 1};
  return encode(map,
                p.dtype == DSPARK_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                3, const_cast<void*>(p.q), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kF16, bool kQuant, bool kScaled>
cudaError_t launch(const PagedAttentionParams& p, const CUtensorMap& mq, const CUtensorMap& mk,
                   const CUtensorMap& mv, int sms, cudaStream_t stream) {
  using C = Cfg<D, kQuant>;
  cudaError_t err =
      cudaFuncSetAttribute(paged_attention_kernel<D, kF16, kQuant, kScaled>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (err != cudaSuccess) return err;
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  // both launches may be set up while the one before them ends, and wait for it
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, paged_attention_kernel<D, kF16, kQuant, kScaled>, mq, mk, mv, p);
  if (err != cudaSuccess || p.whole) return err;
  cfg.gridDim = dim3(grid, 16);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, p, kF16 ? 7 : 0);
}

template <int D>
cudaError_t launch_dim(const PagedAttentionParams& p, const CUtensorMap& mq, const CUtensorMap& mk,
                       const CUtensorMap& mv, int sms, cudaStream_t stream) {
  if (p.kv.dtype == DSPARK_E4M3) return launch<D, true, true, false>(p, mq, mk, mv, sms, stream);
  if (p.kv.k_scale)
    return p.dtype == DSPARK_F16 ? launch<D, true, false, true>(p, mq, mk, mv, sms, stream)
                                 : launch<D, false, false, true>(p, mq, mk, mv, sms, stream);
  return p.dtype == DSPARK_F16 ? launch<D, true, false, false>(p, mq, mk, mv, sms, stream)
                               : launch<D, false, false, false>(p, mq, mk, mv, sms, stream);
}

}  // namespace

size_t paged_attention_workspace_bytes(int B, int Hq, int Hkv, int D) {
  (void)B;
  (void)Hq;
  (void)Hkv;
  return Ws(D).total;
}

cudaError_t launch_paged_attention(PagedAttentionParams p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess)
    err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess) return err;
  CUtensorMap mq = {}, mk, mv;
  const dspark_paged_kv& kv = p.kv;
  // the most key tiles a unit can have
  int64_t keys = static_cast<int64_t>(p.M) << p.page_shift;
  if (p.window > 0) {
    // (without a causal mask a unit sees from its first token's window to the end)
    const int64_t tokens = p.causal ? 2 * (kRows / (p.Hq / kv.kv_heads)) : p.T;
    keys = min(keys, p.window + tokens);
  }
  p.whole = (keys + kKeys - 1) / kKeys + (p.window > 0 ? 1 : 0) <=
            (3 * p.B * kv.kv_heads >= sms ? kWholeTiles : kWholeTilesFewUnits);
  if (!make_map(&mk, kv.k, kv, kv.k_block_stride, kv.k_head_stride, kv.k_token_stride) ||
      !make_map(&mv, kv.v, kv, kv.v_block_stride, kv.v_head_stride, kv.v_token_stride))
    return cudaErrorInvalidValue;
  if (!make_q_map(&mq, p)) return cudaErrorInvalidValue;
  return kv.head_dim == 64 ? launch_dim<64>(p, mq, mk, mv, sms, stream)
                           : launch_dim<128>(p, mq, mk, mv, sms, stream);
}

}  // namespace dspark
