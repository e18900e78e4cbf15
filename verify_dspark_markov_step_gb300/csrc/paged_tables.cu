// paged_tables.cu -- a step's block tables, query offsets, positions and slot
// map from the request lengths, in one launch.
//
// The step is three prefix sums over the requests (new tokens; blocks
// returned and taken; new tokens and taken blocks of the requests that can be
// served) and then independent work per token and per block: a token finds
// its request by bisection of the offsets, and the i-th block taken is the
// i-th entry from the top of the free stack, which is either in free_blocks
// or, if requests return blocks in the same step, one of their table entries.
//
// Every CTA computes the prefix sums for itself (one request per thread, at
// most 1024: two dependent rounds of loads and three scans) and then
// takes its share of the tokens, so no CTA waits for another. What the others
// still read -- held counts, cached lengths, the pool, the table entries of
// returned blocks -- is changed by the CTA that finishes last, found with a
// counter that it resets. Table entries that are new and stack entries above
// the old top are read by nobody and are written at once.
//
// Bound: latency. A decode step is one CTA: two dependent rounds of loads, three
// scans, a dependent round for the tokens (32 requests x 8 tokens: 4.5 us back to
// back, 8.5 with cold caches). For long prompts a thread places eight tokens, each
// by a bisection and a dependent load (256 requests, room for 262 thousand tokens,
// 4.2 MB of positions and slots: 9.6 us, 11.7 cold; the bytes alone are 0.6). Where
// blocks are shared, a request's thread looks at two blocks, and warps at those of a length
// that was lowered, two more dependent rounds of loads each: 32 requests x 8 tokens 4.1 us
// for 3.6 without, 1024 x 8 9.1 for 7.5; one row lowered by 65536 blocks 24 us (a block after
// the other 4575; every row by warps alone, 1024 x 8 38.8).
#include <cuda_runtime.h>
#include <stdint.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "paged.h"

namespace dspark {

namespace {

// Tokens per CTA: 8 per thread at 256 threads. Fewer would repeat the prefix
// sums for little work, more would leave SMs idle in mid-sized steps.
constexpr int kTokensPerCta = 2048;
constexpr int kMaxB = DSPARK_MAX_PAGED_BATCH;
// Where blocks are shared: those of a request that its thread looks at, and of a longer
// one that a warp looks at in one go.
constexpr int kFew = 2, kLook = 256;

struct TablesSmem {
  unsigned long long warp[33];
  int start[kMaxB + 1];   // first new token of each request
  int cached[kMaxB];
  int slot[kMaxB];        // row of the block table
  int held[kMaxB];
  int need[kMaxB];        // = held for a request that is not served
  int take0[kMaxB];       // blocks taken by the requests before
  int after[kMaxB];       // blocks returned by the requests after
  int last;
  int n_long;
};

__device__ __forceinline__ bool is_shared(const PagedTablesParams& P, int id) {
  return id >= 0 && id < P.N && P.shares[id] > 0;
}

template <bool kShared>
__global__ void __launch_bounds__(1024) paged_tables_kernel(PagedTablesParams P) {
  __shared__ TablesSmem sm;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int B = P.B, M = P.M, N = P.N, T = P.T, sh = P.page_shift;
  const bool first = blockIdx.x == 0;  // reports errors

  // ---- the request of this thread --------------------------------------------
  int slot = -1, held = 0;
  int64_t cached = 0, fresh = 0, need = 0;
  bool ok = false;
  int count = 0;
  if (B > 0) count = P.pool[0];
  if (count < 0 || count > N) {
    if (first && tid == 0) report(P.status, DSPARK_ERR_BOUNDS);
    count = count < 0 ? 0 : N;
  }
  if (tid < B) {
    slot = P.rsi[tid];
    fresh = P.new_lens[tid];
    const int acc = P.num_accepted ? P.num_accepted[tid] : -1;
    if (slot >= 0) {
      if (slot < P.S) {
        held = P.held_blocks[slot];
        const int c = P.cached_lens[slot];
        cached = static_cast<int64_t>(c) + acc + 1;
        need = (cached + fresh + (1 << sh) - 1) >> sh;
        ok = acc >= -1 && c >= 0 && fresh >= 0 && held >= 0 && held <= M && need <= M;
      }
    }
  }
  if constexpr (kShared) {
    // A block that other rows hold too is not this call's to put on the stack, nor new
    // tokens' to write into. A step's are one or two; a length that was lowered leaves as
    // many as the row holds, which the warps share out.
    if (tid == 0) sm.n_long = 0;
    __syncthreads();
    bool listed = false;
    if (ok) {
      const int j0 = static_cast<int>(fresh > 0 ? cached >> sh : need);
      const int32_t* row = P.block_table + static_cast<int64_t>(slot) * M;
#pragma unroll
      for (int u = 0; u < kFew; ++u)
        if (j0 + u < held && is_shared(P, row[j0 + u])) ok = false;
      listed = ok && j0 + kFew < held;
      if (listed) {
        const int i = atomicAdd(&sm.n_long, 1);
        sm.take0[i] = tid;
        sm.slot[tid] = slot;
        sm.held[tid] = held;
        sm.need[tid] = j0 + kFew;
        sm.after[tid] = 0;  // one was found
      }
    }
    __syncthreads();
    const int n_long = sm.n_long, parts = n_long < nw ? nw / max(n_long, 1) : 1;
    for (int w = warp; w < n_long * parts; w += nw) {
      const int b = sm.take0[w / parts], end = sm.held[b];
      const int32_t* row = P.block_table + static_cast<int64_t>(sm.slot[b]) * M;
      bool found = false;
      for (int j = sm.need[b] + w % parts * kLook; j < end && !found; j += parts * kLook) {
        int id[kLook / 32];  // (all on their way before the first count is)
#pragma unroll
        for (int u = 0; u < kLook / 32; ++u)
          id[u] = j + 32 * u + lane < end ? row[j + 32 * u + lane] : -1;
#pragma unroll
        for (int u = 0; u < kLook / 32; ++u) found |= is_shared(P, id[u]);
        found = __any_sync(0xFFFFFFFFu, found);
      }
      if (found && lane == 0) sm.after[b] = 1;
    }
    __syncthreads();
    if (listed && sm.after[tid]) ok = false;
  }
  if (tid < B && slot >= 0 && !ok && first) report(P.status, DSPARK_ERR_BOUNDS);
  unsigned long long total;
  const unsigned long long tcum = block_scan(ok ? fresh : 0, sm.warp, &total);
  if (ok && fresh != 0 && tcum > static_cast<unsigned long long>(T)) {
    ok = false;
    if (first) report(P.status, DSPARK_ERR_BOUNDS);
  }
  const unsigned int release = ok && held > need ? static_cast<unsigned int>(held - need) : 0u;
  unsigned int take = ok && need > held ? static_cast<unsigned int>(need - held) : 0u;
  const unsigned long long rt =
      block_scan((static_cast<unsigned long long>(release) << 32) | take, sm.warp, &total);
  const unsigned int released = static_cast<unsigned int>(total >> 32);
  const int64_t top = static_cast<int64_t>(count) + released;
  if (take != 0u && static_cast<int64_t>(rt & 0xFFFFFFFFull) > top) {
    ok = false;
    take = 0u;
    if (first) report(P.status, DSPARK_ERR_CACHE_FULL);
  }
  if (first && tid == 0 && top > N) report(P.status, DSPARK_ERR_BOUNDS);
  const unsigned long long nt = block_scan(
      (static_cast<unsigned long long>(ok ? fresh : 0) << 32) | take, sm.warp, &total);
  const int tokens = static_cast<int>(total >> 32);
  const unsigned int taken = static_cast<unsigned int>(total);
  const int n = ok ? static_cast<int>(fresh) : 0;
  if (tid < B) {
    sm.start[tid] = static_cast<int>(nt >> 32) - n;
    sm.cached[tid] = static_cast<int>(cached);
    sm.slot[tid] = ok ? slot : -1;
    sm.held[tid] = held;
    sm.need[tid] = ok ? static_cast<int>(need) : held;
    sm.take0[tid] = static_cast<int>(static_cast<unsigned int>(nt) - take);
    sm.after[tid] = static_cast<int>(released - static_cast<unsigned int>(rt >> 32));
  }
  if (tid == 0) sm.start[B] = tokens;
  __syncthreads();

  // Entry i of the free stack with the returned blocks on it.
  auto stack = [&](int64_t i) -> int {
    if (i < count) return P.free_blocks[i];
    // the request whose returned blocks hold place r (after[] falls with b)
    const int r = static_cast<int>(i - count);
    int lo = 0, hi = B - 1;  // the first b with after[b] <= r
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (sm.after[mid] <= r)
        hi = mid;
      else
        lo = mid + 1;
    }
    const int j = sm.held[lo] - 1 - (r - sm.after[lo]);
    return P.block_table[static_cast<int64_t>(sm.slot[lo]) * M + j];
  };

  if (first) {
    for (int b = tid; b <= B; b += blockDim.x) P.query_start[b] = sm.start[b];
    if (tid < B) P.seq_lens[tid] = ok ? static_cast<int>(cached + fresh) : 0;
  }
  // ---- tokens ------------------------------------------------------------------
  for (int t = blockIdx.x * blockDim.x + tid; t < T; t += gridDim.x * blockDim.x) {
    int64_t pos = -1, at = -1;
    if (t < tokens) {
      int lo = 0, hi = B - 1;  // the last b with start[b] <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (sm.start[mid] <= t)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int p = sm.cached[lo] + (t - sm.start[lo]);
      const int j = p >> sh;
      const int h = sm.held[lo];
      const int id = j < h ? P.block_table[static_cast<int64_t>(sm.slot[lo]) * M + j]
                           : stack(top - 1 - (sm.take0[lo] + (j - h)));
      pos = p;
      at = (static_cast<int64_t>(id) << sh) + (p & ((1 << sh) - 1));
    }
    P.positions[t] = pos;
    P.slot_map[t] = at;
  }
  // ---- blocks: new table entries, returned blocks onto the stack ----------------
  for (int b = blockIdx.x * nw + warp; b < B; b += gridDim.x * nw) {
    if (sm.slot[b] < 0) continue;
    int32_t* row = P.block_table + static_cast<int64_t>(sm.slot[b]) * M;
    const int h = sm.held[b], nd = sm.need[b];
    for (int j = h + lane; j < nd; j += 32) row[j] = stack(top - 1 - (sm.take0[b] + (j - h)));
    for (int j = nd + lane; j < h; j += 32) {
      const int64_t at = static_cast<int64_t>(count) + sm.after[b] + (h - 1 - j);
      if (at < N) P.free_blocks[at] = row[j];
    }
  }
  if (B == 0) return;

  // ---- what other CTAs read, by the CTA that finishes last -----------------------
  __syncthreads();
  if (gridDim.x > 1) {
    if (tid == 0) {
      __threadfence();
      const unsigned int done = atomicAdd(reinterpret_cast<unsigned int*>(P.pool) + 1, 1u);
      sm.last = done == gridDim.x - 1;
      __threadfence();
    }
    __syncthreads();
    if (!sm.last) return;
  }
  if (tid < B && ok) {
    P.held_blocks[slot] = static_cast<int>(need);
    if (P.num_accepted) P.cached_lens[slot] = static_cast<int>(cached);
  }
  if (released != 0u) {
    for (int b = warp; b < B; b += nw) {
      if (sm.slot[b] < 0) continue;
      int32_t* row = P.block_table + static_cast<int64_t>(sm.slot[b]) * M;
      for (int j = sm.need[b] + lane; j < sm.held[b]; j += 32) row[j] = -1;
    }
  }
  if (tid == 0) {
    const int64_t left = top - taken;
    P.pool[0] = static_cast<int>(left > N ? N : left);
    P.pool[1] = 0;
  }
}

}  // namespace

cudaError_t launch_paged_tables(const PagedTablesParams& p, cudaStream_t stream) {
  const int threads = p.B <= 256 ? 256 : (p.B + 31) / 32 * 32;
  int ctas = (p.T + kTokensPerCta - 1) / kTokensPerCta;
  if (ctas < 1) ctas = 1;
  if (ctas > 304) ctas = 304;
  // (may be set up while the kernel before it ends, and waits for it)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.shares ? paged_tables_kernel<true> : paged_tables_kernel<false>,
                            p);
}

}  // namespace dspark
