// paged_blocks.cu -- the upkeep of the paged cache: slots forked and freed, the
// blocks compacted, and blocks copied in all layers.
//
// The table calls are prefix sums over the call's slots and then independent work
// per block of them, as for the step's tables (paged_tables.cu), with two
// differences. A block that several rows hold is counted (`shares`: the rows beyond
// the first), and whether a block comes free is only known once every row of the call
// has given it up; and compaction renumbers all blocks. Both are a few phases over
// the same data with a barrier between them: one launch of one cluster of CTAs (a
// single CTA where there is little to do), whose barrier is the hardware's. A fork has
// no such phases, only lengths and pool that are written once every CTA has read them;
// it uses the same cluster, and so eight SMs.
//
// Which row puts a shared block on the stack must not depend on timing: after all
// rows of the call have taken their share off the count, each of a block that came
// out below zero lowers it further to -2 - (its place in the call); the lowest, the
// last request, wins and pushes the block.
//
// Copies are bound by memory: a thread has eight 16-byte pieces on their way (2.8 GB
// read and written: 413 us, 6.8 TB/s, what the plain copy of a large tensor makes; with
// four 440). The table calls are bound by latency, long ones by the eight SMs of the
// cluster (cold caches: 128 forks of 44 thousand entries 14 us, freeing them 30; fork,
// copy and free with a cluster of four 1.4 times as long, on one SM 3.4 times): a fork or
// free of a few requests takes 4 to 8 us, a compaction of 27 thousand blocks 20.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "block_scan.cuh"
#include "common.cuh"
#include "paged.h"

namespace dspark {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxN = DSPARK_MAX_PAGED_BATCH;
constexpr int kCluster = 8;
// Up to this many table entries a single CTA does them all: a cluster's barriers cost
// more than its threads gain.
constexpr int kFewEntries = 4096;
static_assert(kMaxN <= kThreads, "a slot per thread");
// Entries a thread has under way at a time: each is a load or two and perhaps an atomic.
constexpr int kAbreast = 4;

// The last b < n with start[b] <= e.
__device__ __forceinline__ int find(const int* start, int n, int e) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= e)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The entries of a warp, a run of all the call's: which slot each is of. Lanes' entries
// go up, so the slot is found by bisection once and then looked for from the last one's
// (a bisection an entry took half as long again: 128 slots of 344 blocks).
struct Run {
  const int* start;  // [n + 1] first entries of the slots, then their number
  int n, w0, w1;
  int slot0;         // of w0
  __device__ __forceinline__ Run(const int* start_, int n_, int entries, int rank, int size)
      : start(start_), n(n_) {
    const int warp = threadIdx.x >> 5;
    const int each = (entries + size - 1) / size, per = ((each + kWarps - 1) / kWarps + 31) & ~31;
    w0 = min(rank * each + min(warp * per, each), entries);
    w1 = min(rank * each + min((warp + 1) * per, each), entries);
    slot0 = w0 < w1 ? find(start, n, w0) : 0;
  }
  __device__ __forceinline__ int slot(int from, int e) const {
    while (start[from + 1] <= e) ++from;
    return from;
  }
};

// For each i < n whether `clash(i, j)` for some j < n, by the block's warps; into bad[].
template <typename Clash>
__device__ __forceinline__ void find_clashes(int n, int* bad, Clash clash) {
  for (int i = threadIdx.x >> 5; i < n; i += kWarps) {
    bool any = false;
    for (int j = threadIdx.x & 31; j < n; j += 32) any |= clash(i, j);
    any = __any_sync(0xFFFFFFFFu, any);
    if ((threadIdx.x & 31) == 0) bad[i] = any;
  }
  __syncthreads();
}

// The sum over the cluster's CTAs of `mine`, and of those before this one.
__device__ __forceinline__ int cluster_sum(cg::cluster_group& cl, int* shared, int mine,
                                           int* before) {
  if (threadIdx.x == 0) *shared = mine;
  cl.sync();
  int total = 0, first = 0;
  const int rank = static_cast<int>(cl.block_rank()), size = static_cast<int>(cl.num_blocks());
  for (int c = 0; c < size; ++c) {
    const int v = *cl.map_shared_rank(shared, c);
    if (c < rank) first += v;
    total += v;
  }
  cl.sync();  // read by all
  *before = first;
  return total;
}

__device__ __forceinline__ int pool_count(const int32_t* pool, int N, bool tell, int32_t* status) {
  const int count = pool[0];
  if (count >= 0 && count <= N) return count;
  if (tell) report(status, DSPARK_ERR_BOUNDS);
  return count < 0 ? 0 : N;
}

struct ForkSmem {
  unsigned long long warp[33];
  int src[kMaxN], dst[kMaxN];
  int bad[kMaxN];
  int start[kMaxN + 1];  // first entry of each fork, their number
  int keep[kMaxN];       // shared blocks
  int take0[kMaxN];      // blocks taken by the forks before
};

__global__ void __launch_bounds__(kThreads, 1) paged_fork_kernel(PagedForkParams P) {
  __shared__ ForkSmem sm;
  cg::cluster_group cl = cg::this_cluster();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, rank = static_cast<int>(cl.block_rank());
  const int size = static_cast<int>(cl.num_blocks());
  const bool first = rank == 0;  // reports errors
  const int M = P.M, N = P.N, sh = P.page_shift;
  const int count = pool_count(P.pool, N, first && tid == 0, P.status);

  int src = -1, dst = -1;
  if (tid < P.n) {
    src = P.src[tid];
    dst = P.dst[tid];
    if (src < 0 || dst < 0) src = dst = -1;
    sm.src[tid] = src;
    sm.dst[tid] = dst;
  }
  __syncthreads();
  // a dst that is named before, or is a src
  find_clashes(P.n, sm.bad, [&](int i, int j) {
    return sm.src[i] >= 0 && (sm.dst[j] == sm.src[i] || (j < i && sm.dst[j] == sm.dst[i]));
  });
  bool ok = false;
  int len = 0, need = 0, keep = 0;
  if (src >= 0) {
    bool bad = src >= P.S || dst >= P.S || sm.bad[tid];
    if (!bad) {
      len = P.cached_lens[src];
      const int held = P.held_blocks[src];
      need = static_cast<int>((static_cast<int64_t>(len) + (1 << sh) - 1) >> sh);
      bad = len < 0 || held > M || need > held || P.held_blocks[dst] != 0;
    }
    ok = !bad;
    if (bad && first) report(P.status, DSPARK_ERR_BOUNDS);
    if (!ok) need = 0;
    keep = P.shares ? (ok ? len >> sh : 0) : 0;
  }
  unsigned long long total;
  int take = need - keep;
  const unsigned long long taken = block_scan(static_cast<unsigned int>(take), sm.warp, &total);
  if (ok && take > 0) {
    if (taken > static_cast<unsigned long long>(count)) {
      ok = false;
      if (first) report(P.status, DSPARK_ERR_CACHE_FULL);
    } else if (taken > static_cast<unsigned long long>(P.C)) {
      ok = false;
      if (first) report(P.status, DSPARK_ERR_BOUNDS);
    }
  }
  if (!ok) need = take = 0;
  const unsigned long long ends = block_scan(
      (static_cast<unsigned long long>(need) << 32) | static_cast<unsigned int>(take), sm.warp,
      &total);
  const int entries = static_cast<int>(total >> 32), all = static_cast<int>(total);
  if (tid < P.n) {
    sm.start[tid] = static_cast<int>(ends >> 32) - need;
    sm.keep[tid] = keep;
    sm.take0[tid] = static_cast<int>(static_cast<unsigned int>(ends)) - take;
  }
  if (tid == 0) sm.start[P.n] = entries;
  __syncthreads();
  const Run run(sm.start, P.n, entries, rank, size);
  int i = run.slot0;
  for (int e0 = run.w0 + (tid & 31); e0 < run.w1; e0 += 32 * kAbreast) {
    int id[kAbreast], fresh[kAbreast], at[kAbreast];  // at: the copy's place, < 0 if shared
    int64_t to[kAbreast];
#pragma unroll
    for (int u = 0; u < kAbreast; ++u) {
      const int e = e0 + 32 * u;
      if (e >= run.w1) break;
      i = run.slot(i, e);
      const int j = e - sm.start[i], k = j - sm.keep[i];
      id[u] = P.block_table[static_cast<int64_t>(sm.src[i]) * M + j];
      to[u] = static_cast<int64_t>(sm.dst[i]) * M + j;
      at[u] = k < 0 ? -1 : sm.take0[i] + k;
      fresh[u] = k < 0 ? 0 : P.free_blocks[count - 1 - at[u]];
    }
#pragma unroll
    for (int u = 0; u < kAbreast; ++u) {
      if (e0 + 32 * u >= run.w1) break;
      const bool there = id[u] >= 0 && id[u] < N;
      if (!there) report(P.status, DSPARK_ERR_BOUNDS);
      if (at[u] < 0) {
        if (there) atomicAdd(P.shares + id[u], 1);
      } else {
        P.copies[at[u]] = make_int2(id[u], fresh[u]);
        id[u] = fresh[u];
      }
      P.block_table[to[u]] = id[u];
    }
  }
  cl.sync();  // every CTA has read the lengths and the pool
  if (!first) return;
  if (ok) {
    P.held_blocks[dst] = need;
    P.cached_lens[dst] = len;
  }
  if (tid == 0) {
    P.pool[0] = count - all;
    *P.count = all;
  }
}

struct FreeSmem {
  unsigned long long warp[33];
  int slot[kMaxN];
  int bad[kMaxN];
  int start[kMaxN + 1];
  int sums[kWarps];
  int shared;
};

__global__ void __launch_bounds__(kThreads, 1) paged_free_kernel(PagedFreeParams P) {
  __shared__ FreeSmem sm;
  cg::cluster_group cl = cg::this_cluster();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cl.block_rank()), size = static_cast<int>(cl.num_blocks());
  const bool first = rank == 0;
  const int M = P.M, N = P.N;
  const int count = pool_count(P.pool, N, first && tid == 0, P.status);
  int slot = -1, held = 0;
  if (tid < P.n) sm.slot[tid] = slot = P.slots[tid];
  __syncthreads();
  find_clashes(P.n, sm.bad, [&](int i, int j) { return j < i && sm.slot[j] == sm.slot[i]; });
  if (slot >= 0) {
    bool bad = slot >= P.S || sm.bad[tid];
    if (!bad) {
      held = P.held_blocks[slot];
      bad = held < 0 || held > M;
    }
    if (bad) {
      if (first) report(P.status, DSPARK_ERR_BOUNDS);
      slot = -1;
      held = 0;
    }
  }
  unsigned long long total;
  const unsigned long long ends = block_scan(static_cast<unsigned int>(held), sm.warp, &total);
  if (tid < P.n) sm.start[tid] = static_cast<int>(ends) - held;
  const int entries = static_cast<int>(total);
  if (tid == 0) sm.start[P.n] = entries;
  __syncthreads();

  const Run run(sm.start, P.n, entries, rank, size);
  const int w0 = run.w0, w1 = run.w1;
  // Block and slot (place in the call) of kAbreast entries; -1 past the end.
  int id[kAbreast], of[kAbreast];
  int32_t* at[kAbreast];
  int i = run.slot0;
  auto entries_of = [&](int e0) {
    if (e0 < w0 + 32) i = run.slot0;  // a new pass
#pragma unroll
    for (int u = 0; u < kAbreast; ++u) {
      const int e = e0 + 32 * u;
      id[u] = -1;
      at[u] = nullptr;
      of[u] = 0;
      if (e >= w1) continue;
      of[u] = i = run.slot(i, e);
      at[u] = P.block_table + static_cast<int64_t>(sm.slot[i]) * M + (e - sm.start[i]);
      id[u] = *at[u];
      if (id[u] < 0 || id[u] >= N) id[u] = -2;
    }
  };
  constexpr int kStep = 32 * kAbreast;
  if (P.shares) {
    for (int e = w0 + lane; e < w1; e += kStep) {
      entries_of(e);
#pragma unroll
      for (int u = 0; u < kAbreast; ++u)
        if (id[u] >= 0) atomicSub(P.shares + id[u], 1);
    }
    cl.sync();
    for (int e = w0 + lane; e < w1; e += kStep) {
      entries_of(e);
      int left[kAbreast];
#pragma unroll
      for (int u = 0; u < kAbreast; ++u) left[u] = id[u] >= 0 ? __ldcg(P.shares + id[u]) : 0;
#pragma unroll
      for (int u = 0; u < kAbreast; ++u)
        if (left[u] < 0) atomicMin(P.shares + id[u], -2 - of[u]);
    }
    cl.sync();
  }
  // Whether each puts its block on the stack.
  auto pushes = [&](bool (&push)[kAbreast]) {
    int who[kAbreast];
#pragma unroll
    for (int u = 0; u < kAbreast; ++u)
      who[u] = P.shares && id[u] >= 0 ? __ldcg(P.shares + id[u]) : -2 - of[u];
#pragma unroll
    for (int u = 0; u < kAbreast; ++u) push[u] = id[u] >= 0 && who[u] == -2 - of[u];
  };
  int mine = 0;  // of this warp
  for (int e0 = w0; e0 < w1; e0 += kStep) {
    bool push[kAbreast];
    entries_of(e0 + lane);
    pushes(push);
#pragma unroll
    for (int u = 0; u < kAbreast; ++u) {
      if (id[u] == -2) report(P.status, DSPARK_ERR_BOUNDS);
      mine += __popc(__ballot_sync(0xFFFFFFFFu, push[u]));
    }
  }
  if (lane == 0) sm.sums[warp] = mine;
  __syncthreads();
  int ahead = 0, all = 0;  // of the warps before, of the CTA
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) ahead += sm.sums[w];
    all += sm.sums[w];
  }
  int before;
  const int pushed = cluster_sum(cl, &sm.shared, all, &before);
  int r = before + ahead;
  for (int e0 = w0; e0 < w1; e0 += kStep) {
    bool push[kAbreast];
    entries_of(e0 + lane);
    pushes(push);
#pragma unroll
    for (int u = 0; u < kAbreast; ++u) {
      if (at[u]) *at[u] = -1;
      const unsigned int who = __ballot_sync(0xFFFFFFFFu, push[u]);
      if (push[u]) {
        const int64_t place = static_cast<int64_t>(count) + pushed - 1 -
                              (r + __popc(who & ((1u << lane) - 1u)));
        if (place < N) P.free_blocks[place] = id[u];
        if (P.shares) P.shares[id[u]] = 0;
      }
      r += __popc(who);
    }
  }
  if (!first) return;
  if (slot >= 0) {  // (the lengths were read before the cluster's last barrier)
    P.held_blocks[slot] = 0;
    P.cached_lens[slot] = 0;
  }
  if (tid == 0) {
    const int64_t left = static_cast<int64_t>(count) + pushed;
    if (left > N) report(P.status, DSPARK_ERR_BOUNDS);
    P.pool[0] = static_cast<int>(left > N ? N : left);
  }
}

// With U blocks held, the held ones from U on ("movers") go to the free ones below
// ("holes"), of which there are as many, in ascending order.
__global__ void __launch_bounds__(kThreads, 1) paged_compact_kernel(PagedCompactParams P) {
  __shared__ int sums[2][kWarps];
  __shared__ int shared[2];
  cg::cluster_group cl = cg::this_cluster();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cl.block_rank()), size = static_cast<int>(cl.num_blocks());
  const bool first = rank == 0;
  const int M = P.M, N = P.N, all = size * kThreads, me = rank * kThreads + tid;
  const int count = pool_count(P.pool, N, first && tid == 0, P.status);

  // moved[id]: -1 for a free block, 0 for a held one, 1 + its new number for a mover
  for (int i = me; i < N; i += all) P.moved[i] = 0;
  cl.sync();
  int found = 0;
  for (int i = me; i < count; i += all) {
    const int id = P.free_blocks[i];
    if (id >= 0 && id < N)
      found += atomicExch(P.moved + id, -1) == 0;
    else
      report(P.status, DSPARK_ERR_BOUNDS);
  }
  found = __reduce_add_sync(0xFFFFFFFFu, found);
  if (lane == 0) sums[0][warp] = found;
  __syncthreads();
  found = 0;
  for (int w = 0; w < kWarps; ++w) found += sums[0][w];
  int unused;
  const int U = N - cluster_sum(cl, &shared[0], found, &unused);

  // ranks of holes and movers: each warp a run of blocks
  const int64_t each = (static_cast<int64_t>(N) + size - 1) / size;
  const int64_t per = ((each + kWarps - 1) / kWarps + 31) & ~int64_t(31);
  const int w0 = static_cast<int>(min(rank * each + warp * per, static_cast<int64_t>(N)));
  const int w1 = static_cast<int>(
      min(rank * each + min((warp + 1) * per, each), static_cast<int64_t>(N)));
  constexpr int kStep = 32 * kAbreast;
  // The holes and movers among kAbreast times 32 blocks, as masks of lanes.
  unsigned int is_hole[kAbreast], is_mover[kAbreast];
  auto sort = [&](int i0) {
    int v[kAbreast];
#pragma unroll
    for (int u = 0; u < kAbreast; ++u)
      v[u] = i0 + 32 * u + lane < w1 ? __ldcg(P.moved + i0 + 32 * u + lane) : 0;
#pragma unroll
    for (int u = 0; u < kAbreast; ++u) {
      const int i = i0 + 32 * u + lane;
      is_hole[u] = __ballot_sync(0xFFFFFFFFu, i < w1 && i < U && v[u] != 0);
      is_mover[u] = __ballot_sync(0xFFFFFFFFu, i < w1 && i >= U && v[u] == 0);
    }
  };
  int n_hole = 0, n_mover = 0;
  for (int i0 = w0; i0 < w1; i0 += kStep) {
    sort(i0);
#pragma unroll
    for (int u = 0; u < kAbreast; ++u) {
      n_hole += __popc(is_hole[u]);
      n_mover += __popc(is_mover[u]);
    }
  }
  if (lane == 0) {
    sums[0][warp] = n_hole;
    sums[1][warp] = n_mover;
  }
  __syncthreads();
  int hole = 0, mover = 0, holes = 0, movers = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      hole += sums[0][w];
      mover += sums[1][w];
    }
    holes += sums[0][w];
    movers += sums[1][w];
  }
  int hole0, mover0;
  const int moves = cluster_sum(cl, &shared[0], holes, &hole0);
  cluster_sum(cl, &shared[1], movers, &mover0);
  hole += hole0;
  mover += mover0;
  for (int i0 = w0; i0 < w1; i0 += kStep) {
    sort(i0);
#pragma unroll
    for (int u = 0; u < kAbreast; ++u) {
      const int i = i0 + 32 * u + lane;
      const unsigned int below = (1u << lane) - 1u;
      if (is_hole[u] >> lane & 1u) P.copies[hole + __popc(is_hole[u] & below)].y = i;
      if (is_mover[u] >> lane & 1u) P.copies[mover + __popc(is_mover[u] & below)].x = i;
      hole += __popc(is_hole[u]);
      mover += __popc(is_mover[u]);
    }
  }
  cl.sync();
  for (int i = me; i < moves; i += all) {
    const int from = __ldcg(&P.copies[i].x), to = __ldcg(&P.copies[i].y);
    P.moved[from] = to + 1;
    if (P.shares) {
      P.shares[to] = P.shares[from];
      P.shares[from] = 0;
    }
  }
  cl.sync();
  // The tables, in runs of 32 entries of a row: every warp has as many, its lanes look
  // which of them hold blocks, and then it takes those.
  const int runs = (M + 31) / 32;
  const int64_t items = static_cast<int64_t>(P.S) * runs;
  const int64_t share = (items + size * kWarps - 1) / (size * kWarps);
  const int64_t i_begin = (rank * kWarps + warp) * share, i_end = min(i_begin + share, items);
  for (int64_t base = i_begin; base < i_end; base += 32) {
    int row = 0, run = 0, held = 0;
    if (base + lane < i_end) {
      row = static_cast<int>((base + lane) / runs);
      run = static_cast<int>(base + lane - static_cast<int64_t>(row) * runs);
      held = P.held_blocks[row];
      if (held < 0 || held > M) {
        if (run == 0) report(P.status, DSPARK_ERR_BOUNDS);
        held = held < 0 ? 0 : M;
      }
      held = min(max(held - 32 * run, 0), 32);
    }
    unsigned int todo = __ballot_sync(0xFFFFFFFFu, held > 0);
    while (todo) {
      int32_t* at[kAbreast];
      int id[kAbreast], to[kAbreast];
#pragma unroll
      for (int u = 0; u < kAbreast; ++u) {
        at[u] = nullptr;
        if (todo == 0u) continue;
        const int from = __ffs(todo) - 1;
        todo &= todo - 1;
        const int s = __shfl_sync(0xFFFFFFFFu, row, from), c = __shfl_sync(0xFFFFFFFFu, run, from);
        if (lane < __shfl_sync(0xFFFFFFFFu, held, from)) {
          at[u] = P.block_table + static_cast<int64_t>(s) * M + 32 * c + lane;
          id[u] = *at[u];
        }
      }
#pragma unroll
      for (int u = 0; u < kAbreast; ++u)
        if (at[u]) {
          to[u] = id[u] >= 0 && id[u] < N ? __ldcg(P.moved + id[u]) : -1;
          if (to[u] == 0) to[u] = id[u] + 1;  // held, and stays
        }
#pragma unroll
      for (int u = 0; u < kAbreast; ++u)
        if (at[u]) {
          if (to[u] > 0)
            *at[u] = to[u] - 1;
          else
            report(P.status, DSPARK_ERR_BOUNDS);
        }
    }
  }
  for (int i = me; i < N - U; i += all) P.free_blocks[i] = N - 1 - i;
  if (first && tid == 0) {
    P.pool[0] = N - U;
    *P.count = moves;
  }
}

// ---- copies ------------------------------------------------------------------------
constexpr int kCopyThreads = 256, kCopyEach = 8;  // 16-byte pieces a thread holds
constexpr int kChunk = kCopyThreads * kCopyEach;

// blockIdx.y: keys or values of a layer; blockIdx.x takes chunks in turn, of a large
// block or (kMany) of several small ones: then every piece has a copy of its own to look
// up, which would cost a large block 3%. A chunk of one and of several, two layers: blocks
// of 2 KB (0.98 GB read and written) 761 and 168 us, of 8 KB (1.97 GB) 583 and 300, of 12 KB
// (2.95 GB) 632 and 453, of 16 KB (2.62 GB) 474 and 396; of 32 KB either 384.
template <bool kMany>
__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(PagedCopyParams P) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int which = blockIdx.y & 1;
  uint8_t* base = P.base[blockIdx.y];
  int n = *P.count;
  if (n < 0 || n > P.C) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report(P.status, DSPARK_ERR_BOUNDS);
    n = n < 0 ? 0 : P.C;
  }
  const int chunks = (P.pieces + kChunk - 1) / kChunk;  // of a block
  const int group = kMany ? kChunk / P.pieces : 1;      // blocks of a chunk
  const int step_n = gridDim.x / chunks, step_c = gridDim.x - step_n * chunks;
  int i = blockIdx.x / chunks, c = blockIdx.x - i * chunks;
  for (; static_cast<int64_t>(i) * group < n; i += step_n, c += step_c) {
    if (c >= chunks) {
      c -= chunks;
      if (static_cast<int64_t>(++i) * group >= n) break;
    }
    auto there = [&](int2 m) {
      return m.x >= 0 && m.x < P.num_blocks && m.y >= 0 && m.y < P.num_blocks;
    };
    auto place = [&](int u) -> int64_t {  // of a block's piece
      const int row = u >> P.row_shift;
      return (row >> P.page_shift) * P.head_bytes[which] +
             (row & ((1 << P.page_shift) - 1)) * P.token_bytes[which] +
             ((u & ((1 << P.row_shift) - 1)) << 4);
    };
    uint4 x[kCopyEach];
    if constexpr (kMany) {
      uint8_t* to[kCopyEach];
#pragma unroll
      for (int k = 0; k < kCopyEach; ++k) {
        const int all = k * kCopyThreads + threadIdx.x, b = all / P.pieces, u = all - b * P.pieces;
        to[k] = nullptr;
        if (b >= group || n - i * group <= b) continue;
        const int2 m = P.copies[i * group + b];
        if (there(m)) {
          const int64_t at = place(u);
          x[k] = *reinterpret_cast<const uint4*>(base + m.x * P.block_bytes[which] + at);
          to[k] = base + m.y * P.block_bytes[which] + at;
        } else if (u == 0) {
          report(P.status, DSPARK_ERR_BOUNDS);
        }
      }
#pragma unroll
      for (int k = 0; k < kCopyEach; ++k)
        if (to[k]) *reinterpret_cast<uint4*>(to[k]) = x[k];
    } else {
      const int2 m = P.copies[i];
      if (!there(m)) {
        if (threadIdx.x == 0) report(P.status, DSPARK_ERR_BOUNDS);
        continue;
      }
      const uint8_t* from = base + m.x * P.block_bytes[which];
      uint8_t* to = base + m.y * P.block_bytes[which];
      int64_t at[kCopyEach];
#pragma unroll
      for (int k = 0; k < kCopyEach; ++k) {
        const int u = c * kChunk + k * kCopyThreads + threadIdx.x;
        at[k] = place(u);
        if (u < P.pieces) x[k] = *reinterpret_cast<const uint4*>(from + at[k]);
      }
#pragma unroll
      for (int k = 0; k < kCopyEach; ++k)
        if (c * kChunk + k * kCopyThreads + threadIdx.x < P.pieces)
          *reinterpret_cast<uint4*>(to + at[k]) = x[k];
    }
  }
}

// One cluster of `ctas` CTAs, which may be set up while the kernel before it ends.
template <typename Params>
cudaError_t launch_cluster(void (*kernel)(Params), const Params& p, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_paged_fork(const PagedForkParams& p, cudaStream_t stream) {
  const int64_t entries = static_cast<int64_t>(p.n) * p.M;
  return launch_cluster(paged_fork_kernel, p, entries <= kFewEntries ? 1 : kCluster, stream);
}

cudaError_t launch_paged_free(const PagedFreeParams& p, cudaStream_t stream) {
  const int64_t entries = static_cast<int64_t>(p.n) * p.M;
  return launch_cluster(paged_free_kernel, p, entries <= kFewEntries ? 1 : kCluster, stream);
}

cudaError_t launch_paged_compact(const PagedCompactParams& p, cudaStream_t stream) {
  const int64_t entries = static_cast<int64_t>(p.S) * p.M + p.N;
  return launch_cluster(paged_compact_kernel, p, entries <= kFewEntries ? 1 : kCluster, stream);
}

cudaError_t launch_paged_copy(const PagedCopyParams& p, cudaStream_t stream) {
  // Eight CTAs an SM over all layers, keys and values: four waves of the two that are
  // resident at a time (86 registers a thread), since one wave of them, persistent, took
  // 430 us for 413: the dies' halves are not equally fast, and chunks are dealt beforehand.
  int sms = 0;
  const cudaError_t err = sm_count(&sms);
  if (err != cudaSuccess) return err;
  const int ctas = (sms * 8 + 2 * p.caches - 1) / (2 * p.caches);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 2 * p.caches);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.pieces <= kChunk / 2 ? cudaLaunchKernelEx(&cfg, paged_copy_kernel<true>, p)
                                : cudaLaunchKernelEx(&cfg, paged_copy_kernel<false>, p);
}

}  // namespace dspark
