// paged_api.cu -- the paged-cache calls of include/dspark.h: host-side
// argument checks and launches. No allocation, no host synchronisation, no
// state kept between calls.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dspark.h"
#include "paged.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// Sizes that the calls on the tables' blocks share.
bool blocks_ok(int n, int S, int M, int N) {
  return n >= 0 && n <= DSPARK_MAX_PAGED_BATCH && S >= 1 && M >= 1 && M <= 1 << 20 && N >= 1 &&
         N < 1 << 30;
}

bool half_dtype(int d) { return d == DSPARK_BF16 || d == DSPARK_F16; }

// log2 of a page size the library takes, or -1.
int page_shift_of(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

bool stride_ok(int64_t elements, int elem_bytes) {
  return elements > 0 && elements < int64_t(1) << 38 && elements * elem_bytes % 16 == 0;
}

// The checks both cache calls make of the cache's description. `dtype` is the
// type of the tokens' side.
dspark_status check_cache(const dspark_paged_kv* c, int dtype) {
  if (!c || !c->k || !c->v) return DSPARK_ERR_INVALID_ARG;
  if (!half_dtype(dtype) || (!half_dtype(c->dtype) && c->dtype != DSPARK_E4M3))
    return DSPARK_ERR_INVALID_ARG;
  if (c->num_blocks < 1 || c->num_blocks >= 1 << 30 || c->kv_heads < 1 || c->kv_heads > 1024)
    return DSPARK_ERR_INVALID_ARG;
  if (c->dtype != DSPARK_E4M3 && c->dtype != dtype) return DSPARK_ERR_UNSUPPORTED;
  if (page_shift_of(c->page_size) < 0 || (c->head_dim != 64 && c->head_dim != 128))
    return DSPARK_ERR_UNSUPPORTED;
  const int es = c->dtype == DSPARK_E4M3 ? 1 : 2;
  if (!aligned16(c->k) || !aligned16(c->v)) return DSPARK_ERR_ALIGNMENT;
  if (!stride_ok(c->k_token_stride, es) || !stride_ok(c->v_token_stride, es))
    return DSPARK_ERR_ALIGNMENT;
  if (c->kv_heads > 1 && (!stride_ok(c->k_head_stride, es) || !stride_ok(c->v_head_stride, es)))
    return DSPARK_ERR_ALIGNMENT;
  if (c->num_blocks > 1 && (!stride_ok(c->k_block_stride, es) || !stride_ok(c->v_block_stride, es)))
    return DSPARK_ERR_ALIGNMENT;
  return DSPARK_OK;
}

// Whether T rows of `row` 16-bit values may be written: they do not overlap, and lie where
// they are read from (as there) or apart from it. Rows of the same stride may be
// interleaved with those that are read; of another stride, the ranges do not meet.
bool rows_out_ok(const void* in, const void* out, int64_t in_stride, int64_t out_stride,
                 int64_t row, int T) {
  if (T > 1 && out_stride < row) return false;
  if (in == out) return in_stride == out_stride || T < 2;
  const __int128 a = reinterpret_cast<intptr_t>(in), b = reinterpret_cast<intptr_t>(out);
  const __int128 a_end = a + (static_cast<__int128>(T - 1) * in_stride + row) * 2;
  const __int128 b_end = b + (static_cast<__int128>(T - 1) * out_stride + row) * 2;
  if (a_end <= b || b_end <= a) return true;
  if (in_stride != out_stride || T < 2) return false;
  const int64_t step = in_stride * 2;
  int64_t off = static_cast<int64_t>((b - a) % step);
  if (off < 0) off += step;
  return off >= 2 * row && step - off >= 2 * row;
}

// The checks both rotating calls make of the rotation and the norms.
dspark_status check_rotation(const uint64_t* turns, float factor, int rotary_dim, int interleaved,
                             const void* q_weight, const void* k_weight, float eps, int head_dim) {
  if (interleaved != 0 && interleaved != 1) return DSPARK_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > head_dim || (rotary_dim > 0 && (!turns || !isfinite(factor))))
    return DSPARK_ERR_INVALID_ARG;
  if ((q_weight || k_weight) && !(isfinite(eps) && eps >= 0.f)) return DSPARK_ERR_INVALID_ARG;
  if (rotary_dim % 16 != 0) return DSPARK_ERR_UNSUPPORTED;
  if (!aligned16(q_weight) || !aligned16(k_weight) || (reinterpret_cast<uintptr_t>(turns) & 7u))
    return DSPARK_ERR_ALIGNMENT;
  return DSPARK_OK;
}

// A parameter block with the rotation and the norms.
dspark::QkRopeParams rotation_params(const int64_t* positions, const uint64_t* turns, float factor,
                                     int rotary_dim, int interleaved, const void* q_weight,
                                     const void* k_weight, float eps, int head_dim) {
  dspark::QkRopeParams p = {};
  p.positions = positions;
  p.turns = turns;
  p.weight[0] = q_weight;
  p.weight[1] = k_weight;
  p.factor = factor;
  p.eps = eps;
  p.inv_d = 1.f / static_cast<float>(head_dim);
  p.rotary = rotary_dim;
  p.interleaved = interleaved;
  p.D = head_dim;
  return p;
}

}  // namespace

extern "C" {

dspark_status dspark_paged_tables_shared(
    const int32_t* req_state_idx, const int32_t* new_lens, int32_t* cached_lens,
    const int32_t* num_accepted, int32_t* block_table, int32_t* held_blocks, int32_t* free_blocks,
    int32_t* pool, const int32_t* shares, int32_t* query_start, int32_t* seq_lens,
    int64_t* positions, int64_t* slot_map, int B, int S, int M, int N, int T, int page_size,
    int32_t* status, dspark_stream_t stream) {
  if (B < 0 || B > DSPARK_MAX_PAGED_BATCH || S < 1 || M < 1 || M > 1 << 20 || N < 1 ||
      N >= 1 << 30 || T < 0 || T >= 1 << 30)
    return DSPARK_ERR_INVALID_ARG;
  const int shift = page_shift_of(page_size);
  if (shift < 0) return DSPARK_ERR_UNSUPPORTED;
  if (!query_start || (T > 0 && (!positions || !slot_map))) return DSPARK_ERR_INVALID_ARG;
  if (B > 0 && (!req_state_idx || !new_lens || !cached_lens || !block_table || !held_blocks ||
                !free_blocks || !pool || !seq_lens))
    return DSPARK_ERR_INVALID_ARG;
  dspark::PagedTablesParams p;
  p.rsi = req_state_idx;
  p.new_lens = new_lens;
  p.cached_lens = cached_lens;
  p.num_accepted = num_accepted;
  p.block_table = block_table;
  p.held_blocks = held_blocks;
  p.free_blocks = free_blocks;
  p.pool = pool;
  p.query_start = query_start;
  p.seq_lens = seq_lens;
  p.positions = positions;
  p.slot_map = slot_map;
  p.shares = shares;
  p.B = B;
  p.S = S;
  p.M = M;
  p.N = N;
  p.T = T;
  p.page_shift = shift;
  p.status = status;
  if (dspark::launch_paged_tables(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}

dspark_status dspark_paged_tables(const int32_t* req_state_idx, const int32_t* new_lens,
                                  int32_t* cached_lens, const int32_t* num_accepted,
                                  int32_t* block_table, int32_t* held_blocks,
                                  int32_t* free_blocks, int32_t* pool, int32_t* query_start,
                                  int32_t* seq_lens, int64_t* positions, int64_t* slot_map, int B,
                                  int S, int M, int N, int T, int page_size, int32_t* status,
                                  dspark_stream_t stream) {
  return dspark_paged_tables_shared(req_state_idx, new_lens, cached_lens, num_accepted, block_table,
                                    held_blocks, free_blocks, pool, nullptr, query_start, seq_lens,
                                    positions, slot_map, B, S, M, N, T, page_size, status, stream);
}

dspark_status dspark_paged_fork(const int32_t* src, const int32_t* dst, int32_t* cached_lens,
                                int32_t* block_table, int32_t* held_blocks,
                                const int32_t* free_blocks, int32_t* pool, int32_t* shares,
                                int32_t* copies, int32_t* count, int n, int S, int M, int N,
                                int max_copies, int page_size, int32_t* status,
                                dspark_stream_t stream) {
  if (!blocks_ok(n, S, M, N) || max_copies < 0 || max_copies >= 1 << 30)
    return DSPARK_ERR_INVALID_ARG;
  const int shift = page_shift_of(page_size);
  if (shift < 0) return DSPARK_ERR_UNSUPPORTED;
  if (!count || !pool) return DSPARK_ERR_INVALID_ARG;
  if (n > 0 && (!src || !dst || !cached_lens || !block_table || !held_blocks || !free_blocks ||
                (max_copies > 0 && !copies)))
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned8(copies)) return DSPARK_ERR_ALIGNMENT;
  dspark::PagedForkParams p;
  p.src = src;
  p.dst = dst;
  p.cached_lens = cached_lens;
  p.block_table = block_table;
  p.held_blocks = held_blocks;
  p.free_blocks = free_blocks;
  p.pool = pool;
  p.shares = shares;
  p.copies = reinterpret_cast<int2*>(copies);
  p.count = count;
  p.n = n;
  p.S = S;
  p.M = M;
  p.N = N;
  p.C = max_copies;
  p.page_shift = shift;
  p.status = status;
  if (dspark::launch_paged_fork(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}

dspark_status dspark_paged_free(const int32_t* slots, int32_t* cached_lens, int32_t* block_table,
                                int32_t* held_blocks, int32_t* free_blocks, int32_t* pool,
                                int32_t* shares, int n, int S, int M, int N, int32_t* status,
                                dspark_stream_t stream) {
  if (!blocks_ok(n, S, M, N)) return DSPARK_ERR_INVALID_ARG;
  if (n == 0) return DSPARK_OK;
  if (!slots || !cached_lens || !block_table || !held_blocks || !free_blocks || !pool)
    return DSPARK_ERR_INVALID_ARG;
  dspark::PagedFreeParams p;
  p.slots = slots;
  p.cached_lens = cached_lens;
  p.block_table = block_table;
  p.held_blocks = held_blocks;
  p.free_blocks = free_blocks;
  p.pool = pool;
  p.shares = shares;
  p.n = n;
  p.S = S;
  p.M = M;
  p.N = N;
  p.status = status;
  if (dspark::launch_paged_free(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}

size_t dspark_paged_compact_workspace_bytes(int N) {
  return N < 1 ? 0 : (static_cast<size_t>(N) * 4 + 255) & ~size_t(255);
}

dspark_status dspark_paged_compact(int32_t* block_table, const int32_t* held_blocks,
                                   int32_t* free_blocks, int32_t* pool, int32_t* shares,
                                   int32_t* copies, int32_t* count, int S, int M, int N,
                                   int max_copies, void* workspace, size_t workspace_bytes,
                                   int32_t* status, dspark_stream_t stream) {
  if (!blocks_ok(0, S, M, N) || max_copies < N / 2 || max_copies >= 1 << 30)
    return DSPARK_ERR_INVALID_ARG;
  if (!block_table || !held_blocks || !free_blocks || !pool || !count || (N > 1 && !copies))
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned8(copies)) return DSPARK_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < dspark_paged_compact_workspace_bytes(N) ||
      !aligned16(workspace))
    return DSPARK_ERR_WORKSPACE;
  dspark::PagedCompactParams p;
  p.block_table = block_table;
  p.held_blocks = held_blocks;
  p.free_blocks = free_blocks;
  p.pool = pool;
  p.shares = shares;
  p.copies = reinterpret_cast<int2*>(copies);
  p.count = count;
  p.moved = static_cast<int32_t*>(workspace);
  p.S = S;
  p.M = M;
  p.N = N;
  p.status = status;
  if (dspark::launch_paged_compact(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}

dspark_status dspark_paged_copy(const dspark_paged_kv* caches, int n_caches, const int32_t* copies,
                                const int32_t* count, int max_copies, int32_t* status,
                                dspark_stream_t stream) {
  if (n_caches < 0 || n_caches > 1 << 16 || max_copies < 0 || max_copies >= 1 << 30)
    return DSPARK_ERR_INVALID_ARG;
  if (n_caches > 0 && !caches) return DSPARK_ERR_INVALID_ARG;
  for (int i = 0; i < n_caches; ++i) {
    const dspark_paged_kv& c = caches[i];
    const dspark_status bad = check_cache(&c, c.dtype == DSPARK_E4M3 ? DSPARK_BF16 : c.dtype);
    if (bad != DSPARK_OK) return bad;
    const dspark_paged_kv& o = caches[0];
    if (c.dtype != o.dtype || c.num_blocks != o.num_blocks || c.kv_heads != o.kv_heads ||
        c.page_size != o.page_size || c.head_dim != o.head_dim ||
        c.k_block_stride != o.k_block_stride || c.k_head_stride != o.k_head_stride ||
        c.k_token_stride != o.k_token_stride || c.v_block_stride != o.v_block_stride ||
        c.v_head_stride != o.v_head_stride || c.v_token_stride != o.v_token_stride)
      return DSPARK_ERR_UNSUPPORTED;
  }
  if (n_caches == 0 || max_copies == 0) return DSPARK_OK;
  if (!copies || !count) return DSPARK_ERR_INVALID_ARG;
  if (!aligned8(copies)) return DSPARK_ERR_ALIGNMENT;
  const dspark_paged_kv& o = caches[0];
  const int64_t es = o.dtype == DSPARK_E4M3 ? 1 : 2;
  dspark::PagedCopyParams p;
  p.block_bytes[0] = o.k_block_stride * es;
  p.block_bytes[1] = o.v_block_stride * es;
  p.head_bytes[0] = o.k_head_stride * es;
  p.head_bytes[1] = o.v_head_stride * es;
  p.token_bytes[0] = o.k_token_stride * es;
  p.token_bytes[1] = o.v_token_stride * es;
  p.copies = reinterpret_cast<const int2*>(copies);
  p.count = count;
  p.C = max_copies;
  p.num_blocks = o.num_blocks;
  p.page_shift = page_shift_of(o.page_size);
  p.row_shift = (o.head_dim == 128 ? 3 : 2) + (es == 2 ? 1 : 0);
  p.pieces = (o.kv_heads << p.page_shift) << p.row_shift;
  p.status = status;
  for (int first = 0; first < n_caches; first += dspark::kCopyCaches) {
    p.caches = n_caches - first < dspark::kCopyCaches ? n_caches - first : dspark::kCopyCaches;
    for (int i = 0; i < p.caches; ++i) {
      p.base[2 * i] = static_cast<uint8_t*>(caches[first + i].k);
      p.base[2 * i + 1] = static_cast<uint8_t*>(caches[first + i].v);
    }
    if (dspark::launch_paged_copy(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
      return DSPARK_ERR_CUDA;
  }
  return DSPARK_OK;
}

dspark_status dspark_kv_append(const void* k, const void* v, dspark_dtype dtype, int64_t k_stride,
                               int64_t v_stride, const dspark_paged_kv* cache,
                               const int64_t* slot_map, int T, int32_t* status,
                               dspark_stream_t stream) {
  if (T < 0 || T >= 1 << 30) return DSPARK_ERR_INVALID_ARG;
  const dspark_status bad = check_cache(cache, dtype);
  if (bad != DSPARK_OK || T == 0) return bad;
  if (!k || !v || !slot_map) return DSPARK_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !stride_ok(k_stride, 2) || !stride_ok(v_stride, 2))
    return DSPARK_ERR_ALIGNMENT;
  dspark::KvAppendParams p;
  p.src[0] = k;
  p.src[1] = v;
  p.src_stride[0] = k_stride;
  p.src_stride[1] = v_stride;
  p.dst[0] = cache->k;
  p.dst[1] = cache->v;
  p.block_stride[0] = cache->k_block_stride;
  p.block_stride[1] = cache->v_block_stride;
  p.head_stride[0] = cache->k_head_stride;
  p.head_stride[1] = cache->v_head_stride;
  p.token_stride[0] = cache->k_token_stride;
  p.token_stride[1] = cache->v_token_stride;
  p.scale[0] = cache->k_scale;
  p.scale[1] = cache->v_scale;
  p.slot_map = slot_map;
  p.num_slots = static_cast<int64_t>(cache->num_blocks) * cache->page_size;
  p.dtype = dtype;
  p.cache_dtype = cache->dtype;
  p.T = T;
  p.H = cache->kv_heads;
  p.D = cache->head_dim;
  p.page_shift = page_shift_of(cache->page_size);
  p.status = status;
  if (dspark::launch_kv_append(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}

dspark_status dspark_qk_rope(const void* q, void* q_out, const void* k, void* k_out,
                             dspark_dtype dtype, int64_t q_stride, int64_t q_out_stride,
                             int64_t k_stride, int64_t k_out_stride, const int64_t* positions,
                             const uint64_t* turns, float factor, int rotary_dim, int interleaved,
                             const void* q_weight, const void* k_weight, float eps, int q_heads,
                             int kv_heads, int head_dim, int T, dspark_stream_t stream) {
  if (T < 0 || T >= 1 << 30 || q_heads < 1 || q_heads > 1 << 17 || kv_heads < 0 ||
      kv_heads > 1024 || !half_dtype(dtype))
    return DSPARK_ERR_INVALID_ARG;
  if (head_dim < 16 || head_dim > 256 || head_dim % 16 != 0) return DSPARK_ERR_UNSUPPORTED;
  const dspark_status bad = check_rotation(turns, factor, rotary_dim, interleaved, q_weight,
                                           k_weight, eps, head_dim);
  if (bad != DSPARK_OK || T == 0) return bad;
  const bool keys = kv_heads > 0;
  if (!q || !q_out || !positions || (keys && (!k || !k_out))) return DSPARK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(q_out) || !stride_ok(q_stride, 2) || !stride_ok(q_out_stride, 2))
    return DSPARK_ERR_ALIGNMENT;
  if (keys && (!aligned16(k) || !aligned16(k_out) || !stride_ok(k_stride, 2) ||
               !stride_ok(k_out_stride, 2)))
    return DSPARK_ERR_ALIGNMENT;
  if (!rows_out_ok(q, q_out, q_stride, q_out_stride, int64_t(q_heads) * head_dim, T) ||
      (keys && !rows_out_ok(k, k_out, k_stride, k_out_stride, int64_t(kv_heads) * head_dim, T)))
    return DSPARK_ERR_INVALID_ARG;
  dspark::QkRopeParams p = rotation_params(positions, turns, factor, rotary_dim, interleaved,
                                           q_weight, keys ? k_weight : nullptr, eps, head_dim);
  p.src[0] = q;
  p.src[1] = k;
  p.src_stride[0] = q_stride;
  p.src_stride[1] = k_stride;
  p.dst[0] = q_out;
  p.dst[1] = k_out;
  p.dst_stride[0] = q_out_stride;
  p.dst_stride[1] = k_out_stride;
  p.dtype = dtype;
  p.T = T;
  p.Hq = q_heads;
  p.H = kv_heads;
  if (dspark::launch_qk_rope(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}

dspark_status dspark_qk_rope_append(const void* q, void* q_out, const void* k, const void* v,
                                    dspark_dtype dtype, int64_t q_stride, int64_t q_out_stride,
                                    int64_t k_stride, int64_t v_stride,
                                    const dspark_paged_kv* cache, const int64_t* positions,
                                    const int64_t* slot_map, const uint64_t* turns, float factor,
                                    int rotary_dim, int interleaved, const void* q_weight,
                                    const void* k_weight, float eps, int q_heads, int T,
                                    int32_t* status, dspark_stream_t stream) {
  if (T < 0 || T >= 1 << 30 || q_heads < 1 || q_heads > 1 << 17) return DSPARK_ERR_INVALID_ARG;
  dspark_status bad = check_cache(cache, dtype);
  if (bad == DSPARK_OK)
    bad = check_rotation(turns, factor, rotary_dim, interleaved, q_weight, k_weight, eps,
                         cache->head_dim);
  if (bad != DSPARK_OK || T == 0) return bad;
  if (!q || !q_out || !k || !v || !positions || !slot_map) return DSPARK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v) ||
      !stride_ok(q_stride, 2) || !stride_ok(q_out_stride, 2) || !stride_ok(k_stride, 2) ||
      !stride_ok(v_stride, 2))
    return DSPARK_ERR_ALIGNMENT;
  if (!rows_out_ok(q, q_out, q_stride, q_out_stride, int64_t(q_heads) * cache->head_dim, T))
    return DSPARK_ERR_INVALID_ARG;
  dspark::QkRopeParams p = rotation_params(positions, turns, factor, rotary_dim, interleaved,
                                           q_weight, k_weight, eps, cache->head_dim);
  p.src[0] = q;
  p.src[1] = k;
  p.src[2] = v;
  p.src_stride[0] = q_stride;
  p.src_stride[1] = k_stride;
  p.src_stride[2] = v_stride;
  p.dst[0] = q_out;
  p.dst[1] = cache->k;
  p.dst[2] = cache->v;
  p.dst_stride[0] = q_out_stride;
  p.dst_stride[1] = cache->k_token_stride;
  p.dst_stride[2] = cache->v_token_stride;
  p.block_stride[0] = cache->k_block_stride;
  p.block_stride[1] = cache->v_block_stride;
  p.head_stride[0] = cache->k_head_stride;
  p.head_stride[1] = cache->v_head_stride;
  p.scale[0] = cache->k_scale;
  p.scale[1] = cache->v_scale;
  p.slot_map = slot_map;
  p.num_slots = static_cast<int64_t>(cache->num_blocks) * cache->page_size;
  p.dtype = dtype;
  p.cache_dtype = cache->dtype;
  p.T = T;
  p.Hq = q_heads;
  p.H = cache->kv_heads;
  p.page_shift = page_shift_of(cache->page_size);
  p.status = status;
  if (dspark::launch_qk_rope(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}

size_t dspark_paged_attention_workspace_bytes(int B, int q_heads, int kv_heads, int head_dim) {
  if (B < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return dspark::paged_attention_workspace_bytes(B, q_heads, kv_heads, head_dim);
}

dspark_status dspark_paged_attention(const void* q, dspark_dtype dtype, int64_t q_stride,
                                     const dspark_paged_kv* cache, const int32_t* block_table,
                                     const int32_t* req_state_idx, const int32_t* query_start,
                                     const int32_t* seq_lens, void* out, float* lse, float scale,
                                     int causal, int window, int q_heads, int B, int S, int M,
                                     int T, void* workspace, size_t workspace_bytes,
                                     int32_t* status, dspark_stream_t stream) {
  return dspark_paged_attention_sinks(q, dtype, q_stride, cache, block_table, req_state_idx,
                                      query_start, seq_lens, out, lse, scale, causal, window, 0,
                                      q_heads, B, S, M, T, workspace, workspace_bytes, status,
                                      stream);
}

dspark_status dspark_paged_attention_sinks(
    const void* q, dspark_dtype dtype, int64_t q_stride, const dspark_paged_kv* cache,
    const int32_t* block_table, const int32_t* req_state_idx, const int32_t* query_start,
    const int32_t* seq_lens, void* out, float* lse, float scale, int causal, int window, int sinks,
    int q_heads, int B, int S, int M, int T, void* workspace, size_t workspace_bytes,
    int32_t* status, dspark_stream_t stream) {
  if (B < 0 || B > DSPARK_MAX_PAGED_BATCH || S < 1 || M < 1 || M > 1 << 20 || T < 0 ||
      T >= 1 << 24 || q_heads < 1)
    return DSPARK_ERR_INVALID_ARG;
  if (!isfinite(scale) || (causal != 0 && causal != 1) || window < 0 || sinks < 0)
    return DSPARK_ERR_INVALID_ARG;
  const dspark_status bad = check_cache(cache, dtype);
  if (bad != DSPARK_OK) return bad;
  if (q_heads % cache->kv_heads != 0) return DSPARK_ERR_INVALID_ARG;
  if (q_heads / cache->kv_heads > 128) return DSPARK_ERR_UNSUPPORTED;
  if (B == 0 || T == 0) return DSPARK_OK;
  if (!q || !out || !block_table || !req_state_idx || !query_start || !seq_lens)
    return DSPARK_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !stride_ok(q_stride, 2)) return DSPARK_ERR_ALIGNMENT;
  const size_t need =
      dspark::paged_attention_workspace_bytes(B, q_heads, cache->kv_heads, cache->head_dim);
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return DSPARK_ERR_WORKSPACE;
  dspark::PagedAttentionParams p;
  p.q = q;
  p.q_stride = q_stride;
  p.kv = *cache;
  p.block_table = block_table;
  p.rsi = req_state_idx;
  p.query_start = query_start;
  p.seq_lens = seq_lens;
  p.out = out;
  p.lse = lse;
  p.scale = scale;
  p.causal = causal;
  p.window = window > 1 << 28 ? 0 : window;  // longer than any cache
  p.sinks = p.window == 0 ? 0 : sinks < 1 << 28 ? sinks : 1 << 28;
  p.dtype = dtype;
  p.Hq = q_heads;
  p.B = B;
  p.S = S;
  p.M = M;
  p.T = T;
  p.page_shift = page_shift_of(cache->page_size);
  p.whole = 0;
  p.workspace = workspace;
  p.status = status;
  if (dspark::launch_paged_attention(p, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}

}  // extern "C"
