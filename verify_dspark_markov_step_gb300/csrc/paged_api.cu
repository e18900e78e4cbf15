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

}  // namespace

extern "C" {

dspark_status dspark_paged_tables(const int32_t* req_state_idx, const int32_t* new_lens,
                                  int32_t* cached_lens, const int32_t* num_accepted,
                                  int32_t* block_table, int32_t* held_blocks,
                                  int32_t* free_blocks, int32_t* pool, int32_t* query_start,
                                  int32_t* seq_lens, int64_t* positions, int64_t* slot_map, int B,
                                  int S, int M, int N, int T, int page_size, int32_t* status,
                                  dspark_stream_t stream) {
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
  if (B < 0 || B > DSPARK_MAX_PAGED_BATCH || S < 1 || M < 1 || M > 1 << 20 || T < 0 ||
      T >= 1 << 24 || q_heads < 1)
    return DSPARK_ERR_INVALID_ARG;
  if (!isfinite(scale) || (causal != 0 && causal != 1) || window < 0)
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
