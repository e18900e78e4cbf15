// paged.h -- launch interface between the C-ABI layer of the paged cache
// (paged_api.cu) and its kernels. Internal to the library.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dspark.h"

namespace dspark {

// Block tables and slot map of a step (paged_tables.cu).
struct PagedTablesParams {
  const int32_t* rsi;
  const int32_t* new_lens;
  int32_t* cached_lens;
  const int32_t* num_accepted;  // or null
  int32_t* block_table;
  int32_t* held_blocks;
  int32_t* free_blocks;
  int32_t* pool;
  int32_t* query_start;
  int32_t* seq_lens;
  int64_t* positions;
  int64_t* slot_map;
  int B, S, M, N, T, page_shift;
  int32_t* status;
};
cudaError_t launch_paged_tables(const PagedTablesParams& p, cudaStream_t stream);

// Keys and values of new tokens into their pages (kv_append.cu).
struct KvAppendParams {
  const void* src[2];       // k, v
  int64_t src_stride[2];    // elements between tokens
  void* dst[2];
  int64_t block_stride[2], head_stride[2], token_stride[2];
  const float* scale[2];    // [kv_heads] or null
  const int64_t* slot_map;
  int64_t num_slots;        // num_blocks * page_size
  int dtype, cache_dtype;
  int T, H, D, page_shift;
  int32_t* status;
};
cudaError_t launch_kv_append(const KvAppendParams& p, cudaStream_t stream);

// Attention of new tokens over the pages (paged_attention.cu).
struct PagedAttentionParams {
  const void* q;
  int64_t q_stride;
  dspark_paged_kv kv;
  const int32_t* block_table;
  const int32_t* rsi;
  const int32_t* query_start;
  const int32_t* seq_lens;
  void* out;
  float* lse;
  float scale;
  int causal, window;
  int dtype;
  int Hq, B, S, M, T, page_shift;
  int whole;  // no unit is split over CTAs (set at launch)
  void* workspace;
  int32_t* status;
};
size_t paged_attention_workspace_bytes(int B, int Hq, int Hkv, int D);
cudaError_t launch_paged_attention(PagedAttentionParams p, cudaStream_t stream);

}  // namespace dspark
