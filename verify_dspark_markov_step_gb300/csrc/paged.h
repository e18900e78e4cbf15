// paged.h -- launch interface between the C-ABI layer of the paged cache
// (paged_api.cu) and its kernels. Internal to the library.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "dspark.h"

namespace dspark {

// SMs of the current device.
inline cudaError_t sm_count(int* sms) {
  int dev = 0;
  const cudaError_t err = cudaGetDevice(&dev);
  return err != cudaSuccess ? err
                            : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

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
  const int32_t* shares;  // [N] or null
  int B, S, M, N, T, page_shift;
  int32_t* status;
};
cudaError_t launch_paged_tables(const PagedTablesParams& p, cudaStream_t stream);

// Forking, freeing and compacting the block tables, copying blocks (paged_blocks.cu).
struct PagedForkParams {
  const int32_t* src;
  const int32_t* dst;
  int32_t* cached_lens;
  int32_t* block_table;
  int32_t* held_blocks;
  const int32_t* free_blocks;
  int32_t* pool;
  int32_t* shares;  // or null
  int2* copies;
  int32_t* count;
  int n, S, M, N, C, page_shift;
  int32_t* status;
};
cudaError_t launch_paged_fork(const PagedForkParams& p, cudaStream_t stream);

struct PagedFreeParams {
  const int32_t* slots;
  int32_t* cached_lens;
  int32_t* block_table;
  int32_t* held_blocks;
  int32_t* free_blocks;
  int32_t* pool;
  int32_t* shares;  // or null
  int n, S, M, N;
  int32_t* status;
};
cudaError_t launch_paged_free(const PagedFreeParams& p, cudaStream_t stream);

struct PagedCompactParams {
  int32_t* block_table;
  const int32_t* held_blocks;
  int32_t* free_blocks;
  int32_t* pool;
  int32_t* shares;  // or null
  int2* copies;
  int32_t* count;
  int32_t* moved;   // [N] scratch
  int S, M, N;
  int32_t* status;
};
cudaError_t launch_paged_compact(const PagedCompactParams& p, cudaStream_t stream);

constexpr int kCopyCaches = 64;  // layers of one launch
struct PagedCopyParams {
  uint8_t* base[2 * kCopyCaches];  // keys and values of each layer
  int64_t block_bytes[2], head_bytes[2], token_bytes[2];
  const int2* copies;
  const int32_t* count;
  int C, num_blocks, caches;
  int pieces;                // 16-byte pieces of a block
  int row_shift, page_shift; // pieces of a token's row, tokens of a block (log2)
  int32_t* status;
};
cudaError_t launch_paged_copy(const PagedCopyParams& p, cudaStream_t stream);

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

// Norm and rotation of query and key rows, keys and values into their pages
// (qk_rope.cu).
struct QkRopeParams {
  const void* src[3];       // queries, keys, values
  int64_t src_stride[3];    // elements between tokens
  void* dst[3];             // rows, or (keys and values) the caches
  int64_t dst_stride[3];    // elements between tokens
  int64_t block_stride[2], head_stride[2];
  const float* scale[2];    // [kv_heads] or null
  const int64_t* positions;
  const int64_t* slot_map;  // null: no cache
  int64_t num_slots;
  const uint64_t* turns;    // [rotary / 2]
  const void* weight[2];    // [D] of the rows' type, or null: no norm
  float factor, eps, inv_d;
  int rotary;               // 0: no rotation
  int interleaved, dtype, cache_dtype;
  int T, Hq, H, D, page_shift;
  int32_t* status;
};
cudaError_t launch_qk_rope(const QkRopeParams& p, cudaStream_t stream);

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
  int sinks;  // first tokens seen beside the window (0 without one)
  int dtype;
  int Hq, B, S, M, T, page_shift;
  int whole;  // no unit is split over CTAs (set at launch)
  void* workspace;
  int32_t* status;
};
size_t paged_attention_workspace_bytes(int B, int Hq, int Hkv, int D);
cudaError_t launch_paged_attention(PagedAttentionParams p, cudaStream_t stream);

}  // namespace dspark
