// Appending rotated K and V to a paged cache, and reading cached rows back (declared in fp8mla.h): entries.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "fp8mla.h"

namespace fp8mla {

struct CacheSide {               // one cache: K or V
  const void* x;                 // bf16 rows
  int64_t token, head;           // strides of x in elements
  void* cache;
  const float* scale;            // [1]: the per-tensor scale (E4M3) or the cache scale (E2M1)
  float* row_scales;             // E4M3, one per row
  void* block_scales;            // E2M1, one E4M3 byte per 16 values
};

struct KvAppendArgs {
  CacheSide side[2];             // K, V (side[1].x null: no V)
  const void* q;                 // bf16 queries to rotate along, or null
  int64_t q_token, q_head;
  void* q_out;                   // contiguous [n_tokens, h_q, head_dim]
  const int32_t* slot_mapping;
  const void* positions;
  int positions_64;
  const float* table;            // null: no rotation
  int64_t n_positions;
  int rot, rot_offset, layout;
  int n_tokens, h_q, h_kv, head_dim, page_size, num_blocks;
  fp8mla_kv_dtype_t kv_dtype;
};

struct CacheReadArgs {
  const void* cache;
  const float* scale;
  const float* row_scales;
  const void* block_scales;
  const int32_t* slots;
  void* out;                     // bf16 [n, h_kv, head_dim]
  int n, h_kv, head_dim, page_size, num_blocks;
  fp8mla_kv_dtype_t kv_dtype;
};

fp8mla_status_t kv_append_entry(const KvAppendArgs& a, cudaStream_t stream);
fp8mla_status_t cache_read_entry(const CacheReadArgs& a, cudaStream_t stream);
uint32_t kv_append_read_and_clear_status();

}  // namespace fp8mla
