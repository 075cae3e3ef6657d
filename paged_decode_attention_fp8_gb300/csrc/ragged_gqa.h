// Attention of many query rows to paged E4M3 keys (declared in fp8mla.h): cross attention, shared prefixes; entries.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "fp8mla.h"

namespace fp8mla {

struct RaggedCache {
  const void* k;
  const void* v;
  const float* k_scale;  // [1], or [num_blocks, h_kv, page] where scale_rows
  const float* v_scale;
  int scale_rows, num_blocks, page_size;
};

struct CrossArgs {
  const void* q;
  int64_t q_token, q_head;  // strides in elements, like the output's
  RaggedCache cache;
  const int32_t* q_starts;  // [bs + 1], or null: sequence b has token b
  const int32_t* block_table;
  const int32_t* kv_lens;
  int max_blocks;
  float softmax_scale;
  void* workspace;
  size_t workspace_bytes;
  void* out;
  int64_t out_token, out_head;
  float* lse;
  int fill_out, fill_lse;  // rows of no sequence: zeros, -inf
  int n_tokens, bs, h_q, h_kv, head_dim;
};

struct SharedArgs {
  const void* q;
  RaggedCache cache;
  const int32_t* prefix_table;   // [n_prefixes, prefix_blocks]
  const int32_t* prefix_lens;    // [n_prefixes]
  const int32_t* prefix_starts;  // [n_prefixes + 1]: its sequences
  int n_prefixes, prefix_blocks;
  const int32_t* block_table;
  const int32_t* seqlens;
  int max_blocks;
  float softmax_scale;
  int q_len;
  const uint8_t* spec_mask;
  const float* sinks;
  void* workspace;
  size_t workspace_bytes;
  void* out;
  float* lse;
  int bs, h_q, h_kv, head_dim;
};

fp8mla_status_t cross_entry(const CrossArgs& a, cudaStream_t stream);
size_t cross_workspace_bytes(int n_tokens, int bs, int h_q, int h_kv, int head_dim, long long max_keys);
fp8mla_status_t shared_entry(const SharedArgs& a, cudaStream_t stream);
size_t shared_workspace_bytes(int bs, int q_len, int h_q, int h_kv, int head_dim, int n_prefixes,
                              long long max_prefix_keys, long long max_keys);
// Test hook of the bounded waits: CTA 0 of later launches skips its fault_tile-th tile of K (0 = off); wait_limit_ns
// replaces the wait limit (0 = the default, the most).
cudaError_t ragged_set_wait_test(int fault_tile, uint64_t wait_limit_ns);
uint32_t ragged_read_and_clear_status();

}  // namespace fp8mla
