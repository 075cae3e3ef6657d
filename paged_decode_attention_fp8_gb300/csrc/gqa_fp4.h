// Paged GQA decode over a 4-bit cache (declared in fp8mla.h): entry and host-side sizes.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "fp8mla.h"

namespace fp8mla {

struct Fp4DecodeArgs {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const void* k_block_scales;
  const void* v_block_scales;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* seqlens;
  const uint8_t* spec_mask;
  const float* sinks;
  void* workspace;
  size_t workspace_bytes;
  void* out;
  float* lse;
  float softmax_scale;
  int num_blocks, max_blocks, q_len, window, num_splits, bs, h_q, h_kv, head_dim, page_size;
};

fp8mla_status_t fp4_decode_entry(const Fp4DecodeArgs& a, cudaStream_t stream);
size_t fp4_workspace_bytes(int bs, int h_q, int h_kv, int head_dim, int q_len, long long max_seqlen, int window,
                           int num_splits);
uint32_t fp4_read_and_clear_status();

}  // namespace fp8mla
