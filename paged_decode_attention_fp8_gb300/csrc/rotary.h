// Rotary positions (declared in fp8mla.h): entries.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "fp8mla.h"

namespace fp8mla {

struct RotaryArgs {
  const void* x[2];          // q and k (k may be absent: heads[1] = 0)
  void* out[2];
  int64_t x_token[2], x_head[2], out_token[2], out_head[2];  // strides in elements
  int heads[2];
  const void* positions;     // int32 or int64 [n_tokens]
  int positions_64;
  const float* table;        // [n_positions, rot / 2, 2]
  int64_t n_positions;
  int n_tokens, head_dim, rot, rot_offset, layout, inverse;
  fp8mla_dtype_t dtype;
};

fp8mla_status_t rotary_table_entry(const double* inv_freq, int half, int64_t n_positions, double factor, float* table,
                                   cudaStream_t stream);
fp8mla_status_t rotary_apply_entry(const RotaryArgs& a, cudaStream_t stream);
uint32_t rotary_read_and_clear_status();

}  // namespace fp8mla
