// Joining attention results over disjoint keys (declared in fp8mla.h): entry.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "fp8mla.h"

namespace fp8mla {

struct MergeArgs {
  const void* const* outs;  // host arrays of `parts` device pointers
  const int64_t* out_tokens;
  const int64_t* out_heads;  // strides in elements
  const float* const* lses;
  int parts;
  void* out;
  int64_t token, head;
  float* lse;
  int n_tokens, heads, dim;
};

fp8mla_status_t merge_entry(const MergeArgs& a, cudaStream_t stream);

}  // namespace fp8mla
