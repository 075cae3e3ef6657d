// Rotary positions: the table of cosines and sines, and the rotation of query
// and key heads by it.
//
// A pair (a, b) of a head at position p turns by the angle p f_i of its
// frequency: (a c - b s, b c + a s), c = factor cos(p f_i), s = factor
// sin(p f_i).  Pair i is dims (i, i + rot / 2) of the rotated part (half
// layout) or (2i, 2i + 1) (interleaved); the part is `rot` dims from
// rot_offset, the rest of the head is copied.  The inverse turns by -p f_i:
// the transpose of the rotation, so also its gradient.
//
// The table is float32, its angles and functions are computed in 64 bits: at
// position 10^6 a float32 angle is off by 0.03.  A rotation is two products
// and a sum, each rounded to float32 (no fused multiply-add, so that the
// append kernel, which quantises the result, takes the same decisions), and
// one rounding to the head's type.
//
// HBM-bound: every head is read and written once (4 bytes a bf16 value).  A
// thread keeps one piece of the rotated part (8 pairs, 32 bytes of values
// for 64 of table) and its cosines and sines, and goes over heads with it, up
// to four heads' loads in flight.  Those loads go out first, the position and
// the table's row behind them: the other way round two memory latencies stood
// before every load.  8191 tokens x 40 heads x 128 in bf16: 32.1 us, 5.36 TB/s,
// 0.79 of the measured copy bandwidth (45.6 us with the position first); 65536
// tokens 0.88; float32 58.7 us, 0.85.  At three CTAs of 80 registers the half
// layout's three instances spill 12 to 14 bytes; more registers a thread were
// slower (see Shape).  Sizes, strides or addresses that are no multiples of 8
// values go a pair at a time: head_dim 126 63 us, 0.39.
//
// The table is made once: a 64-bit cosine and sine per entry bound it (131072
// positions of 64 pairs 466 us, the bytes alone 10).
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "host_util.h"
#include "rotary.h"

namespace fp8mla {
namespace {

__device__ uint32_t g_status_rot;

constexpr int kThreads = 256;
// Heads whose values a thread has in flight, and CTAs of an SM (bf16, heads x CTAs: 4 x 3 32.3 us, 2 x 4 33.8, 3 x 3
// 35.3, 4 x 2 40.1; float32: 2 x 3 58.7, 1 x 4 61.1, 4 x 2 62.5, 2 x 4 66.5, 4 x 3 85.4, spilled).
template <typename T>
struct Shape {
  static constexpr int kHeads = sizeof(T) == 4 ? 2 : 4;
  static constexpr int kCtas = 3;
};

__global__ void __launch_bounds__(256) rotary_table_kernel(const double* __restrict__ inv_freq, int half,
                                                           int64_t total, double factor, float2* __restrict__ table) {
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t p = i / half;
    double s, c;
    sincos(static_cast<double>(p) * __ldg(inv_freq + (i - p * half)), &s, &c);
    table[i] = make_float2(static_cast<float>(c * factor), static_cast<float>(s * factor));
  }
}

// kV consecutive values of T <-> float
template <typename T, int kV>
struct Vec {
  static_assert(kV == 1 || kV == 8, "");
  alignas(kV == 1 ? sizeof(T) : 16) T v[kV];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kV == 1) {
      v[0] = *p;
    } else {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        reinterpret_cast<uint4*>(v)[i] = *(reinterpret_cast<const uint4*>(p) + i);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kV == 1) {
      *p = v[0];
    } else {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
        *(reinterpret_cast<uint4*>(p) + i) = reinterpret_cast<const uint4*>(v)[i];
    }
  }
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f(float x, __half& y) { y = __float2half_rn(x); }

struct Params {
  const void* x[2];
  void* out[2];
  int64_t x_token[2], x_head[2], out_token[2], out_head[2];
  int heads[2];
  const void* positions;
  const float2* table;
  int64_t n_positions;
  int n_tokens, rot, rot_offset, inverse, positions_64, head_dim;
  int zero;         // bit w: out[w]'s rows of tokens without a position become zeros
  int units;        // pieces of a head: rotated ones, then (unless in place) copied ones
  int rot_units;
  int unit_lanes, head_lanes, token_lanes;  // a thread's piece, head and token within its block
};

// Zeros for the rows of this thread's token, which has no position: its share of the dims of its heads.  (A call of its
// own, so that the kernel's registers do not know of it.)
template <typename T, int kV>
__device__ __noinline__ void zero_rows(const Params& prm) {
  const int ul = threadIdx.x % prm.unit_lanes;
  const int hl = threadIdx.x / prm.unit_lanes % prm.head_lanes;
  const int64_t token =
      static_cast<int64_t>(blockIdx.x) * prm.token_lanes + threadIdx.x / (prm.unit_lanes * prm.head_lanes);
  const Vec<T, kV> none = {};
  for (int w = 0; w < 2; ++w) {
    if (!((prm.zero >> w) & 1)) continue;
    for (int h = hl; h < prm.heads[w]; h += prm.head_lanes)
      for (int d = ul * kV; d < prm.head_dim; d += prm.unit_lanes * kV)
        none.store(static_cast<T*>(prm.out[w]) + token * prm.out_token[w] + h * prm.out_head[w] + d);
  }
}

// kV: pairs of a piece (8, or 1 where the sizes, strides or addresses do not allow 16-byte accesses); a copied
// piece is kV values.
template <typename T, int kV, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, Shape<T>::kCtas) rotary_kernel(const __grid_constant__ Params prm) {
  constexpr int kHeadsInFlight = Shape<T>::kHeads;
  griddep_wait();
  const int ul = threadIdx.x % prm.unit_lanes;
  const int hl = threadIdx.x / prm.unit_lanes % prm.head_lanes;
  const int tl = threadIdx.x / (prm.unit_lanes * prm.head_lanes);
  const int64_t token = static_cast<int64_t>(blockIdx.x) * prm.token_lanes + tl;
  if (tl >= prm.token_lanes || token >= prm.n_tokens) return;
  const int heads = prm.heads[0] + prm.heads[1];
  auto head_in = [&](int h) {
    const int w = h >= prm.heads[0];
    return static_cast<const T*>(prm.x[w]) + token * prm.x_token[w] + (h - (w ? prm.heads[0] : 0)) * prm.x_head[w];
  };
  auto head_out = [&](int h) {
    const int w = h >= prm.heads[0];
    return static_cast<T*>(prm.out[w]) + token * prm.out_token[w] + (h - (w ? prm.heads[0] : 0)) * prm.out_head[w];
  };
  int64_t pos = -1;
  bool known = false;
  auto skipped = [&]() {  // asked after the first heads' loads have gone out: whether the token has no position
    if (!known) {
      pos = prm.positions_64 ? __ldg(static_cast<const long long*>(prm.positions) + token)
                             : __ldg(static_cast<const int32_t*>(prm.positions) + token);
      known = true;
      if (pos >= prm.n_positions) {
        if (ul == 0 && hl == 0) atomicOr(&g_status_rot, FP8MLA_DEV_BAD_POSITION);
        pos = -1;
      }
    }
    return pos < 0;  // padding, or past the table
  };
  for (int u = ul; u < prm.units; u += prm.unit_lanes) {
    if (u < prm.rot_units) {
      // first value of each half of the piece; kV pairs
      const int d0 = prm.rot_offset + (kInterleaved ? 2 * kV * u : kV * u);
      const int d1 = kInterleaved ? d0 + kV : d0 + prm.rot / 2;
      float2 cs[kV];
      for (int h0 = hl; h0 < heads; h0 += prm.head_lanes * kHeadsInFlight) {
        Vec<T, kV> a[kHeadsInFlight], b[kHeadsInFlight];
#pragma unroll
        for (int k = 0; k < kHeadsInFlight; ++k) {
          const int h = h0 + k * prm.head_lanes;
          if (h < heads) {
            const T* p = head_in(h);
            a[k].load(p + d0);
            b[k].load(p + d1);
          }
        }
        if (skipped()) {
          if (prm.zero != 0) zero_rows<T, kV>(prm);
          return;
        }
        if (h0 == hl) {
          const float2* row = prm.table + pos * (prm.rot / 2) + kV * u;
          if constexpr (kV == 1) {
            cs[0] = __ldg(row);
          } else {
#pragma unroll
            for (int i = 0; i < kV / 2; ++i) {
              const float4 x = __ldg(reinterpret_cast<const float4*>(row) + i);
              cs[2 * i] = make_float2(x.x, x.y), cs[2 * i + 1] = make_float2(x.z, x.w);
            }
          }
          if (prm.inverse) {
#pragma unroll
            for (int i = 0; i < kV; ++i) cs[i].y = -cs[i].y;
          }
        }
#pragma unroll
        for (int k = 0; k < kHeadsInFlight; ++k) {
          const int h = h0 + k * prm.head_lanes;
          if (h < heads) {
            Vec<T, kV> ra, rb;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
              // pair i of the piece: (a[i], b[i]), or two neighbours of the 2 kV values a, b
              const float x = to_f(kInterleaved ? (2 * i < kV ? a[k].v[2 * i % kV] : b[k].v[2 * i % kV]) : a[k].v[i]);
              const float y = to_f(kInterleaved
                                       ? (2 * i + 1 < kV ? a[k].v[(2 * i + 1) % kV] : b[k].v[(2 * i + 1) % kV])
                                       : b[k].v[i]);
              const float rx = __fsub_rn(__fmul_rn(x, cs[i].x), __fmul_rn(y, cs[i].y));
              const float ry = __fadd_rn(__fmul_rn(y, cs[i].x), __fmul_rn(x, cs[i].y));
              if constexpr (kInterleaved) {
                from_f(rx, 2 * i < kV ? ra.v[2 * i % kV] : rb.v[2 * i % kV]);
                from_f(ry, 2 * i + 1 < kV ? ra.v[(2 * i + 1) % kV] : rb.v[(2 * i + 1) % kV]);
              } else {
                from_f(rx, ra.v[i]);
                from_f(ry, rb.v[i]);
              }
            }
            T* p = head_out(h);
            ra.store(p + d0);
            rb.store(p + d1);
          }
        }
      }
    } else {  // a copied piece, outside the rotated part
      if (skipped()) {
        if (prm.zero != 0) zero_rows<T, kV>(prm);
        return;
      }
      int d = (u - prm.rot_units) * kV;
      if (d >= prm.rot_offset) d += prm.rot;
      for (int h = hl; h < heads; h += prm.head_lanes) {
        Vec<T, kV> a;
        a.load(head_in(h) + d);
        a.store(head_out(h) + d);
      }
    }
  }
}

template <typename T>
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t stream) {
  Params p;
  bool in_place = true, wide = true;
  for (int w = 0; w < 2; ++w) {
    p.x[w] = a.x[w], p.out[w] = a.out[w];
    p.x_token[w] = a.x_token[w], p.x_head[w] = a.x_head[w];
    p.out_token[w] = a.out_token[w], p.out_head[w] = a.out_head[w];
    p.heads[w] = a.heads[w];
    if (a.heads[w] == 0) continue;
    in_place &= a.x[w] == a.out[w] && a.x_token[w] == a.out_token[w] && a.x_head[w] == a.out_head[w];
    wide &= ((reinterpret_cast<uintptr_t>(a.x[w]) | reinterpret_cast<uintptr_t>(a.out[w])) & 15u) == 0 &&
            ((a.x_token[w] | a.x_head[w] | a.out_token[w] | a.out_head[w]) & 7) == 0;
  }
  wide &= a.head_dim % 8 == 0 && a.rot_offset % 8 == 0 && a.rot % 16 == 0 &&
          (reinterpret_cast<uintptr_t>(a.table) & 15u) == 0;
  const int v = wide ? 8 : 1;
  p.positions = a.positions;
  p.positions_64 = a.positions_64;
  p.table = reinterpret_cast<const float2*>(a.table);
  p.n_positions = a.n_positions;
  p.n_tokens = a.n_tokens;
  p.rot = a.rot;
  p.rot_offset = a.rot_offset;
  p.inverse = a.inverse;
  p.head_dim = a.head_dim;
  p.zero = a.layout / FP8MLA_ROTARY_ZERO_Q;
  p.rot_units = a.rot / (2 * v);
  p.units = p.rot_units + (in_place ? 0 : (a.head_dim - a.rot) / v);
  const int heads = a.heads[0] + a.heads[1];
  p.unit_lanes = std::min(p.units, kThreads);
  p.head_lanes = std::min(kThreads / p.unit_lanes, (heads + Shape<T>::kHeads - 1) / Shape<T>::kHeads);
  p.token_lanes = std::min(kThreads / (p.unit_lanes * p.head_lanes), a.n_tokens);
  const int threads = (p.unit_lanes * p.head_lanes * p.token_lanes + 31) / 32 * 32;
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(a.n_tokens) + p.token_lanes - 1) / p.token_lanes);
  const dim3 grid(blocks), block(threads);
  if (wide)
    return a.layout & FP8MLA_ROTARY_INTERLEAVED ? launch_dependent(rotary_kernel<T, 8, true>, grid, block, 0, stream, p)
                         : launch_dependent(rotary_kernel<T, 8, false>, grid, block, 0, stream, p);
  return a.layout & FP8MLA_ROTARY_INTERLEAVED ? launch_dependent(rotary_kernel<T, 1, true>, grid, block, 0, stream, p)
                       : launch_dependent(rotary_kernel<T, 1, false>, grid, block, 0, stream, p);
}

}  // namespace

fp8mla_status_t rotary_table_entry(const double* inv_freq, int half, int64_t n_positions, double factor, float* table,
                                   cudaStream_t stream) {
  if (half < 1 || half > 4096 || n_positions < 0 || n_positions > (1ll << 40) / half || !(factor > 0.0) ||
      factor > 1e30)
    return FP8MLA_ERR_INVALID_ARG;
  if (n_positions == 0) return FP8MLA_OK;
  if (inv_freq == nullptr || table == nullptr || (reinterpret_cast<uintptr_t>(inv_freq) & 7u) ||
      (reinterpret_cast<uintptr_t>(table) & 7u))
    return FP8MLA_ERR_INVALID_ARG;
  const int64_t total = n_positions * half;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((total + 255) / 256, device_sms() * 8));
  rotary_table_kernel<<<blocks, 256, 0, stream>>>(inv_freq, half, total, factor, reinterpret_cast<float2*>(table));
  return cudaGetLastError() == cudaSuccess ? FP8MLA_OK : FP8MLA_ERR_CUDA;
}

fp8mla_status_t rotary_apply_entry(const RotaryArgs& a, cudaStream_t stream) {
  if (a.n_tokens < 0 || a.heads[0] < 1 || a.heads[1] < 0 || a.heads[0] > (1 << 20) || a.heads[1] > (1 << 20) ||
      a.head_dim < 2 || a.head_dim > 8192 || a.rot < 2 || a.rot % 2 != 0 || a.rot_offset < 0 ||
      a.rot > a.head_dim - a.rot_offset || a.n_positions < 1 || a.layout < 0 ||
      a.layout > (FP8MLA_ROTARY_INTERLEAVED | FP8MLA_ROTARY_ZERO_Q | FP8MLA_ROTARY_ZERO_K))
    return FP8MLA_ERR_INVALID_ARG;
  if (a.n_tokens == 0) return FP8MLA_OK;
  if (a.positions == nullptr || a.table == nullptr || misaligned(a.positions, a.positions_64 ? 8 : 4) ||
      misaligned(a.table, 8))
    return FP8MLA_ERR_INVALID_ARG;
  const uintptr_t size = a.dtype == FP8MLA_F32 ? 4 : 2;
  for (int w = 0; w < 2; ++w) {
    if (a.heads[w] == 0) continue;
    if (a.x[w] == nullptr || a.out[w] == nullptr || reinterpret_cast<uintptr_t>(a.x[w]) % size ||
        reinterpret_cast<uintptr_t>(a.out[w]) % size)
      return FP8MLA_ERR_INVALID_ARG;
  }
  if (a.dtype != FP8MLA_BF16 && a.dtype != FP8MLA_F16 && a.dtype != FP8MLA_F32) return FP8MLA_ERR_UNSUPPORTED_DTYPE;
  // an output takes its own input's place or no tensor's: rows are read and written by many threads in any order
  Rows in[2], out[2];
  for (int w = 0; w < 2; ++w) {
    in[w] = rows_of(a.x[w], a.x_token[w], a.x_head[w], a.n_tokens, a.heads[w], a.head_dim, size);
    out[w] = rows_of(a.out[w], a.out_token[w], a.out_head[w], a.n_tokens, a.heads[w], a.head_dim, size);
  }
  if (rows_overlap_themselves(out[0]) || rows_overlap_themselves(out[1]) || rows_overlap(out[0], out[1]) ||
      clobbers(out[0], in[0]) || clobbers(out[1], in[1]) || rows_overlap(out[0], in[1]) || rows_overlap(out[1], in[0]))
    return FP8MLA_ERR_INVALID_ARG;
  cudaError_t e;
  switch (a.dtype) {
    case FP8MLA_BF16: e = launch_rotary<__nv_bfloat16>(a, stream); break;
    case FP8MLA_F16: e = launch_rotary<__half>(a, stream); break;
    default: e = launch_rotary<float>(a, stream); break;
  }
  return e == cudaSuccess ? FP8MLA_OK : FP8MLA_ERR_CUDA;
}

uint32_t rotary_read_and_clear_status() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_status_rot, sizeof(v));
  cudaMemcpyToSymbol(g_status_rot, &z, sizeof(z));
  return v;
}

}  // namespace fp8mla
