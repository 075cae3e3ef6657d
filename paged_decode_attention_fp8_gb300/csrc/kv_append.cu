// Appending a step's K and V to a paged cache with the rotary position applied
// on the way, and reading cached rows back as bf16.
//
// Append: K's row (token, head) is rotated (see rotary.cu: two float32
// products and a sum a value), V's is taken as it is; both are quantised from
// float32, without a rounding to bf16 between, and land in the token's slot:
//   E4M3, per-tensor scale: code = E4M3(x * inv), inv = fp32(1 / scale)
//   E4M3, per-row scales:   scale = fp32(amax / 448), inv = fp32(448 / amax)
//                           (1 for a zero row; a row with amax < 2^-64 is
//                           lifted by 2^64 first), as the cache write does
//   E2M1 in blocks of 16:   s8 = E4M3(amax * fp32(1 / fp32(6 scale))),
//                           code = E2M1(x * fp32(1 / fp32(s8 * scale))),
//                           0 where s8 is 0; a NaN, for which E2M1 has no
//                           code, makes s8 and so its block NaN
// Every float operation and conversion rounds to nearest even, conversions
// saturate.  The same launch can rotate the step's queries (bf16 in and out).
//
// HBM-bound: 2 bytes in and 1 (or 9/16) out per value.  A group of L lanes
// owns a row and each lane two 16-byte chunks of it at a time: those of a
// rotated piece are partners (half layout: c and c + rot / 16, so a rotation
// stays in the lane; interleaved: neighbours), the others neighbours.  A block
// of 16 values is a lane's two chunks, or in the half layout the same chunk of
// two neighbouring lanes: one shuffle.  K, V and Q rows are three classes of
// CTAs of one grid, one wave of them, and each warp walks its rows in a
// pipeline: the chain position -> table row -> rotation is longer than a
// memory access, so slots and positions come two steps ahead, values and the
// table's rows (into L1) one.  A 16384-token prompt, 8 KV heads of 128, E4M3:
// 22.0 us, 4.97 TB/s, 0.73 of the measured copy bandwidth (131072 tokens 0.85:
// the rest is ramp); 2049 latent rows of 576 with 16 query heads 13.0 us, 0.90.
// With row scales, whose amax and two divisions stand before a row's codes,
// 25.5 us, 0.64 (131072 tokens 0.74).  Into 4 bits 24.4 us, 0.57, and 0.61 at
// 131072 tokens, so not the ramp but the arithmetic holds it: per 16 values an
// amax, two conversions of a scale, a reciprocal, their exchange between lanes
// and 16 products and conversions.  Reading 65537 rows x 8 heads back takes 34.8
// us, 0.86 (4 bits 32.0, 0.79; 8193 rows 6.2, 0.51: ramp).  8193 tokens into 4
// bits (12.8 us) and both caches read back: 24.9 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "host_util.h"
#include "kv_append.h"

namespace fp8mla {
namespace {

__device__ uint32_t g_status_append;

constexpr int kThreads = 256;
constexpr int kReadCtasPerSm = 5;
// CTAs of an SM: registers for one piece a lane in flight, or for two and three.
template <int kP>
__host__ __device__ constexpr int append_ctas() {
  return kP == 1 ? 4 : (kP == 2 ? 3 : 2);
}
constexpr int kMaxHeadDim = 1024;
constexpr float kTinyAmax = 5.42101086242752217e-20f;  // 2^-64
constexpr float kTinyLift = 1.84467440737095516e19f;   // 2^64

enum Kind { kTensor = 0, kRowScales = 1, kFp4 = 2, kQuery = 3 };

struct Source {
  const uint16_t* x;
  int64_t token, head;
  uint8_t* out;        // cache, or the rotated queries
  const float* scale;
  float* row_scales;
  uint8_t* block_scales;
  FastDiv heads;
  uint32_t rows;       // tokens * heads
};

struct Params {
  Source src[3];       // K, V, Q
  const int32_t* slots;
  const void* positions;
  const float2* table;  // null: no rotation
  int64_t n_positions;
  FastDiv page;
  uint32_t num_slots;
  int positions_64, rot, rot_offset, interleaved, head_dim;
  int zero_q;          // queries of tokens without a position become zeros
  uint32_t first[4];   // CTAs [first[i], first[i + 1]) take class i
};

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
}

template <bool kNan = false>  // kNan: NaN where a value is
__device__ __forceinline__ float amax8(const float (&x)[8]) {
  auto max3 = [](float a, float b, float c) { return kNan ? fmax3_nan(a, b, c) : fmax3(a, b, c); };
  float m = max3(fabsf(x[0]), fabsf(x[1]), fabsf(x[2]));
  m = max3(m, fabsf(x[3]), fabsf(x[4]));
  m = max3(m, fabsf(x[5]), fabsf(x[6]));
  return max3(m, m, fabsf(x[7]));
}

__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(x[i], inv);
  return make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]), pack_e4m3x4(y[4], y[5], y[6], y[7]));
}

// One row's piece of a lane: chunks c0 and c1 (8 values each) as floats.
struct Piece {
  float a[8], b[8];
};

// What a step needs to know of its rows, and their values.
struct Where {
  int32_t slot, pos;  // pos: -1 padding, -2 past the table
};
template <int kP>
struct Values {
  uint4 a[kP], b[kP];
};

// Zeros for a row of queries without a position, by the lanes of its group.  (A call of its own, out of the loop's
// registers: selecting the values instead cost the latent case 0.4 us.)
__device__ __noinline__ void zero_row(uint8_t* row, int head_dim, int sub, int lanes) {
  for (int c = sub; c < head_dim / 8; c += lanes) reinterpret_cast<uint4*>(row)[c] = make_uint4(0, 0, 0, 0);
}

// kL lanes a row, kP pairs of chunks a lane.  A warp's steps are a pipeline: slots and positions two steps ahead,
// values one ahead, and the table's rows asked into L1 one ahead (where every lane has one piece: a prompt's K and V
// 23.4 us, without 25.4; with two pieces, of which a latent row's lanes turn few, it cost 1.4 us of 17.9).
template <int kL, int kP, int kKind>
__device__ __forceinline__ void run_class(const Params& prm, const Source& src, bool rotate, uint32_t cta,
                                          uint32_t ctas) {
  constexpr int kWarpRows = 32 / kL;
  const int lane = threadIdx.x % 32, sub = lane % kL, grp = lane / kL;
  const int pairs = prm.head_dim / 16;
  const int rot_pairs = rotate ? prm.rot / 16 : 0;
  const int off_chunk = prm.rot_offset / 8;
  const bool half = rotate && !prm.interleaved;
  // the lane's chunks and whether they turn; half layout: rotated pairs first, then the rest in order
  int c0[kP], c1[kP];
  bool turn[kP], live[kP];
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    const int p = sub + j * kL;
    live[j] = p < pairs;
    if (half) {
      turn[j] = p < rot_pairs;
      if (turn[j]) {
        c0[j] = off_chunk + p;
        c1[j] = c0[j] + rot_pairs;
      } else {
        c0[j] = 2 * (p - rot_pairs);
        c1[j] = c0[j] + 1;
        if (c0[j] >= off_chunk) c0[j] += 2 * rot_pairs;
        if (c1[j] >= off_chunk) c1[j] += 2 * rot_pairs;
      }
    } else {
      c0[j] = 2 * p;
      c1[j] = c0[j] + 1;
      turn[j] = rotate && c0[j] >= off_chunk && c0[j] < off_chunk + 2 * rot_pairs;
    }
  }
  float tensor_inv = 1.f, scale = 1.f, inv6 = 1.f;
  if constexpr (kKind == kTensor) tensor_inv = __frcp_rn(__ldg(src.scale));
  if constexpr (kKind == kFp4) {
    scale = __ldg(src.scale);
    inv6 = __frcp_rn(__fmul_rn(scale, 6.f));
  }
  // the 8 pairs of a turning piece in the row of a position
  auto table_at = [&](int32_t pos, int j) {
    const int pair0 = half ? 8 * (sub + j * kL) : 4 * (c0[j] - off_chunk);
    return reinterpret_cast<const float4*>(prm.table + static_cast<int64_t>(pos) * (prm.rot / 2) + pair0);
  };

  auto look = [&](uint32_t base, Where& w) {
    const uint32_t row = base + grp;
    w.slot = -1;
    w.pos = -1;
    if (row < src.rows) {
      const uint32_t token = fast_div(row, src.heads);
      w.slot = kKind == kQuery ? 0 : __ldg(prm.slots + token);
      w.pos = 0;
      if (prm.table != nullptr) {
        const int64_t p = prm.positions_64 ? __ldg(static_cast<const long long*>(prm.positions) + token)
                                           : __ldg(static_cast<const int32_t*>(prm.positions) + token);
        w.pos = p < 0 ? -1 : (p < prm.n_positions ? static_cast<int32_t>(p) : -2);
      }
    }
  };
  auto load = [&](uint32_t base, Values<kP>& v) {
    const uint32_t row = base + grp;
#pragma unroll
    for (int j = 0; j < kP; ++j) v.a[j] = v.b[j] = make_uint4(0, 0, 0, 0);
    if (row < src.rows) {
      const uint32_t token = fast_div(row, src.heads), head = row - token * src.heads.d;
      const uint4* x = reinterpret_cast<const uint4*>(src.x + token * src.token + head * src.head);
#pragma unroll
      for (int j = 0; j < kP; ++j)
        if (live[j]) {
          v.a[j] = __ldcs(x + c0[j]);
          v.b[j] = __ldcs(x + c1[j]);
        }
    }
  };
  auto ask = [&](const Where& w) {  // the table's row into L1
    if (kP == 1 && rotate && w.pos >= 0 && live[0] && turn[0])
      asm volatile("prefetch.global.L1 [%0];" ::"l"(table_at(w.pos, 0)));
  };
  auto process = [&](uint32_t base, const Where& w, const Values<kP>& v) {
    const uint32_t row = base + grp;
    bool ok = row < src.rows && w.slot >= 0 && w.pos >= 0;
    if (w.pos == -2 && w.slot >= 0 && sub == 0) atomicOr(&g_status_append, FP8MLA_DEV_BAD_POSITION);
    if (ok && kKind != kQuery && static_cast<uint32_t>(w.slot) >= prm.num_slots) {
      if (sub == 0) atomicOr(&g_status_append, FP8MLA_DEV_BAD_SLOT);
      ok = false;
    }
    Piece p[kP];
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      unpack8(v.a[j], p[j].a);
      unpack8(v.b[j], p[j].b);
      if (ok && live[j] && turn[j]) {
        const float4* at = table_at(w.pos, j);
        float4 cs[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = __ldg(at + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // two pairs at a time: (cos, sin, cos, sin)
          auto turned = [](float& x, float& y, float c, float s) {
            const float rx = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
            y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
            x = rx;
          };
          if (half) {
            turned(p[j].a[2 * i], p[j].b[2 * i], cs[i].x, cs[i].y);
            turned(p[j].a[2 * i + 1], p[j].b[2 * i + 1], cs[i].z, cs[i].w);
          } else {
            float(&x)[8] = i < 2 ? p[j].a : p[j].b;
            turned(x[4 * (i % 2)], x[4 * (i % 2) + 1], cs[i].x, cs[i].y);
            turned(x[4 * (i % 2) + 2], x[4 * (i % 2) + 3], cs[i].z, cs[i].w);
          }
        }
      }
    }
    if constexpr (kKind == kQuery) {
      if (ok) {
        uint4* dst = reinterpret_cast<uint4*>(src.out) + static_cast<int64_t>(row) * (prm.head_dim / 8);
#pragma unroll
        for (int j = 0; j < kP; ++j)
          if (live[j]) {
            const auto& a = p[j].a;
            const auto& b = p[j].b;
            dst[c0[j]] = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                                    pack_bf16x2(a[6], a[7]));
            dst[c1[j]] = make_uint4(pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3]), pack_bf16x2(b[4], b[5]),
                                    pack_bf16x2(b[6], b[7]));
          }
      } else if (prm.zero_q && row < src.rows) {
        zero_row(src.out + static_cast<int64_t>(row) * prm.head_dim * 2, prm.head_dim, sub, kL);
      }
      return;
    }
    // the row in the cache: (block * h_kv + head) * page + offset
    const uint32_t head = row - fast_div(row, src.heads) * src.heads.d;
    const uint32_t block = fast_div(static_cast<uint32_t>(w.slot) & 0x7FFFFFFFu, prm.page);
    const int64_t dst_row = (static_cast<int64_t>(block) * src.heads.d + head) * prm.page.d +
                            (static_cast<uint32_t>(w.slot) - block * prm.page.d);
    if constexpr (kKind == kFp4) {
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        // Block of a chunk: a lane's two chunks, or (half layout) one chunk of this lane and of its neighbour, so
        // that two lanes share two blocks.  Each lane works out one scale; neighbours then swap.
        const float ma = amax8<true>(p[j].a), mb = amax8<true>(p[j].b);
        const bool shared = half && turn[j];
        const bool odd = shared && (sub & 1);
        const float theirs = __shfl_xor_sync(0xffffffffu, odd ? ma : mb, 1);
        const float other = shared ? theirs : mb;
        const float amax = fmax3_nan(odd ? mb : ma, other, other);
        const uint32_t s8 = pack_e4m3x2(__fmul_rn(amax, inv6), 0.f) & 0xFFu;
        const float inv = __frcp_rn(__fmul_rn(f16_lo(e4m3x2_to_f16x2(s8)), scale));
        const uint32_t s8x = __shfl_xor_sync(0xffffffffu, s8, 1);
        const float invx = __shfl_xor_sync(0xffffffffu, inv, 1);
        if (ok && live[j]) {
          const uint32_t s8a = odd ? s8x : s8, s8b = shared && !odd ? s8x : s8;
          const float ia = odd ? invx : inv, ib = shared && !odd ? invx : inv;
          float ya[8], yb[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            ya[i] = __fmul_rn(p[j].a[i], ia);
            yb[i] = __fmul_rn(p[j].b[i], ib);
          }
          uint32_t* dst = reinterpret_cast<uint32_t*>(src.out + dst_row * (prm.head_dim / 2));
          dst[c0[j]] = s8a != 0 ? pack_e2m1x8(ya) : 0u;
          dst[c1[j]] = s8b != 0 ? pack_e2m1x8(yb) : 0u;
          uint8_t* sc = src.block_scales + dst_row * (prm.head_dim / 16);
          if ((c0[j] & 1) == 0) sc[c0[j] / 2] = static_cast<uint8_t>(s8a);
          if ((c1[j] & 1) == 0) sc[c1[j] / 2] = static_cast<uint8_t>(s8b);
        }
      }
    } else {
      float inv = tensor_inv;
      if constexpr (kKind == kRowScales) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < kP; ++j) m = fmax3(m, amax8(p[j].a), amax8(p[j].b));
#pragma unroll
        for (int o = kL / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool lifted = m < kTinyAmax;
        if (lifted) {
#pragma unroll
          for (int j = 0; j < kP; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              p[j].a[i] = __fmul_rn(p[j].a[i], kTinyLift);
              p[j].b[i] = __fmul_rn(p[j].b[i], kTinyLift);
            }
        }
        inv = m > 0.f ? __fdiv_rn(448.f, lifted ? __fmul_rn(m, kTinyLift) : m) : 1.f;
        if (ok && sub == 0) src.row_scales[dst_row] = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
      }
      if (ok) {
        uint2* dst = reinterpret_cast<uint2*>(src.out + dst_row * prm.head_dim);
#pragma unroll
        for (int j = 0; j < kP; ++j)
          if (live[j]) {
            dst[c0[j]] = encode8(p[j].a, inv);
            dst[c1[j]] = encode8(p[j].b, inv);
          }
      }
    }
  };

  uint32_t base = (cta * (kThreads / 32) + threadIdx.x / 32) * kWarpRows;
  if (base >= src.rows) return;  // the same for the whole warp
  const uint32_t stride = ctas * (kThreads / 32) * kWarpRows;  // sums stay below 2^32: rows are below 2^31
  Where w0, w1, w2;
  Values<kP> v0, v1;
  look(base, w0);
  load(base, v0);
  look(base + stride, w1);
  for (;;) {
    const bool more = base + stride < src.rows;
    if (more) {
      load(base + stride, v1);
      look(base + 2 * stride, w2);
      ask(w1);
    }
    process(base, w0, v0);
    if (!more) break;
    base += stride;
    w0 = w1;
    w1 = w2;
    v0 = v1;
  }
}

template <int kL, int kP, int kKind>
__global__ void __launch_bounds__(kThreads, append_ctas<kP>()) kv_append_kernel(const __grid_constant__ Params prm) {
  griddep_wait();
  const uint32_t c = blockIdx.x;
  if (c < prm.first[1])
    run_class<kL, kP, kKind>(prm, prm.src[0], prm.table != nullptr, c, prm.first[1]);
  else if (c < prm.first[2])
    run_class<kL, kP, kKind>(prm, prm.src[1], false, c - prm.first[1], prm.first[2] - prm.first[1]);
  else
    run_class<kL, kP, kQuery>(prm, prm.src[2], true, c - prm.first[2], prm.first[3] - prm.first[2]);
}

template <int kL, int kP>
cudaError_t launch_append(Params& p, int kind, cudaStream_t stream) {
  constexpr uint32_t kBlockRows = kThreads / 32 * (32 / kL);
  // One wave of resident CTAs, shared out by the classes' rows.  A rotated row of K takes longer than one of V (a
  // prompt: 21.9 us with 13 : 10, 23.2 with 1 : 1, 23.4 with 2 : 1), less so where quantising weighs more.
  const uint64_t cap = static_cast<uint64_t>(device_sms()) * append_ctas<kP>();
  const uint64_t weight[3] = {p.table == nullptr ? 10u : (kind == kFp4 ? 11u : 13u), 10, 10};
  const uint64_t rows = weight[0] * p.src[0].rows + weight[1] * p.src[1].rows + weight[2] * p.src[2].rows;
  p.first[0] = 0;
  for (int i = 0; i < 3; ++i) {
    const uint64_t need = (p.src[i].rows + kBlockRows - 1) / kBlockRows;
    const uint64_t share = std::max<uint64_t>(1, cap * weight[i] * p.src[i].rows / rows);
    p.first[i + 1] = p.first[i] + static_cast<uint32_t>(std::min(need, share));
  }
  const dim3 grid(p.first[3]), block(kThreads);
  switch (kind) {
    case kTensor: return launch_dependent(kv_append_kernel<kL, kP, kTensor>, grid, block, 0, stream, p);
    case kRowScales: return launch_dependent(kv_append_kernel<kL, kP, kRowScales>, grid, block, 0, stream, p);
    default: return launch_dependent(kv_append_kernel<kL, kP, kFp4>, grid, block, 0, stream, p);
  }
}

// ------------------------------------------------------------------ read ----

struct ReadParams {
  const uint8_t* cache;
  const float* scale;
  const float* row_scales;
  const uint8_t* block_scales;
  const int32_t* slots;
  uint4* out;
  FastDiv heads, page;
  uint32_t rows, num_slots;
  int head_dim;
};

// Rows of a paged cache as bf16: value = fp32(E4M3 * scale), or fp32(E2M1 * fp32(s8 * scale)), rounded once.
// A group of kL lanes per row, kW values (16; 8 where head_dim is no multiple of 16) a lane at a time.  The same
// pipeline as the append: slots two steps ahead, codes and scales one ahead.  One row a step and five CTAs an SM
// (65537 x 8 rows 35.1 us, 8193 x 8 rows 6.0; two rows and three CTAs 35.1 and 6.6; one row, six 33.5 and 6.0 but
// 32768 x 8 rows 19.8 instead of 16.1; four 36.9, eight 42.7).
template <int kL, int kKind, int kW>
__global__ void __launch_bounds__(kThreads, kReadCtasPerSm) cache_read_kernel(const __grid_constant__ ReadParams prm) {
  constexpr int kBytes = kKind == kFp4 ? kW / 2 : kW;  // of codes a lane takes
  griddep_wait();
  const int lane = threadIdx.x % 32, sub = lane % kL, grp = lane / kL;
  const int pieces = prm.head_dim / kW;
  const int per_lane = (pieces + kL - 1) / kL;  // 1 up to head_dim 512
  float scale = 1.f;
  if constexpr (kKind != kRowScales) scale = __ldg(prm.scale);

  struct Row {
    int64_t src;  // row in the cache, or -1
    uint4 w;      // first piece's codes
    float s;      // and their scale
  };
  auto slot_of = [&](uint32_t base) {
    const uint32_t row = base + grp;
    return row < prm.rows ? __ldg(prm.slots + fast_div(row, prm.heads)) : -1;
  };
  auto fetch = [&](int64_t src, int piece, uint4& w, float& s) {
    const uint8_t* at = prm.cache + src * (kKind == kFp4 ? prm.head_dim / 2 : prm.head_dim) + piece * kBytes;
    w = make_uint4(0, 0, 0, 0);
    if constexpr (kBytes == 16) {
      w = __ldcs(reinterpret_cast<const uint4*>(at));
    } else {
      const uint2 x = __ldcs(reinterpret_cast<const uint2*>(at));
      w.x = x.x, w.y = x.y;
    }
    if constexpr (kKind == kFp4) {
      const uint32_t s8 = __ldg(prm.block_scales + src * (prm.head_dim / 16) + piece);
      s = __fmul_rn(f16_lo(e4m3x2_to_f16x2(s8)), scale);
    } else if constexpr (kKind == kRowScales) {
      s = __ldg(prm.row_scales + src);
    } else {
      s = scale;
    }
  };
  auto load = [&](uint32_t base, int32_t slot, Row& x) {
    const uint32_t row = base + grp;
    const uint32_t head = row - fast_div(row, prm.heads) * prm.heads.d;
    x.src = -1;
    x.s = 0.f;
    x.w = make_uint4(0, 0, 0, 0);
    if (slot >= 0 && static_cast<uint32_t>(slot) >= prm.num_slots) {
      if (sub == 0) atomicOr(&g_status_append, FP8MLA_DEV_BAD_SLOT);
    } else if (slot >= 0) {
      const uint32_t block = fast_div(static_cast<uint32_t>(slot), prm.page);
      x.src = (static_cast<int64_t>(block) * prm.heads.d + head) * prm.page.d + (slot - block * prm.page.d);
      if (sub < pieces) fetch(x.src, sub, x.w, x.s);
    }
  };
  auto store = [&](uint32_t row, int piece, const uint4& w, float s) {
    uint32_t o[kW / 2];
    if constexpr (kKind == kFp4) {
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < kW / 8; ++k) {
        e2m1x8_to_f16x2(k ? w.y : w.x, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[4 * k + i] = h[i];
      }
    } else {
      const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < kW / 4; ++i) {
        o[2 * i] = e4m3x2_to_f16x2(q[i]);
        o[2 * i + 1] = e4m3x2_to_f16x2(q[i] >> 16);
      }
    }
#pragma unroll
    for (int i = 0; i < kW / 2; ++i) o[i] = pack_bf16x2(__fmul_rn(f16_lo(o[i]), s), __fmul_rn(f16_hi(o[i]), s));
    uint4* dst = prm.out + (static_cast<int64_t>(row) * prm.head_dim + piece * kW) / 8;
#pragma unroll
    for (int i = 0; i < kW / 8; ++i) __stcs(dst + i, make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
  };
  auto process = [&](uint32_t base, const Row& x) {
    const uint32_t row = base + grp;
    if (row >= prm.rows) return;
    const bool none = x.src < 0;  // a row of zeros
    if (sub < pieces) store(row, sub, none ? make_uint4(0, 0, 0, 0) : x.w, none ? 0.f : x.s);
    for (int j = 1; j < per_lane; ++j) {
      const int piece = sub + j * kL;
      if (piece >= pieces) break;
      uint4 w = make_uint4(0, 0, 0, 0);
      float s = 0.f;
      if (x.src >= 0) fetch(x.src, piece, w, s);
      store(row, piece, w, s);
    }
  };

  constexpr uint32_t kWarpRows = 32 / kL;
  uint32_t base = (blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * kWarpRows;
  if (base >= prm.rows) return;  // the same for the whole warp
  const uint32_t stride = gridDim.x * (kThreads / 32) * kWarpRows;
  Row x0, x1;
  load(base, slot_of(base), x0);
  int32_t s1 = slot_of(base + stride), s2 = -1;
  for (;;) {
    const bool more = base + stride < prm.rows;
    if (more) {
      load(base + stride, s1, x1);
      s2 = slot_of(base + 2 * stride);
    }
    process(base, x0);
    if (!more) break;
    base += stride;
    x0 = x1;
    s1 = s2;
  }
}

template <int kL, int kW>
cudaError_t launch_read(const ReadParams& p, int kind, cudaStream_t stream) {
  constexpr uint32_t kBlockRows = kThreads / 32 * (32 / kL);
  const unsigned blocks = std::min<unsigned>((p.rows + kBlockRows - 1) / kBlockRows, device_sms() * kReadCtasPerSm);
  const dim3 grid(blocks), block(kThreads);
  switch (kind) {
    case kTensor: return launch_dependent(cache_read_kernel<kL, kTensor, kW>, grid, block, 0, stream, p);
    case kRowScales: return launch_dependent(cache_read_kernel<kL, kRowScales, kW>, grid, block, 0, stream, p);
    default: return launch_dependent(cache_read_kernel<kL, kFp4, 16>, grid, block, 0, stream, p);
  }
}

// The cache's kind from the scales given, or -1: E4M3 takes one scale or one per row, E2M1 one scale and the blocks'.
int kind_of(fp8mla_kv_dtype_t t, const void* scale, const void* row_scales, const void* block_scales) {
  if (t == FP8MLA_KV_E2M1)
    return scale != nullptr && block_scales != nullptr && row_scales == nullptr ? kFp4 : -1;
  if (block_scales != nullptr || (scale == nullptr) == (row_scales == nullptr)) return -1;
  return scale != nullptr ? kTensor : kRowScales;
}

// Whether what an append writes overlaps: caches, scales and the rotated queries each other, or a tensor that it reads
// (the rotated queries may take the queries' place).
bool shares_memory(const KvAppendArgs& a, int kind, bool has_v) {
  const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.page_size * a.h_kv;
  Rows written[7], read[3];
  int w = 0, r = 0;
  for (int i = 0; i < (has_v ? 2 : 1); ++i) {
    const CacheSide& s = a.side[i];
    written[w++] = block_of(s.cache, rows * a.head_dim / (kind == kFp4 ? 2 : 1));
    if (kind == kRowScales) written[w++] = block_of(s.row_scales, rows * 4);
    if (kind == kFp4) written[w++] = block_of(s.block_scales, rows * a.head_dim / 16);
    read[r++] = rows_of(s.x, s.token, s.head, a.n_tokens, a.h_kv, a.head_dim, 2);
  }
  const Rows q = rows_of(a.q, a.q_token, a.q_head, a.n_tokens, a.h_q, a.head_dim, 2);
  if (a.q != nullptr) {
    const Rows out = rows_of(a.q_out, static_cast<int64_t>(a.h_q) * a.head_dim, a.head_dim, a.n_tokens, a.h_q,
                             a.head_dim, 2);
    if (!same_rows(out, q)) read[r++] = q;
    written[w++] = out;
  }
  for (int i = 0; i < w; ++i) {
    for (int j = 0; j < i; ++j)
      if (rows_overlap(written[i], written[j])) return true;
    for (int j = 0; j < r; ++j)
      if (rows_overlap(written[i], read[j])) return true;
  }
  return false;
}

}  // namespace

fp8mla_status_t kv_append_entry(const KvAppendArgs& a, cudaStream_t stream) {
  if (a.kv_dtype != FP8MLA_KV_E4M3 && a.kv_dtype != FP8MLA_KV_E2M1) return FP8MLA_ERR_UNSUPPORTED_DTYPE;
  if (a.n_tokens < 0 || a.h_kv < 1 || a.head_dim < 16 || a.head_dim % 16 != 0 || a.head_dim > kMaxHeadDim ||
      a.page_size < 1 || a.num_blocks < 1 || (a.q != nullptr && a.h_q < 1) || a.layout < 0 ||
      a.layout > (FP8MLA_ROTARY_INTERLEAVED | FP8MLA_ROTARY_ZERO_Q))
    return FP8MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(a.n_tokens) * std::max(a.h_kv, a.q != nullptr ? a.h_q : 1) >= (1ll << 31) ||
      static_cast<int64_t>(a.num_blocks) * a.page_size >= (1ll << 31))
    return FP8MLA_ERR_INVALID_ARG;
  const bool has_v = a.side[1].x != nullptr || a.side[1].cache != nullptr;
  const int kind = kind_of(a.kv_dtype, a.side[0].scale, a.side[0].row_scales, a.side[0].block_scales);
  if (kind < 0) return FP8MLA_ERR_INVALID_ARG;
  if (has_v && kind_of(a.kv_dtype, a.side[1].scale, a.side[1].row_scales, a.side[1].block_scales) != kind)
    return FP8MLA_ERR_INVALID_ARG;
  if (a.table != nullptr) {
    const bool interleaved = a.layout & FP8MLA_ROTARY_INTERLEAVED;
    if (a.rot < 16 || a.rot % 16 != 0 || a.rot_offset < 0 || a.rot_offset % (interleaved ? 16 : 8) != 0 ||
        a.rot > a.head_dim - a.rot_offset || a.n_positions < 1 || a.n_positions > 0x7FFFFFFF || misaligned(a.table, 16))
      return FP8MLA_ERR_INVALID_ARG;
    // blocks of 16 values do not straddle a half layout's pieces
    if (kind == kFp4 && !interleaved && (a.rot % 32 != 0 || a.rot_offset % 16 != 0)) return FP8MLA_ERR_INVALID_ARG;
  } else if (a.q != nullptr) {
    return FP8MLA_ERR_INVALID_ARG;  // nothing to rotate the queries with
  }
  if (a.n_tokens == 0) return FP8MLA_OK;
  if (a.slot_mapping == nullptr || misaligned(a.slot_mapping, 4)) return FP8MLA_ERR_INVALID_ARG;
  if (a.table != nullptr && (a.positions == nullptr || misaligned(a.positions, a.positions_64 ? 8 : 4)))
    return FP8MLA_ERR_INVALID_ARG;
  for (int i = 0; i < (has_v ? 2 : 1); ++i) {
    const CacheSide& s = a.side[i];
    if (s.x == nullptr || s.cache == nullptr || misaligned(s.x, 16) || misaligned(s.cache, 16) ||
        (s.token | s.head) % 8 != 0 || misaligned(s.row_scales, 4) || misaligned(s.scale, 4))
      return FP8MLA_ERR_INVALID_ARG;
  }
  if (a.q != nullptr && (a.q_out == nullptr || misaligned(a.q, 16) || misaligned(a.q_out, 16) ||
                         (a.q_token | a.q_head) % 8 != 0))
    return FP8MLA_ERR_INVALID_ARG;
  if (shares_memory(a, kind, has_v)) return FP8MLA_ERR_INVALID_ARG;
  Params p;
  for (int i = 0; i < 2; ++i) {
    const CacheSide& s = a.side[i];
    p.src[i].x = static_cast<const uint16_t*>(s.x);
    p.src[i].token = s.token;
    p.src[i].head = s.head;
    p.src[i].out = static_cast<uint8_t*>(s.cache);
    p.src[i].scale = s.scale;
    p.src[i].row_scales = s.row_scales;
    p.src[i].block_scales = static_cast<uint8_t*>(s.block_scales);
    p.src[i].heads = make_fast_div(a.h_kv);
    p.src[i].rows = i == 0 || has_v ? static_cast<uint32_t>(a.n_tokens) * a.h_kv : 0;
  }
  p.src[2] = Source{static_cast<const uint16_t*>(a.q), a.q_token, a.q_head, static_cast<uint8_t*>(a.q_out), nullptr,
                    nullptr, nullptr, make_fast_div(a.q != nullptr ? a.h_q : 1),
                    a.q != nullptr ? static_cast<uint32_t>(a.n_tokens) * a.h_q : 0};
  p.slots = a.slot_mapping;
  p.positions = a.positions;
  p.positions_64 = a.positions_64;
  p.table = reinterpret_cast<const float2*>(a.table);
  p.n_positions = a.n_positions;
  p.page = make_fast_div(a.page_size);
  p.num_slots = static_cast<uint32_t>(static_cast<int64_t>(a.num_blocks) * a.page_size);
  p.rot = a.rot;
  p.rot_offset = a.rot_offset;
  p.interleaved = a.layout & FP8MLA_ROTARY_INTERLEAVED;
  p.zero_q = a.layout & FP8MLA_ROTARY_ZERO_Q;
  p.head_dim = a.head_dim;
  const int pairs = a.head_dim / 16;
  cudaError_t e;
  // the fewest lanes with one piece each; three where that leaves fewer of them idle (head_dim 192, 576).  Rows above
  // 768 values take two pieces a lane, and at three CTAs of 80 registers spill 28 to 88 bytes: no cache here has them
  if (pairs <= 1) e = launch_append<1, 1>(p, kind, stream);
  else if (pairs <= 2) e = launch_append<2, 1>(p, kind, stream);
  else if (pairs <= 4) e = launch_append<4, 1>(p, kind, stream);
  else if (pairs <= 8) e = launch_append<8, 1>(p, kind, stream);
  else if (pairs <= 12) e = launch_append<4, 3>(p, kind, stream);
  else if (pairs <= 16) e = launch_append<16, 1>(p, kind, stream);
  else if (pairs <= 32) e = launch_append<32, 1>(p, kind, stream);
  else if (pairs <= 48) e = launch_append<16, 3>(p, kind, stream);
  else e = launch_append<32, 2>(p, kind, stream);
  return e == cudaSuccess ? FP8MLA_OK : FP8MLA_ERR_CUDA;
}

fp8mla_status_t cache_read_entry(const CacheReadArgs& a, cudaStream_t stream) {
  if (a.kv_dtype != FP8MLA_KV_E4M3 && a.kv_dtype != FP8MLA_KV_E2M1) return FP8MLA_ERR_UNSUPPORTED_DTYPE;
  if (a.n < 0 || a.h_kv < 1 || a.page_size < 1 || a.num_blocks < 1 || a.head_dim < 8 || a.head_dim > kMaxHeadDim ||
      a.head_dim % (a.kv_dtype == FP8MLA_KV_E2M1 ? 16 : 8) != 0)
    return FP8MLA_ERR_INVALID_ARG;
  const int kind = kind_of(a.kv_dtype, a.scale, a.row_scales, a.block_scales);
  if (kind < 0) return FP8MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(a.n) * a.h_kv >= (1ll << 31) ||
      static_cast<int64_t>(a.num_blocks) * a.page_size >= (1ll << 31))
    return FP8MLA_ERR_INVALID_ARG;
  if (a.n == 0) return FP8MLA_OK;
  if (a.cache == nullptr || a.slots == nullptr || a.out == nullptr || misaligned(a.cache, 16) ||
      misaligned(a.out, 16) || misaligned(a.slots, 4) || misaligned(a.scale, 4) || misaligned(a.row_scales, 4))
    return FP8MLA_ERR_INVALID_ARG;
  const uint64_t rows = static_cast<uint64_t>(a.num_blocks) * a.page_size * a.h_kv;
  const Rows out = block_of(a.out, static_cast<uint64_t>(a.n) * a.h_kv * a.head_dim * 2);
  if (rows_overlap(out, block_of(a.cache, rows * a.head_dim / (kind == kFp4 ? 2 : 1))) ||
      rows_overlap(out, block_of(a.row_scales, rows * 4)) ||
      rows_overlap(out, block_of(a.block_scales, rows * a.head_dim / 16)))
    return FP8MLA_ERR_INVALID_ARG;
  ReadParams p;
  p.cache = static_cast<const uint8_t*>(a.cache);
  p.scale = a.scale;
  p.row_scales = a.row_scales;
  p.block_scales = static_cast<const uint8_t*>(a.block_scales);
  p.slots = a.slots;
  p.out = static_cast<uint4*>(a.out);
  p.heads = make_fast_div(a.h_kv);
  p.page = make_fast_div(a.page_size);
  p.rows = static_cast<uint32_t>(a.n) * a.h_kv;
  p.num_slots = static_cast<uint32_t>(static_cast<int64_t>(a.num_blocks) * a.page_size);
  p.head_dim = a.head_dim;
  const int pieces = a.head_dim / 16;
  cudaError_t e;
  if (a.head_dim % 16 != 0) e = launch_read<32, 8>(p, kind, stream);  // a rare width: lanes may idle
  else if (pieces <= 1) e = launch_read<1, 16>(p, kind, stream);
  else if (pieces <= 2) e = launch_read<2, 16>(p, kind, stream);
  else if (pieces <= 4) e = launch_read<4, 16>(p, kind, stream);
  else if (pieces <= 8) e = launch_read<8, 16>(p, kind, stream);
  else if (pieces <= 16) e = launch_read<16, 16>(p, kind, stream);
  else e = launch_read<32, 16>(p, kind, stream);
  return e == cudaSuccess ? FP8MLA_OK : FP8MLA_ERR_CUDA;
}

uint32_t kv_append_read_and_clear_status() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_status_append, sizeof(v));
  cudaMemcpyToSymbol(g_status_append, &z, sizeof(z));
  return v;
}

}  // namespace fp8mla
