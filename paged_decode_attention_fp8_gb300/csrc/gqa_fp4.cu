// Paged GQA decode over a cache held in 4 bits, sm_103a.
//
// The operation: for sequence b, query token i and query head h,
//   out = softmax_j(scale * q . k_j) @ v_j,
// k_j[d] = k_scale * s8_k[j, d / 16] * E2M1(code_k[j, d]) and v_j likewise:
// E2M1 codes (two to a byte, the even dimension in the low nibble), one E4M3
// scale per 16 dimensions of a row, one float32 scale per cache; KV head
// h / (h_q / h_kv); the masks, windows and sinks of the FP8 entry.
//
// What bounds it: a (key, KV head) pair is head_dim + head_dim / 8 bytes of K
// and V together (144 at 128), read once; the products are a few per cent of
// the tensor rate, but every code has to become a 16-bit operand, so the issue
// slots of turning codes into operands are the second limit.  At the copy
// bandwidth an SM has about six cycles per key of 256 values.
//
// Design:
//   * A warp works alone on tiles of 16 keys: it fetches them into its own
//     ring in shared memory by 16-byte cp.async several tiles ahead, keeps
//     its own running maximum, sum and accumulator, and meets the CTA's other
//     warps only at the end.  No barrier in the loop but __syncwarp.
//   * Codes go from shared memory to registers to the product's A fragment:
//     S^T = K Q^T (M = 16 keys, N = 8 columns, K = head_dim) and
//     O^T = V^T P^T (M = 16 dims, N = 8 columns, K = 16 keys) as register-
//     fragment products, for which a code is converted in the lane that needs
//     it.  A tensor-memory product would need the expanded 16-bit tile written
//     to shared or tensor memory first: 512 bytes a key against the 128 that
//     an SM can store in a cycle, four of the six cycles a key has.
//   * The order of the contraction is free, so each lane takes contiguous
//     bytes: lane (g, t) of K row g holds dims [t hd/4, (t + 1) hd/4), and Q's
//     fragment is laid out to match; of V, lane (g, t) holds the hd/8 dims
//     from g hd/8 of keys t, t + 4, t + 8, t + 12.  A code's byte holds two
//     neighbouring dims; for V the operand pairs two keys instead, formed on
//     the nibbles (two shift-and-select steps for eight codes).
//   * E2M1 * E4M3 has at most six significant bits and lies in f16's range
//     (subnormals included), so K and V operands are exact.  Q is bf16 times
//     a power of two per column, exact in f16 down to 2^-38 of its largest
//     value; P is rounded to f16 (half a step: 2^-11), sums are f32.
//   * A column's reference is 7 (log2) below the largest score it was taken
//     from and moves only when a score passes it by more than 15: P stays
//     within f16 (2^15), weights down to 2^-21 of the largest keep f16's
//     relative precision, and most tiles need no shuffle.
//   * The keys of a (sequence, KV head) are cut into contiguous shards over
//     CTAs when the grid would not fill the GPU, merged by a second kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "gqa_fp4.h"

namespace fp8mla {

__device__ uint32_t g_status_fp4;

namespace fp4 {

constexpr int kTile = 16;       // keys of a tile
constexpr int kWarps = 8;
constexpr int kStages = 4;      // tiles of a warp's ring
constexpr int kMaxQLen = 16;
constexpr int kMaxCols = 128;   // q_len * (h_q / h_kv)
constexpr float kBelow = 7.f;   // a reference lies this far below the largest score (log2) ...
constexpr float kTau = 15.f;    // ... and moves when a score is this far above it

struct Params {
  const uint16_t* q;
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* ks;
  const uint8_t* vs;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_table;
  const int32_t* seqlens;
  const uint8_t* spec_mask;
  const float* sinks;
  uint16_t* out;
  float* lse;
  float4* ws_o;   // [slot][NT * hd / 16][32 lanes] fragments
  float2* ws_ml;  // [slot][NT * 8]
  int num_blocks, max_blocks, h_q, h_kv, group, splits, q_len, window;
  int page_shift;  // log2(page_size / 16)
  float softmax_scale;
};

// Where a tile's bytes lie in a stage: K codes, V codes, K scales, V scales.
template <int kHd>
struct Lay {
  static constexpr int kRow = kHd / 2;            // bytes of codes per key
  static constexpr int kSRow = kHd / 16;          // bytes of scales per key
  static constexpr int kK = 0, kV = kTile * kRow;
  static constexpr int kKs = 2 * kTile * kRow, kVs = kKs + kTile * kSRow;
  static constexpr int kBytes = kVs + kTile * kSRow;
  static constexpr int kChunks = kTile * kRow / 16;    // 16-byte chunks of a code tile
  static constexpr int kSChunks = kTile * kSRow / 16;  // of a scale tile
};

// Byte offset of 16-byte chunk c of K row r in its tile.  A load instruction's
// phase reads rows m and m + 4 (keys are dealt to fragment rows that way);
// rows or chunks are exchanged so that the two fall into different banks.
template <int kHd>
__device__ __forceinline__ int k_place(int r, int c) {
  if constexpr (kHd == 64) return (r ^ (((r >> 2) & 1) << 1)) * 32 + c * 16;
  if constexpr (kHd == 128) return (r ^ ((r >> 2) & 1)) * 64 + c * 16;
  return r * 128 + ((c ^ ((r >> 2) & 1)) << 4);
}
// The same for V, whose phases read four neighbouring rows.
template <int kHd>
__device__ __forceinline__ int v_place(int r, int c) {
  if constexpr (kHd == 64) return r * 32 + c * 16;
  if constexpr (kHd == 128) return r * 64 + ((c ^ (((r >> 1) & 1) << 1)) << 4);
  return r * 128 + ((c ^ ((r & 3) << 1)) << 4);
}

// Power of two e with amax * 2^-e in [2^14, 2^15) (clamped so that 2^e and 2^-e are normal).
__device__ __forceinline__ int q_exponent(float amax) {
  const int expo = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFFu);
  return max(-100, min(100, expo - 127 - 14));
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

// Fragment positions -> keys of the tile: row g of S^T is key (g / 2) + 4 (g % 2), row g + 8 that plus 8, so the
// pairs (2t, 2t + 1) and (2t + 8, 2t + 9) of P^T's contraction are keys t, t + 4 and t + 8, t + 12.

template <int kHd, int kNT>
__global__ void __launch_bounds__(kWarps * 32, kNT == 1 && kHd <= 128 ? 2 : 1) fp4_decode_kernel(const Params prm) {
  using L = Lay<kHd>;
  constexpr int kSteps = kHd / 16;     // products of a tile, for K and for V
  constexpr int kKWords = kHd / 32;    // 32-bit words of a lane's part of a K row
  constexpr int kVWords = kHd >= 64 ? kHd / 64 : 1;  // of a lane's part of a V row
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t s_vis[kMaxQLen];
  __shared__ float s_m[kWarps][kNT * 8], s_l[kWarps][kNT * 8];

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const int split = blockIdx.x % prm.splits;
  const int seq = blockIdx.x / prm.splits;
  const int b = seq / prm.h_kv, kvh = seq % prm.h_kv;
  const int col0 = blockIdx.y * (kNT * 8);
  const int ncols = min(prm.q_len * prm.group - col0, kNT * 8);

  griddep_wait();
  griddep_launch_dependents();

  const int page = kTile << prm.page_shift;
  int s_k = prm.seqlens[b];
  if (s_k < 0 || (static_cast<long long>(s_k) + page - 1) / page > prm.max_blocks) {
    if (threadIdx.x == 0) atomicOr(&g_status_fp4, FP8MLA_DEV_BAD_SEQLEN);
    s_k = 0;
  }
  const int start = s_k - prm.q_len;  // position of the block's first token
  const int k_lo = prm.window > 0 ? max(0, start - prm.window + 1) : 0;
  const int tile_lo = k_lo / kTile;
  const int tiles = max(0, (s_k + kTile - 1) / kTile - tile_lo);
  const int t0 = tile_lo + static_cast<int>(static_cast<long long>(split) * tiles / prm.splits);
  const int t1 = tile_lo + static_cast<int>(static_cast<long long>(split + 1) * tiles / prm.splits);
  const int n_mine = t1 - t0 > warp ? (t1 - t0 - warp + kWarps - 1) / kWarps : 0;

  const int32_t* bt_row = prm.block_table + static_cast<size_t>(b) * prm.max_blocks;
  uint8_t* ring = smem + warp * (kStages * L::kBytes);

  // Entries of the block table, 32 tiles of this warp at a time.
  int entry = 0;
  auto fetch_entries = [&](int i0) {
    const int i = i0 + lane;
    entry = 0;
    if (i < n_mine) {
      entry = __ldg(bt_row + ((t0 + warp + i * kWarps) >> prm.page_shift));
      if (entry < 0 || entry >= prm.num_blocks) {
        atomicOr(&g_status_fp4, FP8MLA_DEV_BAD_PAGE);
        entry = 0;
      }
    }
  };
  auto issue = [&](int i) {
    if (i < n_mine) {
      if ((i & 31) == 0) fetch_entries(i);
      const int blk = __shfl_sync(0xffffffffu, entry, i & 31);
      const int tile = t0 + warp + i * kWarps;
      const int in_page = tile & ((1 << prm.page_shift) - 1);
      const int64_t row = (static_cast<int64_t>(blk) * prm.h_kv + kvh) * page + in_page * kTile;
      const uint32_t st = smem_u32(ring + (i % kStages) * L::kBytes);
      const uint8_t* ksrc = prm.k + row * L::kRow;
      const uint8_t* vsrc = prm.v + row * L::kRow;
#pragma unroll
      for (int c = lane; c < L::kChunks; c += 32) {
        const int r = c / (L::kRow / 16), cc = c % (L::kRow / 16);
        cp_async16(st + L::kK + k_place<kHd>(r, cc), ksrc + c * 16, 16u);
        cp_async16(st + L::kV + v_place<kHd>(r, cc), vsrc + c * 16, 16u);
      }
      if (lane < 2 * L::kSChunks) {
        const bool is_v = lane >= L::kSChunks;
        const int c = is_v ? lane - L::kSChunks : lane;
        cp_async16(st + (is_v ? L::kVs : L::kKs) + c * 16, (is_v ? prm.vs : prm.ks) + row * L::kSRow + c * 16, 16u);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  // Which keys of the speculative block its token i sees: its mask row, or those up to itself.
  if (threadIdx.x < prm.q_len) {
    uint32_t bits = 0;
    if (prm.spec_mask != nullptr) {
      const uint8_t* row = prm.spec_mask + (static_cast<size_t>(b) * prm.q_len + threadIdx.x) * prm.q_len;
      for (int c = 0; c < prm.q_len; ++c)
        if (__ldg(row + c)) bits |= 1u << c;
    } else {
      bits = (2u << threadIdx.x) - 1u;
    }
    s_vis[threadIdx.x] = bits;
  }

  // Q's fragments: lane (g, t) holds dims [t hd/4, (t + 1) hd/4) of column g, as f16 with a power of two out
  uint32_t qf[kNT][kSteps][2];
  float cq[kNT][2];
  int tok[kNT][2];
  {
    const float c0 = prm.softmax_scale * kLog2e * __ldg(prm.k_scale);
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      const int col = col0 + n * 8 + g;
      uint32_t w[kSteps * 2];
      if (n * 8 + g < ncols) {
        const uint16_t* src = prm.q + ((static_cast<size_t>(b) * prm.q_len + col / prm.group) * prm.h_q +
                                       kvh * prm.group + col % prm.group) * kHd + t * (kHd / 4);
#pragma unroll
        for (int j = 0; j < kSteps / 2; ++j) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(src) + j);
          w[4 * j] = x.x, w[4 * j + 1] = x.y, w[4 * j + 2] = x.z, w[4 * j + 3] = x.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < kSteps * 2; ++j) w[j] = 0;
      }
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < kSteps * 2; ++j) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[j])), fabsf(bf16_hi(w[j]))));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = q_exponent(amax);
      const float inv = exp2i(-e), qs = exp2i(e);
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        qf[n][j][0] = pack_f16x2(bf16_lo(w[2 * j]) * inv, bf16_hi(w[2 * j]) * inv);
        qf[n][j][1] = pack_f16x2(bf16_lo(w[2 * j + 1]) * inv, bf16_hi(w[2 * j + 1]) * inv);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        cq[n][k] = c0 * __shfl_sync(0xffffffffu, qs, 4 * (2 * t + k));
        tok[n][k] = min((col0 + n * 8 + 2 * t + k) / prm.group, prm.q_len - 1);
      }
    }
  }
  __syncthreads();  // s_vis

  // Tiles whose keys every column sees: before the speculative block (or, for one token, the end) and, with a
  // window, from the last token's first key on.
  const int full_end = prm.q_len == 1 && prm.spec_mask == nullptr ? s_k : max(0, start);
  const int full_lo = prm.window > 0 ? max(0, s_k - prm.window) : 0;

  float o[kNT][kSteps][4];
  float m[kNT][2], l[kNT][2];
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[n][j][k] = 0.f;
    m[n][0] = m[n][1] = kNegInf;
    l[n][0] = l[n][1] = 0.f;
  }
  const int r0 = (g >> 1) + 4 * (g & 1);  // keys of fragment rows g and g + 8
  const int r1 = r0 + 8;

  for (int i = 0; i < n_mine; ++i) {
    cp_async_wait_group<kStages - 2>();
    __syncwarp();
    issue(i + kStages - 1);
    const uint8_t* st = ring + (i % kStages) * L::kBytes;
    const int tok0 = (t0 + warp + i * kWarps) * kTile;

    // ---- S^T = K Q^T
    float s[kNT][4];
#pragma unroll
    for (int n = 0; n < kNT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
    {
      uint32_t ka[kKWords], kb[kKWords];
      if constexpr (kHd == 64) {
        const uint2 x = *reinterpret_cast<const uint2*>(st + L::kK + k_place<kHd>(r0, t >> 1) + (t & 1) * 8);
        const uint2 y = *reinterpret_cast<const uint2*>(st + L::kK + k_place<kHd>(r1, t >> 1) + (t & 1) * 8);
        ka[0] = x.x, ka[1] = x.y, kb[0] = y.x, kb[1] = y.y;
      } else {
#pragma unroll
        for (int c = 0; c < kKWords / 4; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(st + L::kK + k_place<kHd>(r0, t * (kKWords / 4) + c));
          const uint4 y = *reinterpret_cast<const uint4*>(st + L::kK + k_place<kHd>(r1, t * (kKWords / 4) + c));
          ka[4 * c] = x.x, ka[4 * c + 1] = x.y, ka[4 * c + 2] = x.z, ka[4 * c + 3] = x.w;
          kb[4 * c] = y.x, kb[4 * c + 1] = y.y, kb[4 * c + 2] = y.z, kb[4 * c + 3] = y.w;
        }
      }
      // block scales of the lane's dims (hd / 64 blocks), two f16 copies each
      uint32_t sa[kHd / 64], sb[kHd / 64];
      if constexpr (kHd == 64) {
        const uint32_t x = e4m3x2_to_f16x2(st[L::kKs + r0 * 4 + t] | (st[L::kKs + r1 * 4 + t] << 8));
        sa[0] = prmt(x, 0, 0x1010);
        sb[0] = prmt(x, 0, 0x3232);
      } else {
#pragma unroll
        for (int c = 0; c < kHd / 128; ++c) {
          const uint32_t x = e4m3x2_to_f16x2(
              *reinterpret_cast<const uint16_t*>(st + L::kKs + r0 * L::kSRow + t * (kHd / 64) + 2 * c));
          const uint32_t y = e4m3x2_to_f16x2(
              *reinterpret_cast<const uint16_t*>(st + L::kKs + r1 * L::kSRow + t * (kHd / 64) + 2 * c));
          sa[2 * c] = prmt(x, 0, 0x1010), sa[2 * c + 1] = prmt(x, 0, 0x3232);
          sb[2 * c] = prmt(y, 0, 0x1010), sb[2 * c + 1] = prmt(y, 0, 0x3232);
        }
      }
#pragma unroll
      for (int w = 0; w < kKWords; ++w) {
        uint32_t x[4], y[4];
        e2m1x8_to_f16x2(ka[w], x);
        e2m1x8_to_f16x2(kb[w], y);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[k] = mul_f16x2(x[k], sa[w / 2]);
          y[k] = mul_f16x2(y[k], sb[w / 2]);
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          mma_f16_16x8x16(s[n], x[0], y[0], x[1], y[1], qf[n][2 * w][0], qf[n][2 * w][1]);
          mma_f16_16x8x16(s[n], x[2], y[2], x[3], y[3], qf[n][2 * w + 1][0], qf[n][2 * w + 1][1]);
        }
      }
    }

    // ---- softmax: u = score in log2 units
    const bool whole = tok0 + kTile <= full_end && tok0 >= full_lo;
    bool grow = false;
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[n][k] *= cq[n][k & 1];
      if (!whole) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int p = tok0 + (k < 2 ? r0 : r1);
          const int ti = tok[n][k & 1];
          const int c_blk = p - start;
          const bool vis = p < s_k && (c_blk < 0 || ((s_vis[ti] >> c_blk) & 1u)) &&
                           (prm.window == 0 || ti - c_blk < prm.window);
          if (!vis) s[n][k] = kNegInf;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) grow |= fmaxf(s[n][k], s[n][k + 2]) > m[n][k] + kTau;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float mx = fmaxf(s[n][k], s[n][k + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          if (mx > m[n][k] + kTau) {
            const float alpha = ex2_approx(m[n][k] - (mx - kBelow));
            m[n][k] = mx - kBelow;
            l[n][k] *= alpha;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              o[n][j][k] *= alpha;
              o[n][j][k + 2] *= alpha;
            }
          }
        }
    }
    uint32_t pf[kNT][2];
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
      float p[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = ex2_approx(s[n][k] - (m[n][k & 1] == kNegInf ? 0.f : m[n][k & 1]));
      l[n][0] += p[0] + p[2];
      l[n][1] += p[1] + p[3];
      pf[n][0] = movmatrix_trans(pack_f16x2(p[0], p[1]));
      pf[n][1] = movmatrix_trans(pack_f16x2(p[2], p[3]));
    }

    // ---- O^T += V^T P^T
    {
      uint32_t v[4][kVWords];
      uint32_t sc[4];  // scale bytes of the lane's dims, keys t, t + 4, t + 8, t + 12
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = t + 4 * k;
        if constexpr (kHd == 64) {
          v[k][0] = *reinterpret_cast<const uint32_t*>(st + L::kV + v_place<kHd>(r, g >> 2) + (g & 3) * 4);
          sc[k] = st[L::kVs + r * 4 + (g >> 1)];
        } else if constexpr (kHd == 128) {
          const uint2 x = *reinterpret_cast<const uint2*>(st + L::kV + v_place<kHd>(r, g >> 1) + (g & 1) * 8);
          v[k][0] = x.x, v[k][1] = x.y;
          sc[k] = st[L::kVs + r * 8 + g];
        } else {
          const uint4 x = *reinterpret_cast<const uint4*>(st + L::kV + v_place<kHd>(r, g));
          v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
          sc[k] = *reinterpret_cast<const uint16_t*>(st + L::kVs + r * 16 + 2 * g);
        }
        // a key that no column sees has a zero weight; its scale may be anything (NaN), so it is zeroed
        if (!whole && (tok0 + r >= s_k || tok0 + r < k_lo)) sc[k] = 0;
      }
#pragma unroll
      for (int w = 0; w < kVWords; ++w) {
        if (kHd == 256 && w == 2) {
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[k] >>= 8;
        }
        const uint32_t sab = e4m3x2_to_f16x2((sc[0] & 0xFFu) | ((sc[1] & 0xFFu) << 8));
        const uint32_t scd = e4m3x2_to_f16x2((sc[2] & 0xFFu) | ((sc[3] & 0xFFu) << 8));
        constexpr uint32_t kLow = 0x0F0F0F0Fu;
        uint32_t x[4], y[4], z[4], u[4];
        e2m1x8_to_f16x2((v[0][w] & kLow) | ((v[1][w] << 4) & ~kLow), x);
        e2m1x8_to_f16x2(((v[0][w] >> 4) & kLow) | (v[1][w] & ~kLow), y);
        e2m1x8_to_f16x2((v[2][w] & kLow) | ((v[3][w] << 4) & ~kLow), z);
        e2m1x8_to_f16x2(((v[2][w] >> 4) & kLow) | (v[3][w] & ~kLow), u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a0 = mul_f16x2(x[k], sab), a1 = mul_f16x2(y[k], sab);
          const uint32_t a2 = mul_f16x2(z[k], scd), a3 = mul_f16x2(u[k], scd);
#pragma unroll
          for (int n = 0; n < kNT; ++n) mma_f16_16x8x16(o[n][4 * w + k], a0, a1, a2, a3, pf[n][0], pf[n][1]);
        }
      }
    }
  }

  // ---- the warps' states are merged in shared memory, in fragment order
  cp_async_wait_all();
#pragma unroll
  for (int n = 0; n < kNT; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x = l[n][k];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      l[n][k] = x;
      if (g == 0) {
        s_m[warp][n * 8 + 2 * t + k] = m[n][k];
        s_l[warp][n * 8 + 2 * t + k] = x;
      }
    }
  __syncthreads();  // also: every warp is done with its ring
  float4* part = reinterpret_cast<float4*>(smem);  // [warp][n][j][lane]
#pragma unroll
  for (int n = 0; n < kNT; ++n) {
    float f[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float mx = kNegInf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][n * 8 + 2 * t + k]);
      f[k] = m[n][k] == kNegInf ? 0.f : ex2_approx(m[n][k] - mx);
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
      part[((warp * kNT + n) * kSteps + j) * 32 + lane] =
          make_float4(o[n][j][0] * f[0], o[n][j][1] * f[1], o[n][j][2] * f[0], o[n][j][3] * f[1]);
  }
  __syncthreads();
  const float v_scale = __ldg(prm.v_scale);
  const size_t slot = (static_cast<size_t>(seq) * gridDim.y + blockIdx.y) * prm.splits + split;
  for (int x = threadIdx.x; x < kNT * kSteps * 32; x += kWarps * 32) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 y = part[w * (kNT * kSteps * 32) + x];
      a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
    }
    const int n = x / (kSteps * 32), j = x / 32 % kSteps, gg = x % 32 / 4, tt = x % 4;
    if (prm.splits > 1) prm.ws_o[slot * (kNT * kSteps * 32) + x] = a;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = n * 8 + 2 * tt + k;
      float mx = kNegInf, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][c]);
      if (mx != kNegInf) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_l[w][c] * ex2_approx(s_m[w][c] - mx);
      }
      if (prm.splits > 1) {
        if (j == 0 && gg == 0) prm.ws_ml[slot * (kNT * 8) + c] = make_float2(mx, sum);
        continue;
      }
      if (c >= ncols) continue;
      const int col = col0 + c, hq = kvh * prm.group + col % prm.group;
      const size_t row = (static_cast<size_t>(b) * prm.q_len + col / prm.group) * prm.h_q + hq;
      float fac, lse;
      finish_row(mx, sum, prm.sinks ? prm.sinks[hq] : kNegInf, v_scale, &fac, &lse);
      *reinterpret_cast<uint32_t*>(prm.out + row * kHd + gg * (kHd / 8) + 2 * j) =
          pack_bf16x2((k ? a.y : a.x) * fac, (k ? a.w : a.z) * fac);
      if (j == 0 && gg == 0) prm.lse[row] = lse;
    }
  }
}

// Merge of the shards: one CTA per (sequence, KV head, column tile); thread x owns one float4 of the fragment order
// (two dims of two columns), each weighted by 2^(m_s - M).
template <int kHd, int kNT>
__global__ void __launch_bounds__(256) fp4_combine_kernel(const Params prm) {
  constexpr int kSteps = kHd / 16, kFrag = kNT * kSteps * 32;
  griddep_wait();
  const int seq = blockIdx.x, b = seq / prm.h_kv, kvh = seq % prm.h_kv;
  const int col0 = blockIdx.y * (kNT * 8);
  const int ncols = min(prm.q_len * prm.group - col0, kNT * 8);
  const size_t slot0 = (static_cast<size_t>(seq) * gridDim.y + blockIdx.y) * prm.splits;
  const float v_scale = __ldg(prm.v_scale);
  for (int x = threadIdx.x; x < kFrag; x += 256) {
    const int n = x / (kSteps * 32), j = x / 32 % kSteps, gg = x % 32 / 4, tt = x % 4;
    const int c = n * 8 + 2 * tt;
    if (c >= ncols) continue;
    float m0 = kNegInf, m1 = kNegInf;
    for (int s = 0; s < prm.splits; ++s) {
      const float4 ml = *reinterpret_cast<const float4*>(prm.ws_ml + (slot0 + s) * (kNT * 8) + c);
      m0 = fmaxf(m0, ml.x);
      m1 = fmaxf(m1, ml.z);
    }
    const float b0 = m0 == kNegInf ? 0.f : m0, b1 = m1 == kNegInf ? 0.f : m1;
    float l0 = 0.f, l1 = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < prm.splits; ++s) {
      const float4 ml = *reinterpret_cast<const float4*>(prm.ws_ml + (slot0 + s) * (kNT * 8) + c);
      const float4 y = prm.ws_o[(slot0 + s) * kFrag + x];
      const float w0 = ex2_approx(ml.x - b0), w1 = ex2_approx(ml.z - b1);
      l0 += ml.y * w0;
      l1 += ml.w * w1;
      a.x += y.x * w0, a.y += y.y * w1, a.z += y.z * w0, a.w += y.w * w1;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (c + k >= ncols) continue;
      const int col = col0 + c + k, hq = kvh * prm.group + col % prm.group;
      const size_t row = (static_cast<size_t>(b) * prm.q_len + col / prm.group) * prm.h_q + hq;
      float fac, lse;
      finish_row(k ? m1 : m0, k ? l1 : l0, prm.sinks ? prm.sinks[hq] : kNegInf, v_scale, &fac, &lse);
      *reinterpret_cast<uint32_t*>(prm.out + row * kHd + gg * (kHd / 8) + 2 * j) =
          pack_bf16x2((k ? a.y : a.x) * fac, (k ? a.w : a.z) * fac);
      if (j == 0 && gg == 0) prm.lse[row] = lse;
    }
  }
}

// ---------------------------------------------------------------- host ----

int col_tiles(int cols, int* nt) {  // columns run eight or sixteen to a CTA
  *nt = cols <= 8 ? 1 : 2;
  return (cols + 8 * *nt - 1) / (8 * *nt);
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

template <int kHd, int kNT>
cudaError_t launch(const Params& prm, int seqs, int ct, cudaStream_t stream) {
  const size_t smem = std::max<size_t>(static_cast<size_t>(kWarps) * kStages * Lay<kHd>::kBytes,
                                       static_cast<size_t>(kWarps) * kNT * (kHd / 16) * 32 * sizeof(float4));
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = configure_once(configured, [&] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(fp4_decode_kernel<kHd, kNT>),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  e = launch_dependent(fp4_decode_kernel<kHd, kNT>,
                       dim3(static_cast<unsigned>(seqs) * static_cast<unsigned>(prm.splits), ct), dim3(kWarps * 32),
                       smem, stream, prm);
  if (e != cudaSuccess || prm.splits == 1) return e;
  return launch_dependent(fp4_combine_kernel<kHd, kNT>, dim3(static_cast<unsigned>(seqs), ct), dim3(256), 0, stream,
                          prm);
}

}  // namespace fp4

int fp4_choose_splits(int bs, int h_q, int h_kv, int max_seqlen, int q_len, int window, int num_sms, int num_splits) {
  if (bs < 1 || h_kv < 1 || h_q < h_kv || q_len < 1 || num_sms < 1) return 1;
  long long longest = std::max(max_seqlen, 1);
  if (window > 0) longest = std::min(longest, static_cast<long long>(window) + q_len - 1 + fp4::kTile);
  const long long tiles = (longest + fp4::kTile - 1) / fp4::kTile;
  const long long most = std::max(1LL, std::min(256LL, (tiles + fp4::kWarps - 1) / fp4::kWarps));
  if (num_splits > 0) return static_cast<int>(std::min<long long>(num_splits, most));
  int nt = 1;
  const long long ctas = static_cast<long long>(bs) * h_kv *
                         fp4::col_tiles(static_cast<int>(std::min<long long>(
                             static_cast<long long>(q_len) * (h_q / h_kv), fp4::kMaxCols)), &nt);
  const long long want = (4LL * num_sms + ctas - 1) / ctas;
  return static_cast<int>(std::max(1LL, std::min(want, most)));
}

size_t fp4_workspace_bytes(int bs, int h_q, int h_kv, int head_dim, int q_len, int splits) {
  if (bs < 1 || h_kv < 1 || h_q < h_kv || q_len < 1 || splits < 2) return 0;
  int nt = 1;
  const long long cols = static_cast<long long>(q_len) * (h_q / h_kv);
  if (cols > fp4::kMaxCols) return 0;
  const int ct = fp4::col_tiles(static_cast<int>(cols), &nt);
  const size_t slots = static_cast<size_t>(bs) * h_kv * ct * splits;
  return fp4::round_up(slots * nt * 8 * head_dim * sizeof(float), 256) +
         fp4::round_up(slots * nt * 8 * sizeof(float2), 256);
}

fp8mla_status_t fp4_decode_entry(const Fp4DecodeArgs& a, cudaStream_t stream) {
  if ((a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) || a.bs < 0 || a.h_q < 1 || a.h_kv < 1 ||
      a.h_q % a.h_kv != 0 || a.q_len < 1 || a.q_len > fp4::kMaxQLen ||
      static_cast<long long>(a.q_len) * (a.h_q / a.h_kv) > fp4::kMaxCols || a.window < 0 || a.num_blocks < 1 ||
      a.max_blocks < 1 || a.num_splits < 0 || !(a.softmax_scale > 0.f))
    return FP8MLA_ERR_INVALID_ARG;
  int page_shift = 0;
  while (page_shift < 5 && (fp4::kTile << page_shift) != a.page_size) ++page_shift;
  if (page_shift == 5) return FP8MLA_ERR_INVALID_ARG;  // 16, 32, 64, 128 or 256 keys a page
  if (a.bs == 0) return FP8MLA_OK;
  if (a.q == nullptr || a.k_cache == nullptr || a.v_cache == nullptr || a.k_block_scales == nullptr ||
      a.v_block_scales == nullptr || a.k_scale == nullptr || a.v_scale == nullptr || a.block_table == nullptr ||
      a.seqlens == nullptr || a.out == nullptr || a.lse == nullptr)
    return FP8MLA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k_cache) |
       reinterpret_cast<uintptr_t>(a.v_cache) | reinterpret_cast<uintptr_t>(a.k_block_scales) |
       reinterpret_cast<uintptr_t>(a.v_block_scales) | reinterpret_cast<uintptr_t>(a.out)) & 15u)
    return FP8MLA_ERR_INVALID_ARG;
  const long long capacity = std::min(static_cast<long long>(a.max_blocks) * a.page_size, 0x7FFFFFFFll - 256);
  int splits = fp4_choose_splits(a.bs, a.h_q, a.h_kv, static_cast<int>(capacity), a.q_len, a.window, device_sms(),
                                 a.num_splits);
  int nt = 1;
  const int ct = fp4::col_tiles(a.q_len * (a.h_q / a.h_kv), &nt);
  const size_t need = fp4_workspace_bytes(a.bs, a.h_q, a.h_kv, a.head_dim, a.q_len, splits);
  if (splits > 1) {
    if (a.workspace == nullptr || (reinterpret_cast<uintptr_t>(a.workspace) & 255u)) return FP8MLA_ERR_INVALID_ARG;
    if (a.workspace_bytes < need) return FP8MLA_ERR_WORKSPACE_TOO_SMALL;
  }
  if (static_cast<long long>(a.bs) * a.h_kv * splits > 0x7FFFFFFFll) return FP8MLA_ERR_INVALID_ARG;
  fp4::Params p;
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = static_cast<const uint8_t*>(a.k_cache);
  p.v = static_cast<const uint8_t*>(a.v_cache);
  p.ks = static_cast<const uint8_t*>(a.k_block_scales);
  p.vs = static_cast<const uint8_t*>(a.v_block_scales);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.block_table = a.block_table;
  p.seqlens = a.seqlens;
  p.spec_mask = a.spec_mask;
  p.sinks = a.sinks;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  const size_t slots = static_cast<size_t>(a.bs) * a.h_kv * ct * splits;
  p.ws_o = static_cast<float4*>(a.workspace);
  p.ws_ml = splits > 1 ? reinterpret_cast<float2*>(static_cast<char*>(a.workspace) +
                                                   fp4::round_up(slots * nt * 8 * a.head_dim * sizeof(float), 256))
                       : nullptr;
  p.num_blocks = a.num_blocks;
  p.max_blocks = a.max_blocks;
  p.h_q = a.h_q;
  p.h_kv = a.h_kv;
  p.group = a.h_q / a.h_kv;
  p.splits = splits;
  p.q_len = a.q_len;
  p.window = a.window;
  p.page_shift = page_shift;
  p.softmax_scale = a.softmax_scale;
  const int seqs = a.bs * a.h_kv;
  cudaError_t e;
  switch (a.head_dim + nt) {
    case 64 + 1: e = fp4::launch<64, 1>(p, seqs, ct, stream); break;
    case 64 + 2: e = fp4::launch<64, 2>(p, seqs, ct, stream); break;
    case 128 + 1: e = fp4::launch<128, 1>(p, seqs, ct, stream); break;
    case 128 + 2: e = fp4::launch<128, 2>(p, seqs, ct, stream); break;
    case 256 + 1: e = fp4::launch<256, 1>(p, seqs, ct, stream); break;
    default: e = fp4::launch<256, 2>(p, seqs, ct, stream); break;
  }
  return e == cudaSuccess ? FP8MLA_OK : FP8MLA_ERR_CUDA;
}

uint32_t fp4_read_and_clear_status() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_status_fp4, sizeof(v));
  cudaMemcpyToSymbol(g_status_fp4, &z, sizeof(z));
  return v;
}

}  // namespace fp8mla
