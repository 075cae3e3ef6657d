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
// the tensor rate.  At the copy bandwidth an SM has about six cycles per key of
// 256 values, and every code has to become a 16-bit operand in that time: a
// conversion and a multiplication for two codes, which issue at half rate, so
// the instructions that make operands and the memory are both close to their
// limit.  Measured (32 contexts of 1024 to 16384 keys, 8 KV heads, head_dim
// 128, group 4): 64.4 us a call, 0.75 of the measured copy bandwidth (head_dim
// 256, 4 KV heads 0.77); leaving the loads out would save 1.5 us, the scale
// multiplications 9.5, the conversions of V 10.  Sixteen columns double the
// products and leave twelve warps less to hide with: four-token blocks under a
// 4096-key window 47.5 us, 0.44, without the window 0.55.  More columns convert
// K and V once for every sixteen: 32 columns 166 us, 0.30.  head_dim 64 halves
// the bytes of a tile but not its overhead: the batch 0.55, three contexts of
// 50k to 131k keys 18.8 us, 0.35, of which 8 are the lengths' sums, the first
// tiles, the merge and two launches.
//
// Design:
//   * A warp works alone on tiles of 16 keys: it fetches them into its own
//     ring in shared memory by 16-byte cp.async, two to three steps ahead,
//     keeps its own running maximum, sum and accumulator, and meets the CTA's
//     other warps only at the end of a piece.
//   * Codes go from shared memory to registers to the product's A fragment:
//     S^T = K Q^T (M = 16 keys, N = 8 columns, K = head_dim) and
//     O^T = V^T P^T (M = 16 dims, N = 8 columns, K = 16 keys) as register-
//     fragment products, for which a code is converted in the lane that needs
//     it.  A tensor-memory product would need the expanded 16-bit tile written
//     to shared or tensor memory first: 512 bytes a key against the 128 that
//     an SM can store in a cycle, four of the six cycles a key has.  (The
//     block-scaled 4-bit product takes neither Q and P in 16 bits nor V, whose
//     scales run along the dims and not along the contraction.)
//   * The order of the contraction is free, so each lane takes contiguous
//     bytes: lane (g, t) of K row g holds dims [t hd/4, (t + 1) hd/4), and Q's
//     fragment is laid out to match; of V, lane (g, t) holds the hd/8 dims
//     from g hd/8 of keys t, t + 4, t + 8, t + 12.  A code's byte holds two
//     neighbouring dims; for V the operand pairs two keys instead, formed on
//     the nibbles (a shift and a select for eight codes).  Fragment rows g and
//     g + 8 of S^T are keys (g / 2) + 4 (g % 2) and that plus 8, so that the
//     same pairs come out of the probabilities' transpose.
//   * E2M1 * E4M3 has at most six significant bits and lies in f16's range
//     (subnormals included), so K and V operands are exact.  Q is bf16 times
//     a power of two per column, which puts its largest value into [2^14,
//     2^15): exact in f16 from 2^-31 of that value on, smaller ones off by at
//     most 2^-39 of it (more where the largest is below 2^-86).  P is rounded
//     to f16 (half a step: 2^-11) and its sum is not: a second f16 term of P
//     would double the products to take 1 % off the output's error, which is
//     bf16's rounding.  Sums are f32.
//   * A column's reference is 7 (log2) below the largest score it was taken
//     from and moves only when a score passes it by more than 15: P stays
//     within f16 (2^15), weights down to 2^-21 of the largest keep f16's
//     relative precision, and most tiles need no shuffle.  Scores past 2^22,
//     where the rounding of such a reference would show in the weights, are
//     taken from the largest score itself, which moves with every larger one.
//   * The work -- every (sequence, KV head)'s tiles in one line -- is cut into
//     equal pieces, one per CTA that fits on the GPU at once: lengths are known
//     on the device only, so each CTA sums them itself.  A piece holds the end
//     of one sequence, whole ones, and the beginning of another; whole ones are
//     written at once, the others' partial states merged by a second kernel.
//     Few sequences of short contexts, for which two launches are too many, go
//     uncut, to one CTA of up to sixteen warps each or to a cluster of two to
//     eight, whose CTAs take their tiles in turn and merge over the cluster's
//     shared memory (one context of 777 keys, 8 KV heads: 6.8 us a call; one
//     CTA each 8.2; through pieces, where the block table holds more keys than
//     the rule allows, 8.4 instead of 7.2).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "gqa_fp4.h"
#include "host_util.h"

namespace fp8mla {

__device__ uint32_t g_status_fp4;

namespace fp4 {

constexpr int kTile = 16;       // keys of a tile
constexpr int kMaxQLen = 16;
constexpr int kMaxCols = 128;   // q_len * (h_q / h_kv)
constexpr int kMaxLine = 1024;  // sequences whose lengths a CTA sums
constexpr int kMaxCluster = 8;  // CTAs that share a sequence and merge in shared memory
constexpr int kMinTiles = 8;    // places of a piece, where there are fewer than the GPU takes at once
constexpr int kFixed = 32;      // what a sequence costs a CTA beside its tiles, in tiles: fill, drain and merge
constexpr int kShort = 96;      // tiles up to which a sequence is not cut (200 of 94 tiles: 16.7 us, cut 18.1)
constexpr float kBelow = 7.f;   // a reference lies this far below the largest score (log2) ...
constexpr float kTau = 15.f;    // ... and moves when a score is this far above it
constexpr float kFar = 4194304.f;  // 2^22 (log2): where a reference rounded to float32 is off by up to a quarter

// Warps of a CTA, CTAs of an SM, tiles a warp takes at a time, and stages of its ring.  Throughput: twelve warps of up
// to 168 registers on an SM (eight at head_dim 256, twice the accumulators), in small CTAs, so that a piece's fill and
// merge hide behind the other CTAs' loops (the 32-context batch: 8 warps x 2 CTAs 78 us, 4 x 4 70, 4 x 3 with two
// tiles at a time 63): kFillingCtas, for pieces, and kWholeCtas, for whole sequences and asked-for shards, without the
// code for pieces (456 sequences of one tile 5.3 us, with it 6.2).  kNarrowCtas: two warps, for more sequences of short
// contexts than there are places for those.  kWideCtas: an SM's warps in one CTA, alone or in a cluster, for few
// sequences of short contexts, where a warp's few tiles in a row are what takes the time.
enum Ctas { kFillingCtas, kWholeCtas, kNarrowCtas, kWideCtas };
template <int kHd, int kNT, Ctas kCtas>
struct Shape {
  static constexpr bool kWide = kCtas == kWideCtas, kNarrow = kCtas == kNarrowCtas;
  static constexpr int kWarps = kWide ? (kHd == 256 ? 8 : (kNT == 1 ? 16 : 12)) : (kNarrow ? 2 : 4);
  static constexpr int kPerSm =
      kWide ? 1 : (kHd == 256 ? 2 : (kHd == 64 && kNT == 1 && kCtas != kFillingCtas ? 4 : 3)) * (kNarrow ? 2 : 1);
  static constexpr int kU = kWide || kHd == 256 || kNT == 2 ? 1 : 2;
  static constexpr int kStages = kU == 2 ? 3 : 4;
};

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
  float4* ws_o;    // [slot][NT * hd / 16][32 lanes] fragments
  float2* ws_ml;   // [slot][NT * 8]
  int2* ws_span;   // [bs * h_kv]: first and last piece of a (sequence, KV head) (balanced only)
  int num_blocks, max_blocks, bs, h_q, h_kv, group, q_len, window;
  int splits;      // shards of every sequence, one CTA each (1: no merge), 0: balanced pieces; wide: CTAs of a cluster
  int units;       // balanced: pieces there may be
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

// e with amax * 2^-e in [2^14, 2^15); not below -100 (2^-e has to be a float: smaller queries lose bits, down to 0).
__device__ __forceinline__ int q_exponent(float amax) {
  const int expo = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFFu);
  return min(max(-100, expo - 127 - 14), 113);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Loads that stay where they are written, before the waits that follow.
__device__ __forceinline__ uint4 ldg_now(const uint4* p) {
  uint4 x;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
  return x;
}

__device__ __forceinline__ int32_t ldg_now(const int32_t* p) {
  int32_t x;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ int32_t ldg_now(const uint8_t* p) {
  int32_t x;
  asm volatile("ld.global.u8 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kFar; }

// finish_row, with a NaN sum passed on (finish_row takes one for no key at all).
__device__ __forceinline__ void finish(float m, float l, float sink, float v_scale, float* f, float* lse) {
  finish_row(m, l, sink, v_scale, f, lse);
  if (l != l) *f = *lse = l;
}

// Keys that the call reads of a sequence of length s_k: none, and a status bit, where that is negative or longer
// than the block table; and the first tile that any token's window reaches.
__device__ __forceinline__ int checked_len(const Params& prm, int s_k) {
  const int page = kTile << prm.page_shift;
  if (s_k >= 0 && ((static_cast<long long>(s_k) + page - 1) >> (4 + prm.page_shift)) <= prm.max_blocks) return s_k;
  atomicOr(&g_status_fp4, FP8MLA_DEV_BAD_SEQLEN);
  return 0;
}
__device__ __forceinline__ int first_tile(const Params& prm, int s_k) {
  return prm.window > 0 ? max(0, s_k - prm.q_len - prm.window + 1) / kTile : 0;
}
__device__ __forceinline__ int tiles_of(const Params& prm, int s_k) {
  return max(0, (s_k + kTile - 1) / kTile - first_tile(prm, s_k));
}

template <int kHd, int kNT, Ctas kCtas>
__global__ void __launch_bounds__(Shape<kHd, kNT, kCtas>::kWarps * 32, Shape<kHd, kNT, kCtas>::kPerSm)
    fp4_decode_kernel(const __grid_constant__ Params prm) {
  using L = Lay<kHd>;
  using S = Shape<kHd, kNT, kCtas>;
  constexpr bool kWide = S::kWide, kPieces = kCtas == kFillingCtas, kShards = kCtas == kWholeCtas;
  constexpr int kWarps = S::kWarps, kU = S::kU, kStages = S::kStages;
  constexpr int kStage = kU * L::kBytes;
  constexpr int kSteps = kHd / 16;     // products of a tile, for K and for V
  constexpr int kKWords = kHd / 32;    // 32-bit words of a lane's part of a K row
  constexpr int kVWords = kHd / 64;    // of a lane's part of a V row
  constexpr int kCopies = L::kChunks / 32;
  extern __shared__ __align__(128) uint8_t smem[];  // a 512-byte copy of a warp covers whole 128-byte lines
  __shared__ uint32_t s_vis[kMaxQLen], s_any;
  __shared__ float s_m[kWarps][kNT * 8], s_l[kWarps][kNT * 8];
  __shared__ uint4 s_q[kNT][kSteps / 2][32];  // Q's fragments of two products a lane
  __shared__ float s_cq[kNT * 8];             // score to log2 units, then a finished row's factor
  __shared__ float s_sink[kNT * 8], s_vscale;
  __shared__ float2 s_ml[kNT * 8];                 // this CTA's maxima and sums, for its cluster
  __shared__ float s_weight[kMaxCluster][kNT * 8];  // what the cluster's states are multiplied by
  __shared__ int64_t s_row[kNT * 8];
  __shared__ int s_tok[kNT * 8];              // a column's token
  __shared__ int s_line[kPieces ? kMaxLine + 1 : 1];
  __shared__ int s_part[2][kWarps];

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  const int col0 = blockIdx.y * (kNT * 8);
  const int ncols = min(prm.q_len * prm.group - col0, kNT * 8);
  const int page = kTile << prm.page_shift;

  griddep_wait();

  // ---- this CTA's stretch [cur, end) of a line on which a sequence's KV heads lie one after the other, each
  // taking kFixed places and then one for every tile
  int cur = 0, end = 1;
  const int unit = blockIdx.x;
  if (kPieces) {
    // prefix sums of the sequences' places (of one KV head), a CTA's width of sequences at a time
    constexpr int kThreads = kWarps * 32, kRuns = (kMaxLine + kThreads - 1) / kThreads;
    int len[kRuns];
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const int b = i * kThreads + threadIdx.x;
      len[i] = b < prm.bs ? __ldg(prm.seqlens + b) : 0;
    }
    int before = 0;
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      if (i * kThreads >= prm.bs) break;
      const int b = i * kThreads + threadIdx.x;
      const int tiles = tiles_of(prm, checked_len(prm, len[i]));
      const int places = tiles > 0 ? tiles + kFixed : 0;
      if (tiles == 0 && b < prm.bs && unit == 0 && blockIdx.y == 0)  // nothing to attend to: the merge writes it
        for (int h = 0; h < prm.h_kv; ++h) prm.ws_span[b * prm.h_kv + h] = make_int2(1, 0);
      int inc = places;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      if (lane == 31) s_part[i & 1][warp] = inc;
      __syncthreads();
      int start = before;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) start += s_part[i & 1][w];
        before += s_part[i & 1][w];
      }
      if (b < prm.bs) s_line[b] = start + inc - places;
    }
    if (threadIdx.x == 0) s_line[prm.bs] = before;
    __syncthreads();
    const int work = s_line[prm.bs] * prm.h_kv;
    const int pieces = max(1, min(prm.units, work / kMinTiles));
    if (unit >= pieces) return;
    const int each = work / pieces, rest = work - each * pieces;  // cut u at floor(work u / pieces)
    cur = each * unit + rest * unit / pieces;
    end = each * (unit + 1) + rest * (unit + 1) / pieces;
  }

  // A warp's first tile of a segment, and how far it is to its next.  The CTAs of a cluster take turns.
  const int mine = (kWide ? unit % prm.splits * kWarps : 0) * kU + warp * kU;
  const int stride = kWarps * kU * (kWide ? prm.splits : 1);

  const int c_lane = lane * 16;  // this lane's bytes of a code tile
  uint32_t kdst[kCopies], vdst[kCopies];  // and where they go in a stage
  const uint32_t ring = smem_u32(smem) + warp * (kStages * kStage);
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int c = lane + 32 * i, r = c / (L::kRow / 16), cc = c % (L::kRow / 16);
    kdst[i] = L::kK + k_place<kHd>(r, cc);
    vdst[i] = L::kV + v_place<kHd>(r, cc);
  }
  const bool sc_lane = lane < 2 * L::kSChunks;
  const bool sc_v = lane >= L::kSChunks;
  const uint8_t* sc_base = (sc_v ? prm.vs : prm.ks) + (sc_v ? lane - L::kSChunks : lane) * 16;
  const uint32_t sc_dst = (sc_v ? L::kVs + (lane - L::kSChunks) * 16 : L::kKs + lane * 16);
  const uint8_t* k_base = prm.k + c_lane;
  const uint8_t* v_base = prm.v + c_lane;
  const int r0 = (g >> 1) + 4 * (g & 1);  // keys of fragment rows g and g + 8
  const int r1 = r0 + 8;
  const float c0 = prm.softmax_scale * kLog2e * __ldg(prm.k_scale);
  if (kWide && threadIdx.x == 0) s_vscale = __ldg(prm.v_scale);

  while (cur < end) {
    // ---- the segment: tiles [t0, t1) of one (sequence, KV head)
    int b, kvh, t0, t1, s_k;
    long long slot = -1;  // where its partial state goes, or -1: the rows are finished here
    if (kPieces) {
      const int at = cur / prm.h_kv;
      int lo = 0, hi = prm.bs;  // s_line[lo] <= at < s_line[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (s_line[mid] <= at) lo = mid;
        else hi = mid;
      }
      b = lo;
      const int places = s_line[b + 1] - s_line[b];
      int off = cur - s_line[b] * prm.h_kv;
      kvh = off / places;
      off -= kvh * places;
      const int first = max(0, off - kFixed);
      const int stop = min(end - cur + off, places);
      const int last = max(0, stop - kFixed), tiles = places - kFixed;
      cur += stop - off;
      if (first == last) continue;  // the cut fell into the places before the first tile
      if (last - first < tiles)
        slot = (static_cast<long long>(blockIdx.y) * prm.units + unit) * 2 + (first == 0 ? 1 : 0);
      if (threadIdx.x == 0 && blockIdx.y == 0) {
        if (first == 0) prm.ws_span[b * prm.h_kv + kvh].x = unit;
        if (last == tiles) prm.ws_span[b * prm.h_kv + kvh].y = unit;
      }
      t0 = first;
      t1 = last;
    } else {
      const int seq = (kShards || kWide) && prm.splits > 1 ? unit / prm.splits : unit;
      b = seq / prm.h_kv;
      kvh = seq - b * prm.h_kv;
      if (kShards && prm.splits > 1) slot = static_cast<long long>(blockIdx.y) * gridDim.x + unit;
      cur = end;
    }
    auto lengths = [&]() {
      if (kPieces) {
        s_k = __ldg(prm.seqlens + b);
        t0 += first_tile(prm, s_k);
        t1 += first_tile(prm, s_k);
      } else {
        s_k = checked_len(prm, __ldg(prm.seqlens + b));
        const int tiles = tiles_of(prm, s_k);
        t0 = first_tile(prm, s_k);
        t1 = t0 + tiles;
        if (kShards && prm.splits > 1) {  // (the divisions would cost a short call 0.4 us)
          const int split = unit % prm.splits;
          t1 = t0 + static_cast<int>(static_cast<long long>(split + 1) * tiles / prm.splits);
          t0 += static_cast<int>(static_cast<long long>(split) * tiles / prm.splits);
        }
      }
    };
    const int32_t* bt_row = prm.block_table + static_cast<size_t>(b) * prm.max_blocks;
    // Where a call's latency is what counts (wide), what does not depend on the sequence's length is asked for before
    // it has come: the first tiles' places in the block table (without a window they are known), Q, sinks and mask.
    int32_t guessed = 0;
    bool guess = false;
    if constexpr (kWide) {
      guess = prm.window == 0;
      const int at = (lane / kU * stride + mine + lane % kU) >> prm.page_shift;
      if (guess && at < prm.max_blocks) guessed = ldg_now(bt_row + at);
    } else {
      lengths();
    }
    // Q's values: lane (g, t) of warp n takes dims [t hd/4, (t + 1) hd/4) of column 8 n + g; and the column's sink
    uint4 qx[kSteps / 2];
    float sink = kNegInf;
    if (warp < kNT) {
      const int c = warp * 8 + g, col = col0 + c, token = col / prm.group;
      const int hq = kvh * prm.group + col - token * prm.group;
      const uint4* src = reinterpret_cast<const uint4*>(
          prm.q + ((static_cast<size_t>(b) * prm.q_len + token) * prm.h_q + hq) * kHd + t * (kHd / 4));
#pragma unroll
      for (int j = 0; j < kSteps / 2; ++j) qx[j] = c < ncols ? ldg_now(src + j) : make_uint4(0, 0, 0, 0);
      if (kWide && prm.sinks != nullptr && c < ncols)
        sink = __int_as_float(ldg_now(reinterpret_cast<const int32_t*>(prm.sinks) + hq));
    }
    // The speculative block's mask, by the last warp: lane (r, c) of half-warp r takes byte c of rows r, r + 2, ...
    int32_t seen[kMaxQLen / 2];
    auto ask_mask = [&]() {
      const uint8_t* rows = prm.spec_mask + static_cast<size_t>(b) * prm.q_len * prm.q_len;
#pragma unroll
      for (int i = 0; i < kMaxQLen / 2; ++i) {
        const int r = 2 * i + lane / 16, c = lane % 16;
        seen[i] = r < prm.q_len && c < prm.q_len ? ldg_now(rows + r * prm.q_len + c) : 0;
      }
    };
    if (kWide && prm.spec_mask != nullptr && warp == kWarps - 1) ask_mask();
    if constexpr (kWide) lengths();
    const int start = s_k - prm.q_len;  // position of the block's first token
    const int tok_lo = prm.q_len > 1 ? col0 / prm.group : 0;  // the first token of this CTA's columns
    const int k_lo = prm.window > 0 ? max(0, start + tok_lo - prm.window + 1) : 0;
    const int mine0 = t0 + mine;  // this warp's tiles: kU from here, kU more `stride` later, ...
    const int n_mine = t1 > mine0 ? (t1 - mine0 + stride - 1) / stride : 0;

    // Entries of the block table (as the tile's first row in the cache), 32 tiles of this warp at a time.
    uint32_t entry = 0;
    const uint32_t block_rows = prm.h_kv * page;
    auto fetch_entries = [&](int i0, auto first) {
      const int tile = mine0 + (i0 + lane / kU) * stride + lane % kU;
      entry = 0;
      if (tile < t1) {
        int blk = decltype(first)::value && guess ? guessed : __ldg(bt_row + (tile >> prm.page_shift));
        if (blk < 0 || blk >= prm.num_blocks) {
          atomicOr(&g_status_fp4, FP8MLA_DEV_BAD_PAGE);
          blk = 0;
        }
        entry = blk * block_rows + kvh * page + (tile & ((1 << prm.page_shift) - 1)) * kTile;
      }
    };
    uint32_t put = ring;  // the stage that is filled next
    auto issue = [&](int i, auto first) {
      if (i < n_mine) {
        if (i % (32 / kU) == 0) fetch_entries(i, first);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const uint32_t row = __shfl_sync(0xffffffffu, entry, i % (32 / kU) * kU + u);
          if (u > 0 && mine0 + i * stride + u >= t1) break;  // past the segment's end: an old tile stays there
          const uint8_t* ksrc = k_base + static_cast<uint64_t>(row) * L::kRow;
          const uint8_t* vsrc = v_base + static_cast<uint64_t>(row) * L::kRow;
#pragma unroll
          for (int j = 0; j < kCopies; ++j) {
            cp_async16(put + kdst[j] + u * L::kBytes, ksrc + 512 * j, 16u);
            cp_async16(put + vdst[j] + u * L::kBytes, vsrc + 512 * j, 16u);
          }
          if (sc_lane)
            cp_async16(put + sc_dst + u * L::kBytes, sc_base + static_cast<uint64_t>(row) * L::kSRow, 16u);
        }
        put += kStage;
        if (put == ring + kStages * kStage) put = ring;
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, std::true_type{});

    // Which keys of the speculative block its token i sees: its mask row, or those up to itself; and which keys any
    // token of this CTA's columns sees.
    if (warp == kWarps - 1) {
      uint32_t bits = (2u << lane) - 1u;
      if (!kWide && prm.spec_mask != nullptr) {
        const uint8_t* row = prm.spec_mask + (static_cast<size_t>(b) * prm.q_len + lane) * prm.q_len;
        bits = 0;
        if (lane < prm.q_len)
          for (int c = 0; c < prm.q_len; ++c)
            if (__ldg(row + c)) bits |= 1u << c;
      } else if (prm.spec_mask != nullptr) {
#pragma unroll
        for (int i = 0; i < kMaxQLen / 2; ++i) {
          const uint32_t two = __ballot_sync(0xffffffffu, seen[i] != 0);
          if (lane / 2 == i) bits = lane & 1 ? two >> 16 : two & 0xFFFFu;
        }
      }
      if (lane < prm.q_len) s_vis[lane] = bits;
      const uint32_t near = prm.window == 0 || lane < prm.window ? ~0u : ~0u << (lane - prm.window + 1);
      const bool ours = lane >= tok_lo && lane <= (col0 + ncols - 1) / prm.group;
      const uint32_t any = __reduce_or_sync(0xffffffffu, ours ? bits & near : 0u);
      if (lane == 0) s_any = any;
    }
    if (warp < kNT) {  // Q's fragments, as f16 with a power of two out
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < kSteps / 2; ++j) {
        amax = fmax3(amax, fmaxf(fabsf(bf16_lo(qx[j].x)), fabsf(bf16_hi(qx[j].x))),
                     fmaxf(fabsf(bf16_lo(qx[j].y)), fabsf(bf16_hi(qx[j].y))));
        amax = fmax3(amax, fmaxf(fabsf(bf16_lo(qx[j].z)), fabsf(bf16_hi(qx[j].z))),
                     fmaxf(fabsf(bf16_lo(qx[j].w)), fabsf(bf16_hi(qx[j].w))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = q_exponent(amax);
      const float inv = exp2i(-e);
      auto scaled = [&](uint32_t w) { return pack_f16x2(bf16_lo(w) * inv, bf16_hi(w) * inv); };
#pragma unroll
      for (int j = 0; j < kSteps / 2; ++j)
        s_q[warp][j][lane] = make_uint4(scaled(qx[j].x), scaled(qx[j].y), scaled(qx[j].z), scaled(qx[j].w));
      if (t == 0) {
        s_cq[warp * 8 + g] = c0 * exp2i(e);
        s_tok[warp * 8 + g] = min((col0 + warp * 8 + g) / prm.group, prm.q_len - 1);
        if (kWide) s_sink[warp * 8 + g] = sink;
      }
    }
    __syncthreads();  // s_vis, s_q, s_cq
    float cq[kNT][2];
#pragma unroll
    for (int n = 0; n < kNT; ++n) cq[n][0] = s_cq[n * 8 + 2 * t], cq[n][1] = s_cq[n * 8 + 2 * t + 1];

    // Tiles whose keys every column sees: before the speculative block (or, for one token, the end) and, with a
    // window, from the last token's first key on.
    const int keys_end = min(s_k, t1 * kTile);  // the segment's
    int full_end = min(keys_end, prm.q_len == 1 && prm.spec_mask == nullptr ? s_k : max(0, start));
    const int full_lo = prm.window > 0 ? max(0, s_k - prm.window) : 0;

    // u = score * cq (log2 units); p = 2^(u + neg_m); a score above `limit` moves the reference.  Past kFar the
    // rounding of neg_m would take p out of f16's range (from 2^28 on by more than 2^8), so there the reference is
    // the largest score itself, held in `limit`: p = 2^((score - limit) cq + kBelow), and neg_m is for the merge.  The
    // path for masks has the code for this; a warp that meets such a score takes it from there on (full_end = -1).
    float o[kNT][kSteps][4];
    float neg_m[kNT][2], limit[kNT][2], l[kNT][2];
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[n][j][k] = 0.f;
      neg_m[n][0] = neg_m[n][1] = 0.f;
      limit[n][0] = limit[n][1] = kNegInf;  // no key seen yet
      l[n][0] = l[n][1] = 0.f;
    }

    // eight columns' fragments stay in registers, sixteen are read for every tile
    constexpr bool kQRegs = kNT == 1 && kHd <= 128 && !kWide;
    uint4 qr[kQRegs ? kNT : 1][kQRegs ? kSteps / 2 : 1];
    if constexpr (kQRegs) {
#pragma unroll
      for (int w = 0; w < kSteps / 2; ++w) qr[0][w] = s_q[0][w][lane];
    }

    // S^T = K Q^T of the tile at st
    auto scores = [&](const uint8_t* st, float (&s)[kNT][4]) {
#pragma unroll
      for (int n = 0; n < kNT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
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
          uint4 q;
          if constexpr (kQRegs) q = qr[n][w];
          else q = s_q[n][w][lane];
          mma_f16_16x8x16(s[n], x[0], y[0], x[1], y[1], q.x, q.y);
          mma_f16_16x8x16(s[n], x[2], y[2], x[3], y[3], q.z, q.w);
        }
      }
    };

    auto sees = [&](int p, int c) {  // whether key p is for column c
      const int ti = s_tok[c];
      const int c_blk = p - start;
      return p < keys_end && (c_blk < 0 || ((s_vis[ti] >> c_blk) & 1u)) && (prm.window == 0 || ti - c_blk < prm.window);
    };

    const uint8_t* st = smem + warp * (kStages * kStage);
    const uint8_t* const st_end = st + kStages * kStage;
    int tok0 = mine0 * kTile;
    auto tiles = [&](auto masked) {
      constexpr bool kMasked = decltype(masked)::value;
      float s[kU][kNT][4];
#pragma unroll
      for (int u = 0; u < kU; ++u) scores(st + u * L::kBytes, s[u]);
      uint32_t hidden = 0;  // bit 8 u + 4 n + k: key k / 2 of tile u is not for column k % 2 of column tile n
      if constexpr (kMasked) {
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
          for (int n = 0; n < kNT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (!sees(tok0 + u * kTile + (k < 2 ? r0 : r1), n * 8 + 2 * t + (k & 1))) {
                s[u][n][k] = kNegInf;
                hidden |= 1u << (8 * u + 4 * n + k);
              }
            }
      }
      float top[kNT][2];
      bool grow = false;
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          top[n][k] = fmaxf(s[0][n][k], s[0][n][k + 2]);
          if constexpr (kU == 2) top[n][k] = fmax3(top[n][k], s[kU - 1][n][k], s[kU - 1][n][k + 2]);
          grow |= !(top[n][k] <= limit[n][k]);  // (a NaN score moves it, and its column stays NaN)
        }
      if (__any_sync(0xffffffffu, grow)) {
        if constexpr (!kMasked) {
          bool far = false;
#pragma unroll
          for (int n = 0; n < kNT; ++n)
            far |= is_far(top[n][0] * cq[n][0] - kBelow) || is_far(top[n][1] * cq[n][1] - kBelow);
          if (__any_sync(0xffffffffu, far)) {
            full_end = -1;
            return false;
          }
        }
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mx = top[n][k];
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (!(mx <= limit[n][k])) {
              const float m = mx * cq[n][k] - kBelow;
              float down = -neg_m[n][k] - m;
              if (kMasked && is_far(m) && is_far(neg_m[n][k])) down = (limit[n][k] - mx) * cq[n][k];
              const float alpha = limit[n][k] == kNegInf ? 0.f : ex2_approx(down);
              neg_m[n][k] = -m;
              limit[n][k] = kMasked && is_far(m) ? mx : (m + kTau) / cq[n][k];
              l[n][k] *= alpha;
#pragma unroll
              for (int j = 0; j < kSteps; ++j) {
                o[n][j][k] *= alpha;
                o[n][j][k + 2] *= alpha;
              }
            }
          }
        if constexpr (kMasked) {
          bool far = false;
#pragma unroll
          for (int n = 0; n < kNT; ++n) far |= is_far(neg_m[n][0]) || is_far(neg_m[n][1]);
          if (__any_sync(0xffffffffu, far)) full_end = -1;
        }
      }
      uint32_t pf[kU][kNT][2];
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          float p[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) p[k] = fmaf(s[u][n][k], cq[n][k & 1], neg_m[n][k & 1]);
          if constexpr (kMasked) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (is_far(neg_m[n][k & 1])) p[k] = fmaf(s[u][n][k] - limit[n][k & 1], cq[n][k & 1], kBelow);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) p[k] = ex2_approx(p[k]);
          if constexpr (kMasked) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if ((hidden >> (8 * u + 4 * n + k)) & 1u) p[k] = 0.f;
          }
          l[n][0] += p[0] + p[2];
          l[n][1] += p[1] + p[3];
          pf[u][n][0] = movmatrix_trans(pack_f16x2(p[0], p[1]));
          pf[u][n][1] = movmatrix_trans(pack_f16x2(p[2], p[3]));
        }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint8_t* sv = st + u * L::kBytes;
        uint32_t v[4][kVWords];
        uint32_t sc[4];  // scale bytes of the lane's dims, keys t, t + 4, t + 8, t + 12
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = t + 4 * k;
          if constexpr (kHd == 64) {
            v[k][0] = *reinterpret_cast<const uint32_t*>(sv + L::kV + v_place<kHd>(r, g >> 2) + (g & 3) * 4);
            sc[k] = sv[L::kVs + r * 4 + (g >> 1)];
          } else if constexpr (kHd == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(sv + L::kV + v_place<kHd>(r, g >> 1) + (g & 1) * 8);
            v[k][0] = x.x, v[k][1] = x.y;
            sc[k] = sv[L::kVs + r * 8 + g];
          } else {
            const uint4 x = *reinterpret_cast<const uint4*>(sv + L::kV + v_place<kHd>(r, g));
            v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
            sc[k] = *reinterpret_cast<const uint16_t*>(sv + L::kVs + r * 16 + 2 * g);
          }
        }
        // A weight of zero does not hide a NaN, so a key that no column sees has its scales zeroed, whatever they are,
        // and so has a NaN scale; the columns that see that one get their NaN after the product.
        bool nans = false;
        if constexpr (kMasked) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int p = tok0 + u * kTile + t + 4 * k;
            if (p >= keys_end || p < k_lo || (p >= start && !((s_any >> (p - start)) & 1u))) sc[k] = 0;
#pragma unroll
            for (uint32_t m = 0x7Fu; m <= (kHd == 256 ? 0x7F00u : 0x7Fu); m <<= 8)
              if ((sc[k] & m) == m) sc[k] &= ~(m | (m << 1)), nans = true;
          }
          nans = __any_sync(0xffffffffu, nans);
        }
#pragma unroll
        for (int w = 0; w < kVWords; ++w) {
          uint32_t s01, s23;  // scale bytes of two keys, one beside the other
          if constexpr (kHd == 256) {
            s01 = prmt(sc[0], sc[1], w < 2 ? 0x0040 : 0x0051);
            s23 = prmt(sc[2], sc[3], w < 2 ? 0x0040 : 0x0051);
          } else {
            s01 = sc[0] | (sc[1] << 8);
            s23 = sc[2] | (sc[3] << 8);
          }
          const uint32_t sab = e4m3x2_to_f16x2(s01), scd = e4m3x2_to_f16x2(s23);
          constexpr uint32_t kLow = 0x0F0F0F0Fu;
          uint32_t x[4], y[4], z[4], h[4];
          e2m1x8_to_f16x2((v[0][w] & kLow) | ((v[1][w] << 4) & ~kLow), x);
          e2m1x8_to_f16x2(((v[0][w] >> 4) & kLow) | (v[1][w] & ~kLow), y);
          e2m1x8_to_f16x2((v[2][w] & kLow) | ((v[3][w] << 4) & ~kLow), z);
          e2m1x8_to_f16x2(((v[2][w] >> 4) & kLow) | (v[3][w] & ~kLow), h);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a0 = mul_f16x2(x[k], sab), a1 = mul_f16x2(y[k], sab);
            const uint32_t a2 = mul_f16x2(z[k], scd), a3 = mul_f16x2(h[k], scd);
#pragma unroll
            for (int n = 0; n < kNT; ++n) mma_f16_16x8x16(o[n][4 * w + k], a0, a1, a2, a3, pf[u][n][0], pf[u][n][1]);
          }
        }
        if constexpr (kMasked) {
          if (nans) {
            for (int r = 0; r < kTile; ++r) {
#pragma unroll
              for (int w = 0; w < (kHd == 256 ? 2 : 1); ++w) {
                const int block = kHd == 64 ? g >> 1 : (kHd == 128 ? g : 2 * g + w);
                if ((sv[L::kVs + r * (kHd / 16) + block] & 0x7F) != 0x7F) continue;
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    if (!sees(tok0 + u * kTile + r, n * 8 + 2 * t + k)) continue;
                    constexpr int kOf = kHd == 256 ? kSteps / 2 : kSteps;  // steps of a block's dims
#pragma unroll
                    for (int j = 0; j < kOf; ++j)
                      o[n][w * kOf + j][k] = o[n][w * kOf + j][k + 2] = __int_as_float(0x7FFFFFFF);
                  }
              }
            }
          }
        }
      }
      st += kStage;
      if (st == st_end) st -= kStages * kStage;
      tok0 += stride * kTile;
      return true;
    };
    for (int i = 0; i < n_mine; ++i) {
      cp_async_wait_group<kStages - 2>();
      __syncwarp();
      issue(i + kStages - 1, std::false_type{});
      if (tok0 + kU * kTile > full_end || tok0 < full_lo || !tiles(std::false_type{})) tiles(std::true_type{});
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
        if (g == 0) {
          s_m[warp][n * 8 + 2 * t + k] = limit[n][k] == kNegInf ? kNegInf : -neg_m[n][k];
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
        f[k] = limit[n][k] == kNegInf ? 0.f : ex2_approx(-neg_m[n][k] - mx);
      }
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
        part[((warp * kNT + n) * kSteps + j) * 32 + lane] =
            make_float4(o[n][j][0] * f[0], o[n][j][1] * f[1], o[n][j][2] * f[0], o[n][j][3] * f[1]);
    }
    if (threadIdx.x < kNT * 8) {  // a column's end: its sums, its row, and what its values are multiplied by
      const int c = threadIdx.x;
      float mx = kNegInf, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][c]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        sum += s_m[w][c] == kNegInf ? 0.f : s_l[w][c] * ex2_approx(s_m[w][c] - (mx == kNegInf ? 0.f : mx));
      if ((kPieces || kShards) && slot >= 0) {
        prm.ws_ml[slot * (kNT * 8) + c] = make_float2(mx, sum);
      } else if (kWide && prm.splits > 1) {
        s_ml[c] = make_float2(mx, sum);
      } else if (c < ncols) {
        const int col = col0 + c, token = col / prm.group, hq = kvh * prm.group + col - token * prm.group;
        const int64_t row = (static_cast<int64_t>(b) * prm.q_len + token) * prm.h_q + hq;
        float fac, lse;
        const float sk = kWide ? s_sink[c] : (prm.sinks ? __ldg(prm.sinks + hq) : kNegInf);
        finish(mx, sum, sk, kWide ? s_vscale : __ldg(prm.v_scale), &fac, &lse);
        s_cq[c] = fac;
        s_row[c] = row;
        prm.lse[row] = lse;
      }
    }
    __syncthreads();
    constexpr int kFrag = kNT * kSteps * 32;
    auto write = [&](int x, const float4& a) {  // the finished fragment x
      const int n = x / (kSteps * 32), j = x / 32 % kSteps, c = n * 8 + 2 * (x % 4);
      const int d = x % 32 / 4 * (kHd / 8) + 2 * j;
      if (c < ncols)
        *reinterpret_cast<uint32_t*>(prm.out + s_row[c] * kHd + d) = pack_bf16x2(a.x * s_cq[c], a.z * s_cq[c]);
      if (c + 1 < ncols)
        *reinterpret_cast<uint32_t*>(prm.out + s_row[c + 1] * kHd + d) =
            pack_bf16x2(a.y * s_cq[c + 1], a.w * s_cq[c + 1]);
    };
    for (int x = threadIdx.x; x < kFrag; x += kWarps * 32) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 y = part[w * kFrag + x];
        a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
      }
      if ((kPieces || kShards) && slot >= 0) prm.ws_o[slot * kFrag + x] = a;
      else if (kWide && prm.splits > 1) part[x] = a;  // (the only thread that reads the others of x)
      else write(x, a);
    }
    if (kWide && prm.splits > 1) {
      // The cluster's states, in the order of its CTAs: every CTA works out the weights, and merges its share of the
      // fragments.  (Fetching those beside the weights cost the loop registers: 7.1 us instead of 6.7 for one context.)
      cluster_sync();
      const int rank = unit % prm.splits, share = kFrag / prm.splits;
      if (threadIdx.x < kNT * 8) {
        const int c = threadIdx.x;
        float2 ml[kMaxCluster];
        float mx = kNegInf, sum = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          ml[r] = make_float2(kNegInf, 0.f);
          if (r < prm.splits) ml[r] = ld_cluster(&s_ml[c], r);
        }
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) mx = fmaxf(mx, ml[r].x);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          const float weight = ml[r].x == kNegInf ? 0.f : ex2_approx(ml[r].x - (mx == kNegInf ? 0.f : mx));
          s_weight[r][c] = weight;
          sum += ml[r].y * weight;
        }
        if (c < ncols) {
          const int col = col0 + c, token = col / prm.group, hq = kvh * prm.group + col - token * prm.group;
          const int64_t row = (static_cast<int64_t>(b) * prm.q_len + token) * prm.h_q + hq;
          float fac, lse;
          finish(mx, sum, s_sink[c], s_vscale, &fac, &lse);
          s_cq[c] = fac;
          s_row[c] = row;
          if (rank == 0) prm.lse[row] = lse;
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < share; i += kWarps * 32) {
        const int x = rank * share + i, c = x / (kSteps * 32) * 8 + 2 * (x % 4);
        float4 y[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          y[r] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r < prm.splits) y[r] = ld_cluster(&part[x], r);
        }
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          const float w0 = s_weight[r][c], w1 = s_weight[r][c + 1];
          a.x += y[r].x * w0, a.y += y[r].y * w1, a.z += y[r].z * w0, a.w += y[r].w * w1;
        }
        write(x, a);
      }
      __syncwarp();
      cluster_sync();  // until its last reader, a CTA's shared memory stays
    }
    __syncthreads();  // the ring is free for the next segment's copies
  }
}

// Merge of the shards of one (sequence, KV head) and column tile.  Lane x of a warp owns one float4 of the fragment
// order (two dims of two columns) of one step (16 dims).  With kGroups = 1 the four warps take four steps; with
// more, the warps take shards w, w + kGroups, ... of one step and meet in shared memory (few sequences, many shards:
// three contexts cut into 76 shards each take 17.9 us a call with 16, 18.9 with 8, 20.9 with 4, 19.5 with 32).
template <int kHd, int kNT, int kGroups>
__global__ void __launch_bounds__(kGroups == 1 ? 128 : kGroups * 32)
    fp4_combine_kernel(const __grid_constant__ Params prm) {
  constexpr int kSteps = kHd / 16, kFrag = kNT * kSteps * 32;
  __shared__ float4 s_o[kGroups][32], s_ml[kGroups][32];
  griddep_wait();
  const int seq = blockIdx.x;
  const int group = kGroups == 1 ? 0 : threadIdx.x / 32, lane = threadIdx.x % 32;
  const int frag = kGroups == 1 ? blockIdx.z * 4 + threadIdx.x / 32 : blockIdx.z;
  const int n = frag / kSteps, j = frag % kSteps;
  const int col0 = blockIdx.y * (kNT * 8);
  const int ncols = min(prm.q_len * prm.group - col0, kNT * 8);
  const int c = n * 8 + 2 * (lane % 4);
  // the shards' slots: first, then next, next + step, ...
  long long first, next;
  int step, count;
  if (prm.splits == 0) {
    const int2 span = prm.ws_span[seq];
    if (span.x == span.y) return;  // within one piece: written there
    const long long base = static_cast<long long>(blockIdx.y) * prm.units * 2;
    first = base + 2 * span.x + 1;
    next = base + 2 * (span.x + 1);
    step = 2;
    count = span.y - span.x + 1;  // 0 where there is no key (1, 0)
  } else {
    first = (static_cast<long long>(blockIdx.y) * gridDim.x + seq) * prm.splits;
    next = first + 1;
    step = 1;
    count = prm.splits;
  }
  const int b = seq / prm.h_kv, kvh = seq % prm.h_kv;
  const float v_scale = __ldg(prm.v_scale);
  float sink[2] = {kNegInf, kNegInf};
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (prm.sinks != nullptr && c + k < ncols)
      sink[k] = __ldg(prm.sinks + kvh * prm.group + (col0 + c + k) % prm.group);
  float m0 = kNegInf, m1 = kNegInf, l0 = 0.f, l1 = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = group; s0 < count; s0 += 4 * kGroups) {  // four shards' loads in flight
    float4 ml[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = s0 + kGroups * i;
      ml[i] = make_float4(kNegInf, 0.f, kNegInf, 0.f);
      y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < count) {
        const long long slot = s == 0 ? first : next + (s - 1) * step;
        ml[i] = *reinterpret_cast<const float4*>(prm.ws_ml + slot * (kNT * 8) + c);
        y[i] = prm.ws_o[slot * kFrag + frag * 32 + lane];
      }
    }
    float x0 = m0, x1 = m1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x0 = fmaxf(x0, ml[i].x);
      x1 = fmaxf(x1, ml[i].z);
    }
    const float b0 = x0 == kNegInf ? 0.f : x0, b1 = x1 == kNegInf ? 0.f : x1;
    const float f0 = ex2_approx(m0 - b0), f1 = ex2_approx(m1 - b1);
    m0 = x0, m1 = x1;
    l0 *= f0, l1 *= f1;
    a.x *= f0, a.y *= f1, a.z *= f0, a.w *= f1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float w0 = ex2_approx(ml[i].x - b0), w1 = ex2_approx(ml[i].z - b1);
      l0 += ml[i].y * w0, l1 += ml[i].w * w1;
      a.x += y[i].x * w0, a.y += y[i].y * w1, a.z += y[i].z * w0, a.w += y[i].w * w1;
    }
  }
  if constexpr (kGroups > 1) {
    s_o[group][lane] = a;
    s_ml[group][lane] = make_float4(m0, l0, m1, l1);
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int w = 1; w < kGroups; ++w) {
      m0 = fmaxf(m0, s_ml[w][lane].x);
      m1 = fmaxf(m1, s_ml[w][lane].z);
    }
    const float b0 = m0 == kNegInf ? 0.f : m0, b1 = m1 == kNegInf ? 0.f : m1;
    l0 = l1 = 0.f;
    a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kGroups; ++w) {
      const float4 ml = s_ml[w][lane], y = s_o[w][lane];
      const float w0 = ex2_approx(ml.x - b0), w1 = ex2_approx(ml.z - b1);
      l0 += ml.y * w0, l1 += ml.w * w1;
      a.x += y.x * w0, a.y += y.y * w1, a.z += y.z * w0, a.w += y.w * w1;
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (c + k >= ncols) continue;
    const int col = col0 + c + k, hq = kvh * prm.group + col % prm.group;
    const size_t row = (static_cast<size_t>(b) * prm.q_len + col / prm.group) * prm.h_q + hq;
    float fac, lse;
    finish(k ? m1 : m0, k ? l1 : l0, sink[k], v_scale, &fac, &lse);
    *reinterpret_cast<uint32_t*>(prm.out + row * kHd + lane / 4 * (kHd / 8) + 2 * j) =
        pack_bf16x2((k ? a.y : a.x) * fac, (k ? a.w : a.z) * fac);
    if (j == 0 && lane < 4) prm.lse[row] = lse;
  }
}

// ---------------------------------------------------------------- host ----

int col_tiles(int cols, int* nt) {  // columns run eight or sixteen to a CTA
  *nt = cols <= 8 ? 1 : 2;
  return (cols + 8 * *nt - 1) / (8 * *nt);
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// How a call is laid out: shards of every sequence (1: none, 0: balanced pieces; kWideCtas: CTAs of its cluster),
// pieces, and the workspace.
struct Plan {
  int nt, ct, splits, units;
  Ctas kind;    // kWideCtas: `splits` of them in a cluster for a sequence
  size_t slots, ml, span, bytes;  // partial states, and where (m, l) and the spans of pieces begin
};

// A window no shorter than any sequence hides nothing.
int seen_window(int window, long long capacity) { return window >= capacity ? 0 : window; }

Plan make_plan(int bs, int h_q, int h_kv, int head_dim, int q_len, long long capacity, int window, int num_splits) {
  Plan p;
  const int cols = q_len * (h_q / h_kv);
  p.ct = col_tiles(cols, &p.nt);
  long long longest = std::max(capacity, 1LL);
  window = seen_window(window, capacity);
  if (window > 0) longest = std::min(longest, static_cast<long long>(window) + q_len - 1 + kTile);
  const long long tiles = (longest + kTile - 1) / kTile;
  const long long seqs = static_cast<long long>(bs) * h_kv;
  const int resident = device_sms() * (head_dim == 256 ? 2 : 3);  // Shape::kPerSm
  p.units = 0;
  p.kind = kWholeCtas;
  // Few sequences: an SM's warps in one CTA, and CTAs in a cluster, which merges without a second kernel, while
  // clusters of that size surely fit on the GPU at once: eight CTAs up to a twelfth of the SMs, four up to 4 / 19, two
  // up to 9 / 19 (of 152 SMs 12, 32 and 72 clusters; 15, 36 and 76 did fit, but 16 of eight, in two waves, took 13 us).
  // The lengths are not known here, so what counts is what the block table holds.  A cluster's merge takes 1.4 us,
  // so short contexts stay with one CTA (8 sequences of 25 tiles: 6.3 us, in clusters of eight 7.1; of 50 tiles 7.7 and
  // 7.1; sixteen columns, of 50 tiles 10.5 and 8.6).
  // Cutting into pieces gains by the SMs that would otherwise idle and by equal shares, and pays for the second kernel:
  // with clusters from about three tiles for each of their CTAs on (hd 128, eight columns: 2 x 8 CTAs 50 tiles 6.9 us
  // and cut 8.4, 100 tiles 7.2 and 7.0; 8 x 8 CTAs 100 tiles 7.2 and 7.8, 400 tiles 10.1 and 8.6; 32 x 4 CTAs 200
  // tiles 9.9 and 11.5, 400 tiles 13.4 and 13.4); without, where 36 % to 100 % of the SMs have a CTA, from 64 tiles up
  // to four times as many.
  const long long sms = device_sms();
  long long ctas, uncut;
  int cluster, alone;
  bool few;
  auto lay_out = [&] {
    ctas = seqs * p.ct;
    few = ctas <= sms;
    cluster = ctas * 12 <= sms ? 8 : (ctas * 19 <= sms * 4 ? 4 : (ctas * 19 <= sms * 9 ? 2 : 1));
    alone = (head_dim == 64 ? 56 : (head_dim == 256 ? 20 : (p.nt == 1 ? 36 : 24))) * (cluster > 2 ? 4 : 7) / 4;
    if (!few)
      uncut = kShort;
    else if (cluster == 1)
      uncut = std::min<long long>(256, (head_dim == 256 ? 24 : (p.nt == 1 ? 64 : 36)) * sms / (sms - 3 * ctas / 4));
    else
      uncut = 24 + ctas * cluster * (head_dim == 256 ? 4 : (p.nt == 1 ? 6 : 3)) / 2;
  };
  lay_out();
  if (p.nt == 2 && num_splits == 0 && seqs * ((cols + 7) / 8) <= sms) {
    // SMs to spare: eight columns a CTA, whose keys come from L2 the second time (8 x 16 columns of 25 tiles 8.4 us, in
    // eights 7.1, of 100 tiles 9.6 and 8.4, of 200 tiles 10.0 and 10.4; 32 x 16 of 25 tiles 8.5 and 7.2, of 100 tiles
    // 10.9 and 10.6, of 200 tiles 13.0 and 13.7)
    const Plan sixteen = p;
    p.nt = 1;
    p.ct = (cols + 7) / 8;
    lay_out();
    if (tiles > std::min(uncut, 150LL)) {
      p = sixteen;
      lay_out();
    }
  }
  if (num_splits > 0) {
    p.splits = static_cast<int>(std::min<long long>(num_splits, std::max(1LL, (tiles + 7) / 8)));
  } else if (tiles <= uncut || ctas >= 8LL * resident || bs > kMaxLine ||
             seqs * (tiles + kFixed) > 0x7FFFFFFFll) {
    // Short contexts: one CTA or cluster a sequence takes no longer than pieces and their merge.  Many sequences of
    // like lengths: their CTAs balance by themselves.  A far longer one among them keeps its CTAs alone at the end (512
    // of 1000 keys 122 us, one of them of 131072 keys 752, in four asked-for shards 257).  (The line's places are
    // counted in 32 bits.)
    p.splits = 1;
    if (few && tiles > 4) {
      p.kind = kWideCtas;
      if (tiles > alone) p.splits = cluster;
    } else if (const long long places = sms * (head_dim == 256 ? 2 : (head_dim == 64 && p.nt == 1 ? 4 : 3));
               ctas > places && tiles <= kShort) {
      // More than fit at once (places: Shape::kPerSm of kWholeCtas): half the warps in twice as many places, unless
      // those are left emptier at the end and the contexts are not that short (512 sequences of 7 tiles 10.0 us, narrow
      // 6.6, of 94 tiles 33.2 and 29.0; 1024 of 50 tiles 33.2 and 32.7, of 94 tiles 50.9 and 54.5; head_dim 256, 768 of
      // 13 tiles 23.2 and 21.9, of 50 tiles 46.8 and 52.4)
      const long long rounds = (ctas + places - 1) / places, narrow = (ctas + 2 * places - 1) / (2 * places);
      if (tiles <= (head_dim == 256 ? 20 : 50) || 2 * narrow <= rounds) p.kind = kNarrowCtas;
    }
  } else {
    p.kind = kFillingCtas;
    p.splits = 0;
    p.units = std::max(1, resident / p.ct);
  }
  p.slots = 0;
  if (p.kind == kFillingCtas) p.slots = static_cast<size_t>(p.ct) * 2 * p.units;
  if (p.kind == kWholeCtas && p.splits > 1) p.slots = static_cast<size_t>(p.ct) * seqs * p.splits;
  p.ml = round_up(p.slots * p.nt * 8 * head_dim * sizeof(float), 256);
  p.span = p.ml + round_up(p.slots * p.nt * 8 * sizeof(float2), 256);
  p.bytes = p.span + (p.splits == 0 ? round_up(static_cast<size_t>(seqs) * sizeof(int2), 256) : 0);
  return p;
}

bool sizes_ok(int bs, int h_q, int h_kv, int head_dim, int q_len, int window, int num_splits) {
  return (head_dim == 64 || head_dim == 128 || head_dim == 256) && bs >= 0 && h_q >= 1 && h_kv >= 1 &&
         h_q % h_kv == 0 && q_len >= 1 && q_len <= kMaxQLen &&
         static_cast<long long>(q_len) * (h_q / h_kv) <= kMaxCols && window >= 0 && num_splits >= 0;
}

template <int kHd, int kNT, Ctas kCtas>
cudaError_t launch_decode(const Params& prm, int seqs, int ct, cudaStream_t stream) {
  using S = Shape<kHd, kNT, kCtas>;
  constexpr size_t smem =
      std::max<size_t>(static_cast<size_t>(S::kWarps) * S::kStages * S::kU * Lay<kHd>::kBytes,
                       static_cast<size_t>(S::kWarps) * kNT * (kHd / 16) * 32 * sizeof(float4));
  static_assert(S::kPerSm * (smem + (S::kNarrow ? 10 : 16) * 1024) <= 233472, "the CTAs fit in an SM's shared memory");
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = configure_once(configured, [&] {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(fp4_decode_kernel<kHd, kNT, kCtas>),
                                cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  const unsigned grid = prm.splits == 0 ? static_cast<unsigned>(prm.units)
                                        : static_cast<unsigned>(seqs) * static_cast<unsigned>(prm.splits);
  if (S::kWide && prm.splits > 1)
    return launch_dependent_clusters(prm.splits, fp4_decode_kernel<kHd, kNT, kCtas>, dim3(grid, ct),
                                     dim3(S::kWarps * 32), smem, stream, prm);
  return launch_dependent(fp4_decode_kernel<kHd, kNT, kCtas>, dim3(grid, ct), dim3(S::kWarps * 32), smem, stream, prm);
}

template <int kHd, int kNT>
cudaError_t launch(const Params& prm, Ctas ctas, int seqs, int ct, cudaStream_t stream) {
  if (ctas == kWideCtas) return launch_decode<kHd, kNT, kWideCtas>(prm, seqs, ct, stream);
  if (ctas == kNarrowCtas) return launch_decode<kHd, kNT, kNarrowCtas>(prm, seqs, ct, stream);
  const cudaError_t e = ctas == kWholeCtas ? launch_decode<kHd, kNT, kWholeCtas>(prm, seqs, ct, stream)
                                           : launch_decode<kHd, kNT, kFillingCtas>(prm, seqs, ct, stream);
  if (e != cudaSuccess || prm.splits == 1) return e;
  // warps for the shards that a sequence has on average, four at a time each (100 sequences cut into 5: 19.4 us a call
  // with one warp, 25.3 with sixteen, most of them idle; 6 cut into 76: 17.9 with sixteen, 20.9 with four)
  constexpr unsigned kFrags = kNT * (kHd / 16);
  const unsigned s = static_cast<unsigned>(seqs);
  const int shards = prm.splits == 0 ? prm.units / seqs + 1 : prm.splits;
  if (shards <= 8)
    return launch_dependent(fp4_combine_kernel<kHd, kNT, 1>, dim3(s, ct, kFrags / 4), dim3(128), 0, stream, prm);
  if (shards <= 24)
    return launch_dependent(fp4_combine_kernel<kHd, kNT, 4>, dim3(s, ct, kFrags), dim3(128), 0, stream, prm);
  return launch_dependent(fp4_combine_kernel<kHd, kNT, 16>, dim3(s, ct, kFrags), dim3(512), 0, stream, prm);
}

}  // namespace fp4

size_t fp4_workspace_bytes(int bs, int h_q, int h_kv, int head_dim, int q_len, long long max_seqlen, int window,
                           int num_splits) {
  if (!fp4::sizes_ok(bs, h_q, h_kv, head_dim, q_len, window, num_splits) || bs == 0) return 0;
  return fp4::make_plan(bs, h_q, h_kv, head_dim, q_len, max_seqlen, window, num_splits).bytes;
}

fp8mla_status_t fp4_decode_entry(const Fp4DecodeArgs& a, cudaStream_t stream) {
  if (!fp4::sizes_ok(a.bs, a.h_q, a.h_kv, a.head_dim, a.q_len, a.window, a.num_splits) || a.num_blocks < 1 ||
      a.max_blocks < 1 || !(a.softmax_scale > 0.f))
    return FP8MLA_ERR_INVALID_ARG;
  int page_shift = 0;
  while (page_shift < 5 && (fp4::kTile << page_shift) != a.page_size) ++page_shift;
  if (page_shift == 5) return FP8MLA_ERR_INVALID_ARG;  // 16, 32, 64, 128 or 256 keys a page
  const long long slots = static_cast<long long>(a.num_blocks) * a.page_size;
  if (slots >= (1ll << 32) || slots * a.h_kv >= (1ll << 32)) return FP8MLA_ERR_INVALID_ARG;  // rows: 32 bits
  if (a.bs == 0) return FP8MLA_OK;
  if (a.q == nullptr || a.k_cache == nullptr || a.v_cache == nullptr || a.k_block_scales == nullptr ||
      a.v_block_scales == nullptr || a.k_scale == nullptr || a.v_scale == nullptr || a.block_table == nullptr ||
      a.seqlens == nullptr || a.out == nullptr || a.lse == nullptr)
    return FP8MLA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k_cache) |
       reinterpret_cast<uintptr_t>(a.v_cache) | reinterpret_cast<uintptr_t>(a.k_block_scales) |
       reinterpret_cast<uintptr_t>(a.v_block_scales) | reinterpret_cast<uintptr_t>(a.out)) & 15u)
    return FP8MLA_ERR_INVALID_ARG;
  if (misaligned(a.k_scale, 4) || misaligned(a.v_scale, 4) || misaligned(a.block_table, 4) ||
      misaligned(a.seqlens, 4) || misaligned(a.sinks, 4) || misaligned(a.lse, 4))
    return FP8MLA_ERR_INVALID_ARG;
  const long long capacity = static_cast<long long>(a.max_blocks) * a.page_size;
  if (capacity > 0x7FFFFF00ll) return FP8MLA_ERR_INVALID_ARG;
  const fp4::Plan plan =
      fp4::make_plan(a.bs, a.h_q, a.h_kv, a.head_dim, a.q_len, capacity, a.window, a.num_splits);
  if (plan.bytes > 0) {
    if (a.workspace == nullptr || (reinterpret_cast<uintptr_t>(a.workspace) & 255u)) return FP8MLA_ERR_INVALID_ARG;
    if (a.workspace_bytes < plan.bytes) return FP8MLA_ERR_WORKSPACE_TOO_SMALL;
  }
  const long long seqs = static_cast<long long>(a.bs) * a.h_kv;
  if (seqs * std::max(plan.splits, 1) > 0x7FFFFFFFll) return FP8MLA_ERR_INVALID_ARG;
  // the output may take the queries' place (a row is written after its last reader); nothing else is shared
  const uint64_t rows = static_cast<uint64_t>(a.bs) * a.q_len * a.h_q;
  const Rows q = block_of(a.q, rows * a.head_dim * 2), out = block_of(a.out, rows * a.head_dim * 2);
  const Rows lse = block_of(a.lse, rows * 4), ws = block_of(a.workspace, plan.bytes);
  if (clobbers(out, q) || rows_overlap(lse, q) || rows_overlap(ws, q) || rows_overlap(out, lse) ||
      rows_overlap(out, ws) || rows_overlap(lse, ws))
    return FP8MLA_ERR_INVALID_ARG;
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
  p.ws_o = static_cast<float4*>(a.workspace);
  p.ws_ml = plan.bytes > 0 ? reinterpret_cast<float2*>(static_cast<char*>(a.workspace) + plan.ml) : nullptr;
  p.ws_span = plan.splits == 0 ? reinterpret_cast<int2*>(static_cast<char*>(a.workspace) + plan.span) : nullptr;
  p.num_blocks = a.num_blocks;
  p.max_blocks = a.max_blocks;
  p.bs = a.bs;
  p.h_q = a.h_q;
  p.h_kv = a.h_kv;
  p.group = a.h_q / a.h_kv;
  p.splits = plan.splits;
  p.units = plan.units;
  p.q_len = a.q_len;
  p.window = fp4::seen_window(a.window, capacity);
  p.page_shift = page_shift;
  p.softmax_scale = a.softmax_scale;
  const int n = static_cast<int>(seqs);
  cudaError_t e;
  switch (a.head_dim + plan.nt) {
    case 64 + 1: e = fp4::launch<64, 1>(p, plan.kind, n, plan.ct, stream); break;
    case 64 + 2: e = fp4::launch<64, 2>(p, plan.kind, n, plan.ct, stream); break;
    case 128 + 1: e = fp4::launch<128, 1>(p, plan.kind, n, plan.ct, stream); break;
    case 128 + 2: e = fp4::launch<128, 2>(p, plan.kind, n, plan.ct, stream); break;
    case 256 + 1: e = fp4::launch<256, 1>(p, plan.kind, n, plan.ct, stream); break;
    default: e = fp4::launch<256, 2>(p, plan.kind, n, plan.ct, stream); break;
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
