// Attention of runs of query rows to paged E4M3 keys, all of them visible: cross attention to an encoder's states, and
// the two halves (shared prefix, own keys) of a decode step behind shared prefixes.
//
// A segment is a run of query tokens and the list of pages they all read.  With G query heads to a KV head, the rows of
// (segment, KV head) are its tokens' G heads one token after the other, and
//   out[r] = sum_j softmax_j(c q_r . k_j) v_j,   lse[r] = log sum_j exp(c q_r . k_j).
//
// One CTA an SM walks its share of a line of work: every (segment, KV head, 256 rows) is an item of the line, as long as
// its key tiles of 128 and a fixed part take.  The line is cut into equal shares on the device, since lengths are known
// there alone; an item that a cut meets leaves partial sums in the workspace, merged by a second launch.
//
// Per item the rows are the M of the matrix products (tcgen05): S = Q K^T and O += P V, 128 rows in the lanes of TMEM,
// P written over S by the threads that own the rows.  K is read as it is cached, Q times a power of two per row as two
// E4M3 terms that sum to it; P is f16, and V is turned into f16, which holds it exactly.
//   up to 256 rows: two streams of 128 rows, each with its own S and O; the tensor core works for one while the other's
//     softmax runs.
//   up to 128 rows: one stream, S in two buffers by tile parity, and both softmax warpgroups share a tile's columns.
//   up to 32 rows: the same with the rows in all four quarters of the lanes, each with P for its own 32 keys of a tile
//     (zero for the others) and a reference of its own: eight warps share the softmax, the quarters are summed at the end.
// Warps: 0-3 and 4-7 the two softmax warpgroups, 8-11 lay out Q and turn V into f16, 12 issues the products, 13 and 15
// copy tiles of K and of V (one TMA copy a page), 14 finds the CTA's share, tells the others its items and fills rows of
// no sequence.
//
// Why so.  A key is read once for up to 256 rows; 4 hd operations a row and 2 hd bytes a key make about 140 rows the
// border between HBM and the products.
//   K as codes and Q in two terms: as many tensor cycles as f16 Q and K, but no conversion of K, no f16 tile of it in
//     shared memory and no warps for either (with the TMA copies: document 421 -> 413 us, decode step 90 -> 73).
//   256 rows an item: V's conversion and a tile's copies are paid once for twice the rows; the second stream's products
//     hide the first one's softmax.  128 keys a tile: S and P of both streams and O (head_dim 128) fill TMEM's 512 columns.
//   32 rows in all lane quarters: in one quarter a single warp of each warpgroup would have all the exponentials, so
//     eight share them (decode step 114 -> 90 us).
//   Shares of a line and not an item a CTA: lengths differ by ten times in a batch; lengths by form, head_dim and scales
//     as measured (prompts 39 -> 37 us), empty sequences at their 0.75 us (decode step 54 -> 50).
//   One warp that tells items: with the walk in every role they spilled (605 -> 421 us; 8 to 28 bytes now).  Short code: a launch's
//     instructions come from memory, and a loop of all roles has to stay in the instruction cache (decode step 71 -> 53).
//   No maximum where sums show that none is needed (pair form without row scales): 128 comparisons a row and tile less.
//
// Measured (GB300, calls from a graph over three inputs): 2048 tokens x 32 heads by 16384 keys of 8 heads, head_dim 128,
// 387 us = 1420 TFLOP/s, 0.75 of a library bf16 product; 64 tokens by 128 to 1600 keys with row scales 51 us; 64 tokens by
// 16000 keys 394 us = 0.79 of a copy, with row scales 506 = 0.63 (pages of 16; of 64: 385 and 436); one token by 777 keys
// 12.7 us; 64 sequences behind a prefix of 32768 keys 80 us.
// In the first of them the tensor pipe is active 61 to 63 % of the time, XU 31, ALU 25, DRAM 2: no unit is full.  A tile
// takes either stream about 3400 cycles for 2048 of the tensor core: product, scores loaded (220), weighed (1150), P
// written (250), the issuing warp's turn (600), product with P and the next with K, each queued behind the other
// stream's.  Halving the exponentials takes 2.5 % off, Q K^T 8, P V 5, no conversion 1.5.  A second warp that issues the
// other stream's products interleaves them on the tensor core: 506 us.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "ragged_gqa.h"

namespace fp8mla {

__device__ uint32_t g_status_ragged;

namespace ragged {

constexpr int kTile = 128;      // keys a tile, rows a stream
constexpr int kItemRows = 256;  // rows an item
constexpr int kThreads = 512;
constexpr int kSoftmaxRegs = 192, kConvertRegs = 72, kIssueRegs = 56;  // registers a thread of the warpgroups
constexpr float kLift = 7.f;    // P = 2^(score - reference + 7): 2^15 at most in f16, normal down to 2^-21 of the largest
constexpr uint32_t kNone = 0xFF800000u;  // -inf: the score of a key past the end
constexpr float kFar = 1048576.f;  // 2^20 in log2 units: up to here the lift and the difference keep their fraction
constexpr float kTau = 8.f;     // the reference moves when a score passes it by more
constexpr float kNoRef = -1e30f;  // the reference of a row whose V scales so far are all zero
// V's row scales within 2^+-40 enter the weights, and the sum of exponentials divides them out again.  Past that the
// smallest weights vanish beside the largest, and 1 / scale and the sum leave float32: from the first tile with such a scale
// on, an item's sum is taken from the scores alone, relative to their own maximum.
constexpr float kSmallScale = 0x1p-40f, kLargeScale = 0x1p40f;

// Up to 32 rows lie in all quarters (few), up to 128 are one stream, up to 256 a pair of streams.
constexpr int kFew = 32;
enum { kFormPair = 0, kFormOne = 1, kFormFew = 2, kForms = 3 };

// Lengths of the line, in twentieths of a microsecond: what a key tile takes, and an item's beginning and end, by form.
// Measured as the shares' ends over their items and tiles (decode steps, prompts and prefixes of either kind).
struct Lengths {
  int each[kForms], fixed[kForms];
};
constexpr Lengths kLengths[2][2] = {{{{24, 24, 13}, {60, 30, 26}}, {{42, 34, 15}, {56, 31, 28}}},    // head_dim 64
                                    {{{37, 26, 18}, {80, 45, 38}}, {{52, 35, 20}, {95, 58, 38}}}};  // 128: plain, row scales
constexpr uint32_t kWaitLimit = 3500000000u;  // ns of a wait, in 32 bits
constexpr int kEmpty = 15;  // an item without keys
constexpr int kLeast = 60;  // a share
constexpr int kMostUnits = 256;  // shares (one an SM)
constexpr int kWhole = 140;      // items of a call that is not cut

struct List {
  const int32_t* starts;  // segment s has the tokens [per starts[s], per starts[s + 1]); null: [per s, per (s + 1))
  const int32_t* lens;
  const int32_t* table;
  int n, max_blocks, max_keys, per;
  int most;  // starts at most
  int less;  // the last keys that are left out
};

struct Cut {  // the item that a share begins and does not end
  long long start, end;
  int valid, slot, head, t0, row0, rows;
};

struct Params {
  const uint16_t* q;
  const uint8_t *k, *v;
  const float *k_scale, *v_scale;
  uint16_t* out;
  float* lse;
  long long* lo;        // [units + 1] where the shares begin
  int* units;
  long long* seg_at;    // joined: where the segments begin
  Cut* cuts;            // [units]
  float2* slot_ml;      // [2 units][slot_rows]
  float* slot_o;        // [2 units][slot_rows][hd]
  float2* plane_ml[2];  // joined: whole items of either list, [tokens * h_q]
  float* plane_o[2];
  const uint8_t* spec_mask;
  const float* sinks;
  long long q_tok, q_head, o_tok, o_head;
  List list[2];
  FastDiv group, of_rows, of_heads;  // of_rows: a sequence's of a KV head
  unsigned long long per_unit;  // 2^64 / grid
  float softmax_scale;
  Lengths lengths;
  int joined, whole, tokens, h_q, h_kv, num_blocks, page_shift, slot_rows, fill_out, fill_lse, q_len;
  uint32_t wait_limit, fault_tile;  // of the test hook: ns; the tile of K, from 1 on, that CTA 0 does not copy
};

// ---------------------------------------------------------------- the line --

struct Seg {
  int t0, rows, keys, tiles, row_tiles;
  int full, last;  // length of an item of 256 rows and of the last one
  long long head;  // of all items of a KV head
};

__host__ __device__ __forceinline__ int form_of(int rows) {
  return rows > kTile ? kFormPair : (rows > kFew ? kFormOne : kFormFew);
}

struct Bounds {  // of a segment, as the caller gives them
  int a, b, len;
};
__device__ __forceinline__ Bounds load_bounds(const Params& p, int s) {
  const List& l = s < p.list[0].n ? p.list[0] : p.list[1];
  if (s >= p.list[0].n) s -= p.list[0].n;
  Bounds x{s, s + 1, __ldg(l.lens + s)};
  if (l.starts != nullptr) x.a = __ldg(l.starts + s), x.b = __ldg(l.starts + s + 1);
  return x;
}

constexpr uint32_t kBadRange = 1u << 31;  // beside the status bits, for the kernel alone: a segment's tokens do not fit
__device__ __forceinline__ bool range_ok(const List& l, int a, int b) { return a >= 0 && a <= b && b <= l.most; }

__device__ __forceinline__ int seg_len(const List& l, int n, uint32_t* bad) {
  if (static_cast<uint32_t>(n) <= static_cast<uint32_t>(l.max_keys)) return n;
  *bad |= FP8MLA_DEV_BAD_SEQLEN;
  return 0;
}

__device__ __forceinline__ Seg make_seg(const Params& p, int s, const Bounds& x, uint32_t* bad) {
  const List& l = s < p.list[0].n ? p.list[0] : p.list[1];
  Seg g;
  int a = x.a, b = x.b;
  if (!range_ok(l, a, b)) {
    *bad |= FP8MLA_DEV_BAD_SEQLEN | kBadRange;
    a = b = 0;
  }
  g.t0 = a * l.per;
  const int t1 = b * l.per;
  g.rows = (t1 - g.t0) * static_cast<int>(p.group.d);
  g.keys = max(0, seg_len(l, x.len, bad) - l.less);
  g.tiles = (g.keys + kTile - 1) / kTile;
  g.row_tiles = (g.rows + kItemRows - 1) / kItemRows;
  g.full = g.last = p.joined ? 0 : kEmpty;
  if (g.tiles > 0) {
    const int form = form_of(g.rows - (g.row_tiles - 1) * kItemRows);
    g.full = p.lengths.fixed[kFormPair] + g.tiles * p.lengths.each[kFormPair];
    g.last = p.lengths.fixed[form] + g.tiles * p.lengths.each[form];
  }
  g.head = g.row_tiles > 0 ? static_cast<long long>(g.row_tiles - 1) * g.full + g.last : 0;
  return g;
}

__device__ __forceinline__ Seg read_seg(const Params& p, int s, uint32_t* bad) {
  return make_seg(p, s, load_bounds(p, s), bad);
}

// a / b for 0 <= a < 2^30, 0 < b: a quotient in 24 bits, put right (the division of integers is several times as long, and
// one warp does these while all others wait).
__device__ __forceinline__ int quick_div(int a, int b) {
  int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
  while (q * b > a) --q;
  while (q * b + b <= a) ++q;
  return q;
}

// Where a share that would begin `off` into an item of this length does: at a tile, at least `few` from either end.
__device__ __forceinline__ int cut_at(const Params& p, int off, int len, int form, int tiles, int few) {
  const int fixed = p.lengths.fixed[form], each = p.lengths.each[form];
  if (form != kFormPair) few = min(few, 2);  // little is written and merged
  if (tiles == 0) return off > 0 ? len : 0;
  const int t = off <= fixed ? 0 : quick_div(off - fixed + each / 2, each);
  if (t >= few && tiles - t >= few && !p.whole) return fixed + t * each;
  return 2 * t < tiles ? 0 : len;
}

// One item of a share, or the part of it that lies in the share.
struct Item {
  int list, seg, head, t0, row0, rows, keys, tile_lo, tile_hi;
  int slot;  // where its sums go: kDirect the outputs, kPlane the list's plane, else the workspace's slot
  int form;
  bool end;
};
constexpr int kDirect = -1, kPlane = -2;

// Where a share is: the segment, the item, how far into it, and how much is left.
struct Walk {
  Seg g;
  int seg, head, rt, off;
  long long left, hi;
  bool first;
};

constexpr int kGroups = 64;  // of segments, whose places on the line are kept

// The beginning of CTA `unit`'s share, by one warp; it is short, as its instructions come from memory in every launch.
// First the line's length, with the places where groups of segments begin; then the segments that hold the share's ends.
// Returns whether all segments' tokens fit.
__device__ __forceinline__ bool find_share(const Params& p, int unit, Walk* walk, long long (&group_at)[kGroups]) {
  const int n = p.list[0].n + p.list[1].n;
  const int lane = threadIdx.x % 32;
  const int each = ((n + 31) / 32 + kGroups - 1) / kGroups * 32;  // segments a group
  uint32_t bad = 0;
  // a lane's segment of the 32 from s0 on, and where it begins if those begin at `from`
  Seg g;
  auto place = [&](int s0, const Bounds& x, long long from, long long* len, long long* all) {
    const int s = s0 + lane;
    *len = 0;
    if (s < n) {
      g = make_seg(p, s, x, &bad);
      *len = g.head * p.h_kv;
    }
    long long sum = *len;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    *all = __shfl_sync(0xffffffffu, sum, 31);
    return from + sum - *len;
  };
  long long total = 0, at = 0, len = 0, all;
  Bounds x = {};
  if (n > 0) x = load_bounds(p, min(lane, n - 1));
#pragma unroll 1
  for (int s0 = 0; s0 < n; s0 += 32) {
    const Bounds now = x;
    if (s0 + 32 < n) x = load_bounds(p, min(s0 + 32 + lane, n - 1));
    at = place(s0, now, total, &len, &all);
    if (lane == 0 && s0 % each == 0) group_at[s0 / each] = total;
    // the merge looks segments up: a CTA writes the places of some
    if (p.joined && (s0 >> 5) % gridDim.x == unit && s0 + lane < n) p.seg_at[s0 + lane] = at;
    total += all;
  }
  const bool fits = !__any_sync(0xffffffffu, (bad & kBadRange) != 0);
  if (bad && unit == 0) atomicOr(&g_status_ragged, bad & ~kBadRange);
  int units, few;
  long long raw[2];
  if (total < (1 << 24)) {
    const uint32_t t = static_cast<uint32_t>(total);
    units = static_cast<int>(max(1u, min(gridDim.x, t / kLeast)));
    const float step = __fdividef(static_cast<float>(t), static_cast<float>(units));  // the same in every CTA
    few = static_cast<int>(__fdividef(step, static_cast<float>(3 * p.lengths.each[kFormPair])));
    raw[0] = min(t, static_cast<uint32_t>(step * static_cast<float>(unit)));
    raw[1] = min(t, static_cast<uint32_t>(step * static_cast<float>(unit + 1)));
  } else {
    units = gridDim.x;
    few = 4;
    raw[0] = __umul64hi(total * unit, p.per_unit);  // 2^64 / grid
    raw[1] = __umul64hi(total * (unit + 1), p.per_unit);
  }
  few = max(1, min(4, few));
  if (unit + 1 >= units) raw[1] = total;
  if (unit >= units) raw[0] = total;
  if (lane == 0) {
    walk->left = raw[0];
    walk->hi = total;
    walk->first = true;
    if (!p.joined) p.cuts[unit].valid = 0;
    if (unit == units - 1) {
      p.lo[units] = total;
      *p.units = units;
    }
    if (raw[0] >= total && unit < units) p.lo[unit] = total;
  }
  __syncwarp();
  if (raw[0] < total) {
    const int groups = (n + each - 1) / each;
    const uint32_t below = __ballot_sync(0xffffffffu, lane < groups && group_at[lane] <= raw[0]);
    const uint32_t more = __ballot_sync(0xffffffffu, lane + 32 < groups && group_at[(lane + 32) % kGroups] <= raw[0]);
    int s0 = (__popc(below) + __popc(more) - 1) * each;
    long long from = group_at[s0 / each];
    __syncwarp();
#pragma unroll 1
    for (; s0 < n && from <= raw[1]; s0 += 32) {
      all = total;
      if (n > 32) at = place(s0, load_bounds(p, min(s0 + lane, n - 1)), from, &len, &all);
      from += all;
      // lane 0 takes the share's beginning, lane 1 its end
      const uint32_t begins = __ballot_sync(0xffffffffu, raw[0] >= at && raw[0] < at + len);
      const uint32_t ends = __ballot_sync(0xffffffffu, raw[1] >= at && raw[1] < at + len);
      const uint32_t mine = lane == 0 ? begins : ends;
      const int src = max(__ffs(mine) - 1, 0);
      if ((begins >> lane) & 1) walk->g = g, walk->seg = s0 + lane;
      const long long want = lane == 0 ? raw[0] : raw[1], head = __shfl_sync(0xffffffffu, g.head, src);
      long long in = want - __shfl_sync(0xffffffffu, at, src);
      const int full = __shfl_sync(0xffffffffu, g.full, src), last = __shfl_sync(0xffffffffu, g.last, src);
      const int rows = __shfl_sync(0xffffffffu, g.rows, src), row_tiles = __shfl_sync(0xffffffffu, g.row_tiles, src);
      const int tiles = __shfl_sync(0xffffffffu, g.tiles, src);
      if (lane < 2 && mine != 0) {
        int h = 0;
        while (in >= head) in -= head, ++h;
        // in / full, of up to 2^22 items: the quotient in 24 bits, then put right (a 64-bit division would be a call)
        int rt = min(static_cast<int>(__fdividef(static_cast<float>(in), static_cast<float>(full))), row_tiles - 1);
        while (rt > 0 && static_cast<long long>(rt) * full > in) --rt;
        while (rt < row_tiles - 1 && static_cast<long long>(rt + 1) * full <= in) ++rt;
        const long long before = static_cast<long long>(rt) * full;
        const int item = rt == row_tiles - 1 ? last : full;
        int off = cut_at(p, static_cast<int>(in - before), item, form_of(rows - rt * kItemRows), tiles, few);
        const long long to = want - in + before + off;
        if (lane == 1) {
          walk->hi = to;
        } else {
          if (off == item) {  // the next item's beginning
            off = 0;
            if (++rt == row_tiles) rt = 0, ++h;
          }
          walk->head = h;
          walk->rt = rt;
          walk->off = off;
          p.lo[unit] = to;
          walk->left = to;  // for now
        }
      }
    }
  }
  __syncwarp();
  if (lane == 0) walk->left = walk->hi - walk->left;
  __syncwarp();
  return fits;
}

// The next item of a share (one thread).
__device__ __forceinline__ bool next_item(const Params& p, int unit, Walk* w, Item* it) {
  const long long left = w->left;
  if (left <= 0) return false;
  const int n = p.list[0].n + p.list[1].n;
  while (w->head == p.h_kv || w->g.head == 0) {
    if (++w->seg >= n) return false;
    uint32_t bad = 0;
    w->g = read_seg(p, w->seg, &bad);
    w->head = w->rt = 0;
  }
  const int rt = w->rt, off = w->off, tiles = w->g.tiles;
  const int len = rt == w->g.row_tiles - 1 ? w->g.last : w->g.full;
  const int row0 = rt * kItemRows, rows = min(kItemRows, w->g.rows - row0);
  const int list = w->seg < p.list[0].n ? 0 : 1;
  it->list = list;
  it->seg = list ? w->seg - p.list[0].n : w->seg;
  it->head = w->head;
  it->t0 = w->g.t0;
  it->row0 = row0;
  it->rows = rows;
  it->keys = w->g.keys;
  const int form = form_of(rows);
  it->form = form;
  const int fixed = p.lengths.fixed[form], each = p.lengths.each[form];
  const int tile_lo = off > 0 ? quick_div(off - fixed, each) : 0;
  const bool ends = len - off <= left;
  const int tile_hi = ends ? tiles : quick_div(off + static_cast<int>(left) - fixed, each);
  const bool whole = tile_lo == 0 && tile_hi == tiles;
  const int slot = 2 * unit + (w->first ? 0 : 1);
  it->tile_lo = tile_lo;
  it->tile_hi = tile_hi;
  it->slot = !whole ? slot : (p.joined ? kPlane : kDirect);
  if (!p.joined && tile_lo == 0 && !whole)
    p.cuts[unit] = Cut{w->hi - left, w->hi - left + len, 1, slot, w->head, w->g.t0, row0, rows};
  w->left = ends ? left - (len - off) : 0;
  w->first = false;
  w->off = 0;
  w->rt = rt + 1 == w->g.row_tiles ? 0 : rt + 1;
  if (w->rt == 0) ++w->head;
  return true;
}

// ------------------------------------------------------------- the kernel --

template <int kHd, bool kRows>
struct Lay {
  static constexpr int kQ = 2 * kTile * kHd;         // a stream's Q: two E4M3 terms a value
  static constexpr int kRaw = kTile * kHd;           // a tile of K or V as codes
  static constexpr int kF = kTile * kHd * 2;         // a tile of V in f16
  static constexpr int kKs = kHd == 128 ? 3 : 6, kVs = kHd == 128 ? (kRows ? 2 : 3) : 6, kFs = kHd == 128 ? 2 : 3;
  // Scales of a tile's rows: those of tile i are written once V of tile i - 1 is converted, which waits for the product
  // with P of tile i - 1 - kFs, so the softmax is done with tile i - 1 - kFs.
  static constexpr int kScls = kFs + 1;
  static constexpr int kSum = 2 * 4 * kFew * 32 * 4;  // sums of the quarters, 32 dims of either half; the second Q's place
  static constexpr int kOffK = 2 * kQ, kOffV = kOffK + kKs * kRaw, kOffF = kOffV + kVs * kRaw;
  static constexpr int kOffSum = kHd == 128 ? kQ : kOffF + kFs * kF;
  static constexpr int kOffCtl = kOffF + kFs * kF + (kHd == 128 ? 0 : kSum);
  static_assert(kHd != 128 || kSum <= kQ, "");
  static constexpr uint32_t kSwizzle = kHd == 128 ? SWIZZLE_128B : 4;  // of a row of codes
};

constexpr int kItems = 4;       // items told ahead
constexpr int kItemWarps = 15;  // that are told

template <int kHd, bool kRows>
struct Control {
  using L = Lay<kHd, kRows>;
  uint64_t k_full[L::kKs], k_empty[L::kKs], v_full[L::kVs], v_empty[L::kVs], f_full[L::kFs], f_empty[L::kFs];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t q_full, q_seen, q_empty, pv_done, xchg, scl_full[L::kScls], final_mma;
  uint64_t item_full[kItems], item_empty[kItems];
  Item item[kItems];
  Walk walk;
  long long group_at[kGroups];
  uint32_t tmem_base, abort_flag, never;  // never: the flag of waits that no other warp ends
  uint32_t sums_read;            // warps that are done with a few-row item's sums
  int8_t q_exp[2][kTile];        // of Q's rows, by stream
  float row_l[2][kTile], row_m[kTile];  // (row_l while an item's sum is apart: the largest score of this thread's row)
  alignas(16) float4 scl_k[kRows ? L::kScls : 1][kRows ? kTile / 2 : 1];  // of two keys: K scales, log2 of V scales
  alignas(16) float scl_v[kRows ? L::kScls : 1][kRows ? kTile : 4];       // 1 / V scale (0 where that is far from one)
  alignas(4) uint8_t scl_far[kRows ? L::kScls : 1][4];  // a tile's V scales that are, by warps' keys
  alignas(16) float raw_scl[kRows ? L::kVs : 1][2][kRows ? kTile : 4];
};

template <int kHd, bool kRows>
constexpr size_t smem_bytes() {
  return Lay<kHd, kRows>::kOffCtl + sizeof(Control<kHd, kRows>);
}

// Bounded waits of this kernel, in few instructions (it has to stay in the instruction cache): after the limit of
// polling without success, or once another warp gave up, false; the CTA then reports it at its end.
__device__ __forceinline__ uint32_t timer_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
// (The limit is an argument of the kernel: read from device memory in every wait's loop it is longer code, shared many 135 ->
// 140 us, and with a second count in the waits for items 157.)
struct Waits {
  volatile uint32_t* abort_flag;
  uint32_t limit;
};
// Waits for an item to be told or left take as long as items do, half a minute for 2^30 keys and more with sums apart: they
// have 2^25 polls (3.8 us each, two minutes) before the limit counts.  The warps at work on an item give up long before, and end these waits.
constexpr uint32_t kItemPolls = 1u << 25;
template <uint32_t kPolls = kWaitMinPolls, typename Done>
__device__ __forceinline__ bool wait_until(const Waits& w, Done done) {
  bool ok = done();
  if (!ok) {
    const uint32_t t0 = timer_lo();
    uint32_t polls = 0;
#pragma unroll 1
    do {
      if (*w.abort_flag) break;
      if (++polls > kPolls && timer_lo() - t0 > w.limit) *w.abort_flag = 1u;
      ok = done();
    } while (!ok);
  }
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const Waits& w) {
  return wait_until(w, [&] { return mbar_try_wait(bar, parity); });
}
__device__ __forceinline__ bool warp_wait_item(uint64_t* bar, uint32_t parity, const Waits& w) {
  return wait_until<kItemPolls>(w, [&] { return mbar_try_wait(bar, parity); });
}
// Until *count has reached `want` (it only grows).
__device__ __forceinline__ bool wait_count(volatile uint32_t* count, uint32_t want, const Waits& w) {
  const bool ok = wait_until(w, [&] { return static_cast<int32_t>(*count - want) >= 0; });
  __threadfence_block();
  return ok;
}

__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Smallest e with amax <= 448 * 2^e, from -60 on (what is smaller still makes no score).
__device__ __forceinline__ int exponent_448(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  return max(static_cast<int>(bits >> 23) - 127 - ((bits & 0x7FFFFFu) <= 0x600000u ? 8 : 7), -60);
}

// Rows [first, first + count) of a stream (row0: its first in the item) in shared memory: each times a power of two that
// puts its largest value into (224, 448], as two E4M3 terms, x = E4M3(x) + E4M3(x - E4M3(x)): exact for bf16 from 2^-2 on
// (2^-9.8 of the row's largest value), else off by 2^-10 at most, half of E4M3's last step (2^-17.8 of it).  Where
// `quarters`, in all quarters of the lanes.  head_dim 128: a tile of 128-byte rows per term; 64: both terms in one row.
template <int kHd>
__device__ __forceinline__ void load_q(const Params& p, const Item& it, uint8_t* q_tile, int8_t* q_exp, int row0,
                                       int first, int count, bool quarters, int lane) {
  constexpr int kLanes = kHd / 16, kStep = 32 / kLanes;  // lanes a row, rows a pass
  const int ch = lane % kLanes;
  const int end = min(first + count, it.rows - row0);
  const int item_row = it.row0 + row0, head0 = it.head * static_cast<int>(p.group.d), t0 = it.t0;
  uint4 x[2], ahead[2];
  auto load = [&](int row) {
    ahead[0] = ahead[1] = make_uint4(0, 0, 0, 0);
    if (row < end) {
      const uint32_t r = static_cast<uint32_t>(item_row + row);
      const uint32_t t = fast_div(r, p.group);
      const int head = head0 + static_cast<int>(r - t * p.group.d);
      const uint4* from =
          reinterpret_cast<const uint4*>(p.q + (t0 + static_cast<long long>(t)) * p.q_tok + head * p.q_head + ch * 16);
      ahead[0] = __ldg(from);
      ahead[1] = __ldg(from + 1);
    }
  };
  int row = first + lane / kLanes;
  if (first < end) load(row);
#pragma unroll 1
  for (int base = first; base < end; base += kStep, row += kStep) {
    x[0] = ahead[0], x[1] = ahead[1];
    if (base + kStep < end) load(row + kStep);
    {
      const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = exponent_448(amax);
      const float inv = amax < -kNegInf ? exp2i(-e) : __int_as_float(0x7FFFFFFF);  // an infinity makes no score either
      if (row < end) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          split_e4m3x4(bf16_lo(w[2 * k]) * inv, bf16_hi(w[2 * k]) * inv, bf16_lo(w[2 * k + 1]) * inv,
                       bf16_hi(w[2 * k + 1]) * inv, hi[k], lo[k]);
        constexpr int kLoChunk = kHd == 128 ? 0 : 4, kLoTile = kHd == 128 ? kTile * 128 : 0;
        uint8_t* to = q_tile + row * 128;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (k > 0 && !quarters) break;
          *reinterpret_cast<uint4*>(to + k * 32 * 128 + ((ch ^ (row % 8)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(to + k * 32 * 128 + kLoTile + (((ch + kLoChunk) ^ (row % 8)) << 4)) =
              make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        if (ch == 0) q_exp[row] = static_cast<int8_t>(e);
      }
    }
  }
}

// Eight codes to eight f16 values.
__device__ __forceinline__ uint4 to_f16(uint2 x) {
  return make_uint4(e4m3x2_to_f16x2(x.x), e4m3x2_to_f16x2(x.x >> 16), e4m3x2_to_f16x2(x.y), e4m3x2_to_f16x2(x.y >> 16));
}

template <int kHd, bool kRows>
__global__ void __launch_bounds__(kThreads, 1)
    ragged_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ Params p) {
  using L = Lay<kHd, kRows>;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzle's unit; there is no other shared memory
  Control<kHd, kRows>* sm = reinterpret_cast<Control<kHd, kRows>*>(smem + L::kOffCtl);
  const Waits waits{&sm->abort_flag, p.wait_limit}, to_the_end{&sm->never, p.wait_limit};
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int unit = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kKs; ++i) {
      mbar_init(&sm->k_full[i], 1);
      mbar_init(&sm->k_empty[i], 1);  // commits
    }
    for (int i = 0; i < L::kVs; ++i) {
      mbar_init(&sm->v_full[i], kRows ? 33 : 1);  // the bytes' arrival (+ the scales: one per lane)
      mbar_init(&sm->v_empty[i], 4);              // converter warps
    }
    for (int i = 0; i < L::kFs; ++i) {
      mbar_init(&sm->f_full[i], 4);
      mbar_init(&sm->f_empty[i], 1);  // commits
    }
    for (int i = 0; i < L::kScls; ++i) mbar_init(&sm->scl_full[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->s_full[i], 1);
      mbar_init(&sm->p_full[i], 8);
      mbar_init(&sm->o_full[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sm->item_full[i], 1);
      mbar_init(&sm->item_empty[i], kItemWarps);
    }
    mbar_init(&sm->q_full, 4);  // converter warps
    mbar_init(&sm->q_seen, 8);  // softmax warps: its exponents read
    mbar_init(&sm->q_empty, 1);
    mbar_init(&sm->pv_done, 1);
    mbar_init(&sm->xchg, 8);
    mbar_init(&sm->final_mma, 1);
    sm->abort_flag = sm->never = 0;
    sm->sums_read = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(&sm->tmem_base, 512);
    tmem_relinquish();
  }
  // what the first steps need of the arguments, while the previous kernel ends
  asm volatile("" ::"l"(p.list[0].starts), "l"(p.list[1].lens), "r"(p.page_shift), "l"(p.lo), "l"(p.q_tok),
               "l"(p.plane_o[1]));
  griddep_wait();  // inputs may come from the previous kernel in the stream
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  // the item of number n, or none: every warp's own count
  auto get_item = [&](uint32_t n) -> const Item* {
    if (!warp_wait_item(&sm->item_full[n % kItems], (n / kItems) & 1, waits)) return nullptr;
    const Item* it = &sm->item[n % kItems];
    return it->end ? nullptr : it;
  };
  auto drop_item = [&](uint32_t n) { warp_arrive(&sm->item_empty[n % kItems]); };
  // TMEM columns: S of either stream or tile parity, then O of either stream (one stream: P behind O)
  constexpr uint32_t kTS = 0, kTO = 256;

  if (warp < 8) {
    more_registers<kSoftmaxRegs>();
    // ------------------------------------------------ softmax, epilogue --
    const int wg = warp / 4, w = warp % 4;
    const int r = w * 32 + lane;  // TMEM lane: row of the stream
    const uint32_t lanes = tmem + (static_cast<uint32_t>(w * 32) << 16);
    const float c0 = p.softmax_scale * kLog2e * (kRows ? 1.f : __ldg(p.k_scale));
    uint32_t s_phase = 0, o_phase = 0;  // a bit per barrier
    uint32_t worked = 0, pv_base = 0, tile_no = 0, xchgs = 0;
    int was = -1;
    auto exchange = [&]() -> bool {
      warp_arrive(&sm->xchg);
      return warp_wait(&sm->xchg, xchgs++ & 1, waits);
    };
    for (uint32_t n = 0;; ++n) {
      const Item* it = get_item(n);
      if (it == nullptr) break;
      const int tiles = it->tile_hi - it->tile_lo, form = it->form;
      const bool pair = form == kFormPair, few = form == kFormFew;
      const int row = pair ? wg * kTile + r : (few ? lane : r);  // of the item
      const bool live = row < it->rows;
      const bool busy = __any_sync(0xffffffffu, live);
      float ref = kNegInf, l = 0.f, cc = 1.f;
      [[maybe_unused]] bool apart = false;  // a tile's V scales were far from one (the same in all warps)
      if (tiles > 0) {
        if (!warp_wait(&sm->q_full, worked & 1, waits)) break;
        if (form != was) {
          if (was >= 0 && !exchange()) break;  // the other form's columns are free
          if (few) {               // P: a quarter's own keys alone are written, the others stay zero
            const uint32_t none[32] = {};
            tmem_st32(lanes + kTO + 128 + wg * 64, none);
            tmem_st32(lanes + kTO + 128 + wg * 64 + 32, none);
            tmem_st_wait();
            tc_fence_before();
            if (!exchange()) break;
          }
        }
        was = form;
        const float c = c0 * (live ? exp2i(sm->q_exp[pair ? wg : 0][few ? lane : r]) : 1.f);
        warp_arrive(&sm->q_seen);
        if (!kRows) cc = c;  // units of the reference to log2
        int keys = it->keys - it->tile_lo * kTile;  // left
        auto steps = [&](auto which) {
          constexpr bool kPair = decltype(which)::value;
          constexpr int kOCols = kPair ? kHd : kHd / 2;  // of O that it rescales
          const uint32_t t_o = lanes + kTO + wg * (kPair ? 128 : kOCols);
          // one stream: either warpgroup's columns, of the quarter's 32 where the rows lie in all quarters
          const int cols = few ? 16 : 64, col0 = (few ? w * 32 : 0) + wg * cols, end0 = few ? w * 32 + 32 : 128;
          // O and l follow a new reference.
          auto rescale = [&](int i, float alpha) -> bool {
            if (!kPair && !warp_wait(&sm->pv_done, (pv_base + i - 1) & 1, waits)) return false;
            tc_fence_after();
            if (!kRows || !apart) l *= alpha;
#pragma unroll 1
            for (int k = 0; k < kOCols; k += 16) {
              uint32_t o[16];
              tmem_ld16(t_o + k, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tmem_st16(t_o + k, o);
            }
            return true;
          };
#pragma unroll 1
          for (int i = 0; i < tiles; ++i, keys -= kTile) {
            const int buf = kPair ? wg : (i & 1);
            if (kRows && !warp_wait(&sm->scl_full[tile_no % L::kScls], (tile_no / L::kScls) & 1, waits)) return false;
            [[maybe_unused]] const bool first = !apart;
            if constexpr (kRows)  // (before the wait for S, which hides it)
              apart = apart || *reinterpret_cast<const volatile uint32_t*>(sm->scl_far[tile_no % L::kScls]) != 0;
            if (!warp_wait(&sm->s_full[buf], (s_phase >> buf) & 1, waits)) return false;
            s_phase ^= 1u << buf;
            if (busy) {
              const uint32_t t_s = lanes + kTS + buf * 128;
              const uint32_t t_p = kPair ? t_s : lanes + kTO + 128 + buf * 64;
              tc_fence_after();
              [[maybe_unused]] const float4* kl = sm->scl_k[kRows ? tile_no % L::kScls : 0];
              [[maybe_unused]] const float* iv = sm->scl_v[kRows ? tile_no % L::kScls : 0];
              if (keys < kTile) {  // scores past the end (either warpgroup writes all of them)
                int k = keys;
                const uint32_t none[8] = {kNone, kNone, kNone, kNone, kNone, kNone, kNone, kNone};
#pragma unroll 1
                for (; k % 8 != 0; ++k) tmem_st1(t_s + k, kNone);
#pragma unroll 1
                for (; k < kTile; k += 8) tmem_st8(t_s + k, none);
                tmem_st_wait();
              }
              if constexpr (kRows) {
                if (apart) {  // the sum from the scores alone
                  uint32_t y[16];
                  auto raw = [&](int at) {
                    tmem_ld16(t_s + at, y);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                      const float4 a = kl[(at + j) / 2];
                      const float2 z = make_float2(__uint_as_float(y[j]), __uint_as_float(y[j + 1]));
                      const float2 u = mul_f32x2(mul_f32x2(z, make_float2(c, c)), make_float2(a.x, a.y));
                      y[j] = __float_as_uint(u.x), y[j + 1] = __float_as_uint(u.y);
                    }
                  };
                  // until now l was relative to the reference, which no score passed by more than 48 (both warpgroups
                  // find the same, whatever their own keys' weights)
                  volatile float* top_score = &sm->row_l[wg][r];
                  float was_top = i > 0 ? ref : kNegInf;
                  if (!first) was_top = *top_score;
                  float top = was_top;
#pragma unroll 1
                  for (int at = kPair ? 0 : end0 - 2 * cols; at < (kPair ? kTile : end0); at += 16) {
                    raw(at);
#pragma unroll
                    for (int j = 0; j < 16; ++j) top = fmaxf(top, __uint_as_float(y[j]));
                  }
                  if (top != was_top) l *= ex2_approx(was_top - top);
                  *top_score = top;
                  const float by = top == kNegInf ? 0.f : top;
#pragma unroll 1
                  for (int at = kPair ? 0 : col0; at < (kPair ? kTile : col0 + cols); at += 16) {
                    raw(at);
#pragma unroll
                    for (int j = 0; j < 16; ++j) l += ex2_approx(__uint_as_float(y[j]) - by + kLift);
                  }
                }
              }
              constexpr int kChunk = kPair ? kTile : 16;
              float x[kChunk];
              // scores of column `at` on; with row scales in log2, times their key's K scale and its V scale
              auto scores = [&](int at) {
                if constexpr (kPair) {
#pragma unroll
                  for (int k = 0; k < kChunk; k += 32) tmem_ld32(t_s + k, *reinterpret_cast<uint32_t(*)[32]>(x + k));
                } else {
                  tmem_ld16(t_s + at, *reinterpret_cast<uint32_t(*)[16]>(x));
                }
                tmem_ld_wait();
                if constexpr (kRows) {
#pragma unroll
                  for (int j = 0; j < kChunk; j += 2) {
                    const float4 a = kl[(at + j) / 2];
                    const float2 u = fma_f32x2(mul_f32x2(make_float2(x[j], x[j + 1]), make_float2(c, c)),
                                               make_float2(a.x, a.y), make_float2(a.z, a.w));
                    x[j] = u.x, x[j + 1] = u.y;
                  }
                }
              };
              auto largest = [&](float top) {
                float m0 = x[0], m1 = x[1];
#pragma unroll
                for (int j = 2; j + 4 <= kChunk; j += 4) m0 = fmax3(m0, x[j], x[j + 1]), m1 = fmax3(m1, x[j + 2], x[j + 3]);
                return fmax3(fmax3(top, m0, m1), x[kChunk - 2], x[kChunk - 1]);
              };
              auto subtract = [&](float by) {
#pragma unroll
                for (int j = 0; j < kChunk; j += 2) {
                  const float2 d = add_f32x2(make_float2(x[j], x[j + 1]), make_float2(-by, -by));
                  x[j] = d.x, x[j + 1] = d.y;
                }
              };
              // P = 2^(x cc + bias) to column `at` on, and the sum of the weights.  bias = lift - ref cc, in one
              // operation where the product is small enough for the sum to keep its fraction; else (far) x holds the
              // differences to the reference
              float bias;
              auto weigh = [&](int at) -> float {
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                constexpr int kPut = kPair ? 32 : 16;
#pragma unroll
                for (int k = 0; k < kChunk; k += kPut) {
                  uint32_t h[kPut / 2];
#pragma unroll
                  for (int j = 0; j < kPut; j += 4) {
                    float2 d[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                      const float2 xx = make_float2(x[k + j + 2 * e], x[k + j + 2 * e + 1]);
                      if constexpr (kRows)
                        d[e] = add_f32x2(xx, make_float2(bias, bias));
                      else
                        d[e] = fma_f32x2(xx, make_float2(cc, cc), make_float2(bias, bias));
                      d[e].x = ex2_approx(d[e].x);
                      d[e].y = ex2_approx(d[e].y);
                      h[j / 2 + e] = pack_f16x2(d[e].x, d[e].y);
                    }
                    if constexpr (kRows) {
                      const float4 v = *reinterpret_cast<const float4*>(iv + at + k + j);
                      sum[0] = fma_f32x2(d[0], make_float2(v.x, v.y), sum[0]);
                      sum[1] = fma_f32x2(d[1], make_float2(v.z, v.w), sum[1]);
                    } else {
                      sum[0] = add_f32x2(sum[0], d[0]);
                      sum[1] = add_f32x2(sum[1], d[1]);
                    }
                  }
                  if constexpr (kPair)
                    tmem_st16(t_p + k / 2, h);
                  else
                    tmem_st8(t_p + at / 2, h);
                }
                return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
              };
              if constexpr (kPair) {
                scores(0);
                bool far = fabsf(ref * cc) > kFar && i > 0, less = false;  // less: x holds differences
                // Without row scales no maximum is taken: 128 weights of scores up to the reference sum to 2^14 at most.
                // Where they sum to more than 2^15 (one past the reference by more than 8 does), the reference moves and
                // they are weighed again.
                bool look = kRows || i == 0;
#pragma unroll 1
                for (bool again = false;;) {
                  float by = far && !less ? ref : 0.f;
                  if (look) {
                    const float top = largest(kNegInf);
                    const float step = i == 0 || less ? top : top - ref;  // of the reference, where it moves
                    const bool raise = i > 0 && step * cc > (again ? 0.f : kTau);
                    if (i > 0 && __any_sync(0xffffffffu, raise && live) &&
                        !rescale(i, raise ? ex2_approx(-step * cc) : 1.f))
                      return false;
                    if (i == 0) ref = top == kNegInf ? (kRows ? kNoRef : 0.f) : top;
                    if (raise) ref = less ? ref + top : top;
                    far = less || fabsf(ref * cc) > kFar;
                    by = !far ? 0.f : (less ? (raise ? top : 0.f) : ref);
                  }
                  if (__any_sync(0xffffffffu, by != 0.f)) subtract(by);
                  less = far;
                  bias = far ? kLift : kLift - ref * cc;
                  const float add = weigh(0);
                  if (look || !__any_sync(0xffffffffu, live && !(add <= 32768.f))) {
                    if (!kRows || !apart) l += add;
                    break;
                  }
                  look = again = true;
                }
              } else {
                float top = kNegInf;
#pragma unroll 1
                for (int at = end0 - 2 * cols; at < end0; at += 16) {  // both warpgroups' columns
                  scores(at);
                  top = largest(top);
                }
                const bool raise = (top - ref) * cc > kTau;
                if (i == 0) {
                  ref = top == kNegInf ? (kRows ? kNoRef : 0.f) : top;
                } else if (__any_sync(0xffffffffu, raise && live)) {
                  if (!rescale(i, raise ? ex2_approx((ref - top) * cc) : 1.f)) return false;
                  if (raise) ref = top;
                }
                const bool far = fabsf(ref * cc) > kFar;
                bias = far ? kLift : kLift - ref * cc;
#pragma unroll 1
                for (int at = col0; at < col0 + cols; at += 16) {
                  scores(at);
                  subtract(far ? ref : 0.f);
                  const float add = weigh(at);
                  if (!kRows || !apart) l += add;
                }
              }
              tmem_st_wait();
              tc_fence_before();
            }
            ++tile_no;
            warp_arrive(&sm->p_full[buf]);
            if (kPair && lane == 0) mbar_arrive(&sm->p_full[buf]);  // the barrier counts eight warps
          }
          return true;
        };
        if (!(pair ? steps(std::true_type{}) : steps(std::false_type{}))) break;
        if (pair)
          s_phase ^= (tiles & 1) << (1 - wg);
        else
          pv_base += tiles;
      }
      // Where the results of a row go: rounded to the outputs (kDirect), or as they are to the workspace.  A thread has
      // its lane's row, or (split: the rows lie in all quarters) four dims of row threadIdx.x / 8 at a time.
      const bool split = few && tiles > 0, direct = it->slot == kDirect;
      const int put_row = split ? threadIdx.x / 8 : row;
      const bool put = put_row < it->rows && (split || !few || w == 0);
      const uint32_t rr = static_cast<uint32_t>(it->row0 + put_row), tok = fast_div(rr, p.group);
      const int head = it->head * static_cast<int>(p.group.d) + static_cast<int>(rr - tok * p.group.d);
      const long long token = it->t0 + static_cast<long long>(tok), at = token * p.h_q + head;
      const long long place = it->slot >= 0 ? static_cast<long long>(it->slot) * p.slot_rows + put_row : at;
      uint16_t* out = p.out + token * p.o_tok + head * p.o_head;
      float* sums = (it->slot >= 0 ? p.slot_o : p.plane_o[it->list]) + place * kHd;
      float m = ref * cc, sum = l, part[4];
      // apart: O, relative to the reference, follows the sum (in two steps: either of them stays in float32's range)
      [[maybe_unused]] float half = 1.f;
      if (kRows && apart) {
        const float top_score = sm->row_l[wg][r];
        if (top_score != kNegInf) m = top_score, half = ex2_approx(0.5f * (ref - top_score));
      }
      if (split) {
        sm->row_l[wg][r] = l;
        if (wg == 0) sm->row_m[r] = m;
        if (!exchange()) break;
        m = kNegInf;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          part[k] = sm->row_l[0][k * 32 + put_row] + sm->row_l[1][k * 32 + put_row];
          if (!(part[k] == 0.f)) m = fmaxf(m, sm->row_m[k * 32 + put_row]);
        }
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float f = part[k] == 0.f ? 0.f : ex2_approx(sm->row_m[k * 32 + put_row] - m);
          sum += part[k] * f;
          part[k] = f;
        }
      } else if (form == kFormOne && tiles > 0) {  // either warpgroup has half the keys' weights
        sm->row_l[wg][r] = l;
        if (!exchange()) break;
        sum = sm->row_l[0][r] + sm->row_l[1][r];
        if (!exchange()) break;  // read before the next item's are written
      }
      if (put && (split ? threadIdx.x % 8 == 0 : pair || wg == 0)) {
        if (direct)  // a sequence without keys: -inf
          p.lse[at] = tiles > 0 ? (m + lg2_approx(sum) - kLift) * kLn2 : kNegInf;
        else
          (it->slot >= 0 ? p.slot_ml : p.plane_ml[it->list])[place] = make_float2(m, sum);
      }
      [[maybe_unused]] auto follow = [&](uint32_t (&o)[32]) {
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * half * half);
      };
      const float unit_o = !direct ? 1.f : (tiles > 0 ? (kRows ? 1.f : __ldg(p.v_scale)) / sum : 0.f);
      const int os = pair ? wg : 0;
      if (tiles > 0) {
        ++worked;
        if (!warp_wait(&sm->o_full[os], (o_phase >> os) & 1, waits)) break;
        o_phase ^= pair ? 3u : 1u;
        tc_fence_after();
      }
      if (split) {
        // the quarters' sums [half][quarter][row][dims], 16 bytes swizzled: as many dims at a time as there is room for
        const int rows = kHd == 128 && it->rows <= 16 ? 16 : 32, dims = 1024 / rows;
        float* quarters = reinterpret_cast<float*>(smem + L::kOffSum);
        bool ok = true;
#pragma unroll 1
        for (int k0 = 0; ok && k0 < kHd / 2; k0 += dims) {
#pragma unroll 1
          for (int k = 0; k < dims; k += 32) {
            uint32_t o[32];
            __syncwarp();
            tmem_ld32(lanes + kTO + wg * (kHd / 2) + k0 + k, o);
            tmem_ld_wait();
            if (kRows && apart) follow(o);
            float* to = quarters + ((wg * 4 + w) * rows + lane) * dims + k;
            if (live) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                *reinterpret_cast<uint4*>(to + ((j ^ (lane % 8)) * 4)) =
                    make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
          }
          ok = exchange();
          if (ok && put) {
#pragma unroll 1
            for (int k = 0; k < 2 * dims; k += 32) {  // either half's dims
              const int half = k >= dims ? 1 : 0, in = k - half * dims;
              float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float4 b = *reinterpret_cast<const float4*>(
                    quarters + ((half * 4 + q) * rows + put_row) * dims + in + (((threadIdx.x ^ put_row) % 8) * 4));
                a.x += b.x * part[q], a.y += b.y * part[q], a.z += b.z * part[q], a.w += b.w * part[q];
              }
              const int dim = half * (kHd / 2) + k0 + in + (threadIdx.x % 8) * 4;
              if (direct)
                *reinterpret_cast<uint2*>(out + dim) = make_uint2(pack_bf16x2(a.x * unit_o, a.y * unit_o),
                                                                  pack_bf16x2(a.z * unit_o, a.w * unit_o));
              else
                *reinterpret_cast<float4*>(sums + dim) = a;
            }
          }
          if (ok && k0 + dims < kHd / 2) ok = exchange();  // read before the next are written
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) {
          __threadfence_block();
          atomicAdd(&sm->sums_read, 1u);
        }
      } else if (busy) {
        const int dims = pair ? kHd : kHd / 2, dim0 = pair ? 0 : wg * (kHd / 2);
#pragma unroll 1
        for (int k = dim0; k < dim0 + dims; k += 32) {
          uint32_t o[32] = {};
          __syncwarp();
          if (tiles > 0) {
            tmem_ld32(lanes + kTO + os * 128 + k, o);
            tmem_ld_wait();
            if (kRows && apart) follow(o);
          }
          if (!put) continue;
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            if (direct) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                h[e] = pack_bf16x2(__uint_as_float(o[j + 2 * e]) * unit_o, __uint_as_float(o[j + 2 * e + 1]) * unit_o);
              *reinterpret_cast<uint4*>(out + k + j) = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
              *reinterpret_cast<uint4*>(sums + k + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
              *reinterpret_cast<uint4*>(sums + k + j + 4) = make_uint4(o[j + 4], o[j + 5], o[j + 6], o[j + 7]);
            }
          }
        }
      }
      __syncwarp();
      tc_fence_before();
      drop_item(n);
    }
  } else if (warp < 12) {
    fewer_registers<kConvertRegs>();
    // ---------------------------------------------- V's codes to f16 tiles --
    // A thread takes eight codes of every eighth (hd 64: sixteenth) row: 16 bytes of f16 at a place of the swizzled row
    // that is the same each time, and the quarters of a warp meet every bank once.
    const int tid = threadIdx.x - 256;
    constexpr int kLanes = kHd / 8, kRowsAStep = 128 / kLanes, kSteps = kTile / kRowsAStep;
    const int key0 = tid / kLanes, ch = tid % kLanes;
    const uint32_t from = kHd == 128 ? key0 * 128 + (((ch / 2) ^ (key0 % 8)) << 4) + (ch % 2) * 8
                                     : key0 * 64 + (((ch / 2) ^ ((key0 / 2) % 4)) << 4) + (ch % 2) * 8;
    const uint32_t to = (ch / 8) * (kTile * 128) + key0 * 128 + (((ch % 8) ^ (key0 % 8)) << 4);
    uint32_t done = 0, vs = 0, v_phase = 0, fs = 0, f_phase = 1, worked = 0, sums = 0;
    bool ok = true;
    for (uint32_t n = 0; ok; ++n) {
      const Item* it = get_item(n);
      if (it == nullptr) break;
      const int tiles = it->tile_hi - it->tile_lo;
      if (tiles > 0) {
        // Q, once the products have left the one before, and the softmax has seen it (else it would miss a phase)
        const int form = it->form, w = warp - 8;
        if (worked > 0 && (!warp_wait(&sm->q_empty, (worked - 1) & 1, waits) ||
                           !warp_wait(&sm->q_seen, (worked - 1) & 1, waits)))
          break;
        if (kHd == 128 && form == kFormPair && !wait_count(&sm->sums_read, sums, waits)) break;  // they lie there
        int8_t* q_exp = sm->q_exp[0];
        const int stream = form == kFormPair ? w / 2 : 0;
        const int count = form == kFormPair ? 64 : (form == kFormOne ? 32 : 8);  // a warp's rows
        load_q<kHd>(p, *it, smem + stream * L::kQ, q_exp + stream * kTile, stream * kTile,
                    (form == kFormPair ? w % 2 : w) * count, count, form == kFormFew, lane);
        fence_proxy_async_smem();
        warp_arrive(&sm->q_full);
        ++worked;
        if (form == kFormFew) sums += 8;
      }
      int valid = it->keys - it->tile_lo * kTile;
      drop_item(n);
      for (int i = 0; i < tiles; ++i, ++done, valid -= kTile) {
        ok = false;
        if (!warp_wait(&sm->v_full[vs], v_phase, waits)) break;
        if constexpr (kRows) {  // past the end: one, so that a stale scale cannot turn a zero weight into a NaN
          const float a = tid < valid ? sm->raw_scl[vs][0][tid] : 1.f, b = tid < valid ? sm->raw_scl[vs][1][tid] : 1.f;
          const int ss = done % L::kScls;
          float* two = reinterpret_cast<float*>(&sm->scl_k[ss][tid / 2]) + tid % 2;
          const bool near = b >= kSmallScale && b <= kLargeScale;
          const bool far = __any_sync(0xffffffffu, !near);
          two[0] = a;
          two[2] = b < 0x1p-126f ? lg2_approx(b * 0x1p64f) - 64.f : lg2_approx(b);
          sm->scl_v[ss][tid] = near ? 1.f / b : 0.f;
          if (lane == 0) sm->scl_far[ss][warp - 8] = far;
          warp_arrive(&sm->scl_full[ss]);
        }
        if (done >= L::kFs && !warp_wait(&sm->f_empty[fs], f_phase, waits)) break;
        const uint8_t* src = smem + L::kOffV + vs * L::kRaw + from;
        uint8_t* dst = smem + L::kOffF + fs * L::kF + to;
#pragma unroll
        for (int k = 0; k < kSteps; k += 8) {
          uint2 x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = *reinterpret_cast<const uint2*>(src + (k + j) * 1024);
          if (valid < kTile) {  // rows past the end: zeros
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (key0 + (k + j) * kRowsAStep >= valid) x[j] = make_uint2(0, 0);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(dst + (k + j) * kRowsAStep * 128) = to_f16(x[j]);
        }
        fence_proxy_async_smem();
        warp_arrive(&sm->f_full[fs]);
        warp_arrive(&sm->v_empty[vs]);
        if (++vs == L::kVs) vs = 0, v_phase ^= 1;
        if (++fs == L::kFs) fs = 0, f_phase ^= 1;
        ok = true;
      }
    }
  } else {
    fewer_registers<kIssueRegs>();
    if (warp == 12) {
      // ------------------------------------------------ matrix products --
      constexpr uint32_t idesc_qk = make_idesc(0, 0, 0, 0, kTile, 128);  // E4M3: Q (K-major) x K (K-major)
      constexpr uint32_t idesc_pv = make_idesc(0, 0, 0, 1, kHd, 128);    // f16: P (TMEM) x V (MN-major)
      const bool leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);  // the same in all lanes, as the compiler sees it
      const uint32_t qb = smem_u32(smem), kb = qb + L::kOffK, fb = qb + L::kOffF;
      uint32_t at = 0, p_phase = 0, worked = 0;  // at: tiles before this item's
      bool ok = true;
      auto wait_k = [&](uint32_t t) { return warp_wait(&sm->k_full[t % L::kKs], (t / L::kKs) & 1, waits); };
      auto wait_v = [&](uint32_t t) { return warp_wait(&sm->f_full[t % L::kFs], (t / L::kFs) & 1, waits); };
      auto wait_p = [&](int buf) {
        const bool done = warp_wait(&sm->p_full[buf], (p_phase >> buf) & 1, waits);
        p_phase ^= 1u << buf;
        return done;
      };
      // (descriptors count in 16 bytes; loops are kept short for the instruction cache)
      const uint64_t q_desc = make_sdesc(qb, 16, 1024, SWIZZLE_128B), k_desc = make_sdesc(kb, 16, 8 * kHd, L::kSwizzle);
      const uint64_t v_desc = make_sdesc(fb, kTile * 128, 1024, SWIZZLE_128B);
      auto issue_qk = [&](int q, int buf, uint32_t t) {  // S[buf] = Q[q] K^T, both terms of Q
        tc_fence_after();
        const uint64_t a = q_desc + q * (L::kQ >> 4), b = k_desc + (t % L::kKs) * (L::kRaw >> 4);
#pragma unroll
        for (int term = 0; term < 2; ++term) {
          const uint64_t at_term = a + term * ((kHd == 128 ? kTile * 128 : 64) >> 4);
#pragma unroll
          for (int kk = 0; kk < kHd / 32; ++kk)
            mma_f8_ss_if(leader, tm + kTS + buf * 128, at_term + 2 * kk, b + 2 * kk, idesc_qk,
                         kk > 0 ? 1u : static_cast<uint32_t>(term));
        }
        tc_commit_if(leader, &sm->s_full[buf]);
      };
      auto issue_pv = [&](uint32_t t_o, uint32_t t_p, uint32_t t, bool fresh) {  // O += P V
        tc_fence_after();
        const uint64_t b = v_desc + (t % L::kFs) * (L::kF >> 4);
#pragma unroll
        for (int k = 0; k < kTile / 16; k += 4) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_ts_if(leader, tm + t_o, tm + t_p + (k + kk) * 8, b + (k + kk) * 128, idesc_pv,
                          (kk > 0 || k > 0 || !fresh) ? 1u : 0u);
        }
      };
      auto free_k = [&](uint32_t t) { tc_commit_if(leader, &sm->k_empty[t % L::kKs]); };
      auto free_v = [&](uint32_t t) { tc_commit_if(leader, &sm->f_empty[t % L::kFs]); };
      for (uint32_t n = 0; ok; ++n) {
        const Item* it = get_item(n);
        if (it == nullptr) break;
        const int tiles = __shfl_sync(0xffffffffu, it->tile_hi - it->tile_lo, 0);
        const bool pair = __shfl_sync(0xffffffffu, it->form, 0) == kFormPair;
        drop_item(n);
        if (tiles == 0) continue;
        ok = false;
        if (!warp_wait(&sm->q_full, worked++ & 1, waits)) break;
        // Operation j is a product with P and one with K two operations ahead, in its buffer: with two streams S(j % 2)
        // and a tile in two operations, with one stream the tile's parity and a tile in each.
        const int per = pair ? 2 : 1, ops = tiles * per;
        int j = -2;
#pragma unroll 1
        for (; j < ops; ++j) {
          const int buf = j & 1;
          if (j >= 0) {
            const int i = pair ? j >> 1 : j, o = pair ? buf : 0;
            const bool starts = !pair || buf == 0, ends = !pair || buf == 1;
            if ((starts && !wait_v(at + i)) || !wait_p(buf)) break;
            issue_pv(kTO + o * 128, pair ? kTS + buf * 128 : kTO + 128 + buf * 64, at + i, i == 0);
            if (!pair) tc_commit_if(leader, &sm->pv_done);
            if (ends) free_v(at + i);
            if (i + 1 == tiles) tc_commit_if(leader, &sm->o_full[o]);
          }
          if (j + 2 < ops) {
            const int i = pair ? (j + 2) >> 1 : j + 2;
            const bool starts = !pair || buf == 0, ends = !pair || buf == 1;
            if (starts && !wait_k(at + i)) break;
            issue_qk(pair ? buf : 0, buf, at + i);
            if (ends) free_k(at + i);
            if (j + 3 == ops) tc_commit_if(leader, &sm->q_empty);
          }
        }
        if (j < ops) break;
        at += tiles;
        ok = true;
      }
      if (leader) tc_commit(&sm->final_mma);
      __syncwarp();
      warp_wait(&sm->final_mma, 0, to_the_end);
    } else if (warp != 14) {
      // -------------------------------------- copies of tiles: 13 K, 15 V --
      const bool is_v = warp == 15;
      const CUtensorMap* map = is_v ? &tm_v : &tm_k;
      const uint32_t ring = is_v ? L::kVs : L::kKs;
      uint64_t* full = is_v ? sm->v_full : sm->k_full;
      uint64_t* empty = is_v ? sm->v_empty : sm->k_empty;
      uint8_t* tiles_at = smem + (is_v ? L::kOffV : L::kOffK);
      const bool leader = elect_one();
      if (leader) tma_prefetch_desc(map);
      const uint32_t fault = unit == 0 && !is_v ? p.fault_tile : 0;
      uint32_t done = 0, slot = 0, phase = 1;
      bool ok = true;
      const int chunk_shift = min(p.page_shift, 7);  // keys a copy
      const int chunks = kTile >> chunk_shift, in_page = (1 << p.page_shift) - 1;
      for (uint32_t n = 0; ok; ++n) {
        const Item* it = get_item(n);
        if (it == nullptr) break;
        const int tile_hi = it->tile_hi, keys = it->keys, head = it->head;
        int tile = it->tile_lo;
        const int32_t* table = p.list[it->list].table + static_cast<long long>(it->seg) * p.list[it->list].max_blocks;
        drop_item(n);
        // lane c: the page of chunk c of a tile
        auto fetch = [&](int t) {
          const int key = t * kTile + (lane << chunk_shift);
          return t < tile_hi && lane < chunks && key < keys ? __ldg(table + (key >> p.page_shift)) : 0;
        };
        int block = fetch(tile), next = fetch(tile + 1);
        for (; tile < tile_hi; ++tile, ++done) {
          if (block < 0 || block >= p.num_blocks) {
            atomicOr(&g_status_ragged, FP8MLA_DEV_BAD_PAGE);
            block = 0;
          }
          if (done >= ring && !warp_wait(empty + slot, phase, waits)) {
            ok = false;
            break;
          }
          const int valid = min(kTile, keys - tile * kTile);
          // whole pages, or 128 keys of one
          const int copies = done + 1 == fault ? 0 : ((valid - 1) >> chunk_shift) + 1;
          if (leader && copies > 0) mbar_arrive_expect_tx(full + slot, static_cast<uint32_t>(copies) * (kHd << chunk_shift));
          const int row = ((block * p.h_kv + head) << p.page_shift) + ((tile * kTile) & in_page);
          uint8_t* to = tiles_at + slot * L::kRaw;
#pragma unroll 1
          for (int c = 0; c < copies; ++c) {
            const int from = __shfl_sync(0xffffffffu, row, c);
            if (leader) tma_load_3d(to + c * (kHd << chunk_shift), map, full + slot, 0, from, 0);
          }
          if constexpr (kRows) {
            if (is_v) {  // scales of four keys a lane
              const int key = lane * 4;
              const int from = __shfl_sync(0xffffffffu, row, key >> chunk_shift);
              const int at4 = from + (key & ((1 << chunk_shift) - 1));
              if (key < valid) {
                cp_async16(smem_u32(&sm->raw_scl[slot][0][key]), p.k_scale + at4, 16u);
                cp_async16(smem_u32(&sm->raw_scl[slot][1][key]), p.v_scale + at4, 16u);
              }
              cp_async_mbar_arrive(full + slot);
            }
          }
          block = next;
          next = fetch(tile + 2);
          if (++slot == ring) slot = 0, phase ^= 1;
        }
      }
      if constexpr (kRows) cp_async_wait_all();  // this lane's copies have landed before the CTA can exit
#pragma unroll 1
      for (uint32_t j = done > ring ? done - ring : 0; j < done; ++j)
        if (j + 1 != fault) warp_wait(full + j % ring, (j / ring) & 1, to_the_end);
    } else if (warp == 14) {
      // ------------------------------------------------- the share's items --
      const bool fits = find_share(p, unit, &sm->walk, sm->group_at);
      bool more = true;
#pragma unroll 1
      for (uint32_t n = 0; more; ++n) {
        if (n >= kItems && !warp_wait_item(&sm->item_empty[n % kItems], (n / kItems - 1) & 1, waits)) break;
        Item* it = &sm->item[n % kItems];
        if (lane == 0) it->end = !next_item(p, unit, &sm->walk, it);
        __syncwarp();
        more = !it->end;
        warp_arrive(&sm->item_full[n % kItems]);
      }
      // and rows of no sequence
      if (p.fill_out || p.fill_lse) {
        const List& l = p.list[0];
        auto fill = [&](int t, int h) {
          if (p.fill_out && lane < kHd / 8)
            *reinterpret_cast<uint4*>(p.out + t * p.o_tok + h * p.o_head + lane * 8) = make_uint4(0, 0, 0, 0);
          if (p.fill_lse && lane == 0) p.lse[static_cast<long long>(t) * p.h_q + h] = kNegInf;
        };
        if (fits) {  // those in front of the first one and behind the last
          const int lo = l.starts ? min(max(__ldg(l.starts), 0), p.tokens) : 0;
          const int hi = l.starts ? min(max(__ldg(l.starts + l.n), lo), p.tokens) : min(l.n, p.tokens);
          const uint32_t heads = static_cast<uint32_t>(lo + p.tokens - hi) * p.h_q;
#pragma unroll 1
          for (uint32_t i = unit; i < heads; i += gridDim.x) {
            int t = static_cast<int>(i / p.h_q);
            const int h = static_cast<int>(i - t * p.h_q);
            if (t >= lo) t += hi - lo;
            fill(t, h);
          }
        } else {  // those that no segment has, a bit each: 32 kWords a lane at a time, while all segments pass by
          constexpr int kWords = 4, kTokens = 32 * 32 * kWords;
#pragma unroll 1
          for (int t0 = unit * kTokens; t0 < p.tokens; t0 += gridDim.x * kTokens) {
            uint32_t has[kWords] = {};
#pragma unroll 1
            for (int s0 = 0; s0 < l.n; s0 += 32) {
              const int s = min(s0 + lane, l.n - 1);
              const int a = __ldg(l.starts + s), b = __ldg(l.starts + s + 1);
              uint32_t here = __ballot_sync(0xffffffffu, range_ok(l, a, b) && a < t0 + kTokens && b > t0);
#pragma unroll 1
              for (; here != 0; here &= here - 1) {
                const int from = __shfl_sync(0xffffffffu, a, __ffs(here) - 1), to = __shfl_sync(0xffffffffu, b, __ffs(here) - 1);
#pragma unroll
                for (int k = 0; k < kWords; ++k) {
                  const int first = t0 + (k * 32 + lane) * 32, lo = max(from - first, 0), hi = min(to - first, 32);
                  if (lo < hi) has[k] |= (~0u << lo) & (~0u >> (32 - hi));
                }
              }
            }
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
#pragma unroll 1
              for (int src = 0; src < 32; ++src) {
                uint32_t without = ~__shfl_sync(0xffffffffu, has[k], src);
#pragma unroll 1
                for (; without != 0; without &= without - 1) {
                  const int t = t0 + (k * 32 + src) * 32 + __ffs(without) - 1;
                  if (t >= p.tokens) break;
#pragma unroll 1
                  for (int h = 0; h < p.h_q; ++h) fill(t, h);
                }
              }
            }
          }
        }
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && (sm->abort_flag | sm->never) != 0) atomicOr(&g_status_ragged, FP8MLA_DEV_WAIT_TIMEOUT);
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ merges --
//
// exp2(m_i - m) weighs the pieces' sums and rows, m their largest reference.  Bound by latency: the pieces were just
// written and lie in L2, so what counts is that all of a row's pieces are asked for at once (a lane holds one piece's
// weight and tells it to the others; prompts 49 -> 39 us), the pieces of a row's prefix with those of its own keys, and
// that the code is short (shared_merge 22 KB -> 15: shared batch 82 -> 80 us).  Cold under a profiler cross_merge takes 5
// to 6 us, shared_merge 8 (128 rows) to 16 (6144 with blocks of four keys).

constexpr int kMergeThreads = 128;
// Lanes a row: eight where an item's 256 rows are merged, few pieces each.  Behind shared prefixes four dims a lane where
// rows are few and their prefix lies in many pieces (2048 rows of 12 pieces: a call 80 us, with eight dims 85), eight
// where at four the thread blocks would not all be resident, eight on each of 152 SMs, 32 rows of 128 dims an SM (6144 and
// 8192 rows: 96 -> 91 us, 137 -> 134).
constexpr int kCrossRows = kMergeThreads / 8;
template <int kHd, int kV>
constexpr int kSharedRows = kMergeThreads * kV / kHd;

// A row's share of an item's pieces, in `count` shares from `first` on: the first in slot `slot` of its share, the others
// in slot 0, in row `row` of the slot; an item of one share that is whole lies in row `row` of a plane (ml, o) instead.
struct Pieces {
  int first = 0, count = 0, slot = 0, row = 0;
  const float2* ml = nullptr;
  const float* o = nullptr;
};

// A row's sum, by kLanes lanes: lane d of them owns dims [kV d, kV d + kV).
template <int kHd, int kLanes>
struct RowSum {
  static constexpr int kV = kHd / kLanes;
  static constexpr int kBatch = kV == 16 ? 2 : 4;  // pieces in flight
  float m = kNegInf, l = 0.f, acc[kV] = {};

  // Adds the pieces of up to two items (all lanes of the warp together).  lo: where the shares begin.
  __device__ __forceinline__ void add(const Params& p, const long long* lo, const Pieces& x, const Pieces& y, int d) {
    const int count = x.count + y.count;
    const int most = __reduce_max_sync(0xffffffffu, count);
#pragma unroll 1
    for (int base = 0; base < most; base += kLanes) {
      // a lane's piece
      const int i = base + d;
      const bool second = i >= x.count;
      const int j = second ? i - x.count : i, v = (second ? y.first : x.first) + j;
      const float* plane = second ? y.o : x.o;
      bool ok = i < count;
      if (ok && plane == nullptr && j > 0 && lo[v + 1] <= lo[v]) ok = false;  // a share without work
      const long long idx = plane != nullptr ? (second ? y.row : x.row)
                                             : (2 * v + (j == 0 ? (second ? y.slot : x.slot) : 0)) * p.slot_rows +
                                                   (second ? y.row : x.row);
      const float* at = (plane != nullptr ? plane : p.slot_o) + idx * kHd;
      float2 ml = make_float2(kNegInf, 0.f);
      if (ok) ml = (plane != nullptr ? (second ? y.ml : x.ml) : p.slot_ml)[idx];
      float top = fmaxf(m, ml.x);
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float a = top == kNegInf ? 1.f : ex2_approx(m - top);
      const float w = ok && top != kNegInf ? ex2_approx(ml.x - top) : 0.f;
      float add_l = ok ? w * ml.y : 0.f;
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) add_l += __shfl_xor_sync(0xffffffffu, add_l, o);
      m = top;
      l = l * a + add_l;
#pragma unroll
      for (int i = 0; i < kV; ++i) acc[i] *= a;
      // batches without a remainder, as long code comes from memory in every launch
      const uint32_t there = __ballot_sync(0xffffffffu, ok) >> (threadIdx.x % 32 - d);
      const int n = min(kLanes, most - base);
#pragma unroll 1
      for (int q = 0; q < n; q += kBatch) {
        float4 z[kBatch][kV / 4];
        float wq[kBatch];
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
          wq[e] = __shfl_sync(0xffffffffu, w, q + e, kLanes);
          const unsigned long long from = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(at), q + e, kLanes);
#pragma unroll
          for (int i = 0; i < kV / 4; ++i) {
            z[e][i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if ((there >> (q + e)) & 1) z[e][i] = __ldcg(reinterpret_cast<const float4*>(from) + d * (kV / 4) + i);
          }
        }
#pragma unroll
        for (int e = 0; e < kBatch; ++e) {
#pragma unroll
          for (int i = 0; i < kV / 4; ++i) {
            acc[4 * i] += z[e][i].x * wq[e], acc[4 * i + 1] += z[e][i].y * wq[e];
            acc[4 * i + 2] += z[e][i].z * wq[e], acc[4 * i + 3] += z[e][i].w * wq[e];
          }
        }
      }
    }
  }
  __device__ __forceinline__ void finish(uint16_t* out, float* lse, float sink, float v_scale, int d) {
    float f, ls;
    finish_row(m - kLift, l, sink, v_scale, &f, &ls);
    if (l != l) f = ls = l;  // NaN
#pragma unroll
    for (int i = 0; i < kV; i += 4)
      *reinterpret_cast<uint2*>(out + d * kV + i) =
          make_uint2(pack_bf16x2(acc[i] * f, acc[i + 1] * f), pack_bf16x2(acc[i + 2] * f, acc[i + 3] * f));
    if (d == 0) *lse = ls;
  }
};

// Where the shares begin, in shared memory; how many there are.
__device__ __forceinline__ int load_shares(const Params& p, int grid, long long* lo) {
#pragma unroll 2
  for (int v = threadIdx.x; v <= grid; v += kMergeThreads) lo[v] = p.lo[v];  // (past the last share: anything)
  const int units = *p.units;
  __syncthreads();
  return units;
}

template <int kHd>
__global__ void __launch_bounds__(kMergeThreads, 8) cross_merge_kernel(const __grid_constant__ Params p, int scale_rows) {
  griddep_wait();
  __shared__ long long lo[kMostUnits + 1];
  const int unit = blockIdx.x, row0 = blockIdx.y * kCrossRows;
  const Cut cut = p.cuts[unit];
  const float v_scale = scale_rows ? 1.f : *p.v_scale;
  const int units = load_shares(p, gridDim.x, lo);
  if (unit >= units || cut.valid == 0 || row0 >= cut.rows) return;
  int last = unit;
  while (last + 1 < units && lo[last + 1] < cut.end) ++last;
  const int d = threadIdx.x % 8, row = row0 + threadIdx.x / 8;
  const bool live = row < cut.rows;
  Pieces pieces;
  pieces.first = unit, pieces.count = live ? last - unit + 1 : 0, pieces.slot = cut.slot & 1, pieces.row = row;
  RowSum<kHd, 8> sum;
  sum.add(p, lo, pieces, Pieces(), d);
  if (!live) return;
  const uint32_t r = static_cast<uint32_t>(cut.row0 + row), t = fast_div(r, p.group);
  const int head = cut.head * static_cast<int>(p.group.d) + static_cast<int>(r - t * p.group.d);
  const long long token = cut.t0 + static_cast<long long>(t);
  sum.finish(p.out + token * p.o_tok + head * p.o_head, p.lse + token * p.h_q + head, kNegInf, v_scale, d);
}

// Row = (sequence, KV head, token, head of its group) of a decode step behind shared prefixes: its prefix, its own keys
// before the block, the block's keys that it sees, its sink.
template <int kHd, int kV>
__global__ void __launch_bounds__(kMergeThreads)
    shared_merge_kernel(const __grid_constant__ Params p, int scale_rows, int grid, int total) {
  griddep_wait();
  constexpr int kLanes = kHd / kV;
  __shared__ long long lo[kMostUnits + 1];
  const int d = threadIdx.x % kLanes;
  const int group = static_cast<int>(p.group.d), rows = p.q_len * group;
  // (lanes past the last row compute it again and write nothing: it may lie where Q did)
  const int mine = blockIdx.x * kSharedRows<kHd, kV> + static_cast<int>(threadIdx.x) / kLanes, of_all = min(mine, total - 1);
  const int pair = fast_div(of_all, p.of_rows), row = of_all - pair * rows;
  const int b = fast_div(pair, p.of_heads), kvh = pair - b * p.h_kv;
  const int tok = fast_div(row, p.group), head = kvh * group + row - tok * group;
  const int token = b * p.q_len + tok, at = token * p.h_q + head;
  const float k_scale = scale_rows ? 1.f : *p.k_scale, v_scale = scale_rows ? 1.f : *p.v_scale;
  uint32_t bad = 0;
  const int own = p.list[0].n + b;
  const Bounds own_bounds = load_bounds(p, own);  // (asked for before they are needed, like the prefix's)
  const long long own_at = p.seg_at[own];
  // its prefix (-1: none), looked for by the row's lanes
  int prefix = -1;
#pragma unroll 1
  for (int g0 = 0; g0 < p.list[0].n; g0 += kLanes) {
    const int g = g0 + d;
    if (g < p.list[0].n && prefix < 0) {
      const int first = __ldg(p.list[0].starts + g), end = __ldg(p.list[0].starts + g + 1);
      if (first >= 0 && first <= b && b < end && end <= p.list[0].most) prefix = g;
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) prefix = max(prefix, __shfl_xor_sync(0xffffffffu, prefix, o));
  }
  const int some = max(prefix, 0);
  const Bounds bounds = load_bounds(p, some);  // (without prefixes: a sequence's)
  const long long prefix_at = p.seg_at[some];
  const int units = load_shares(p, grid, lo);
  auto shares_below = [&](long long x) {  // how many begin before x
    int n = 0;
#pragma unroll 1
    for (int step = 256; step > 0; step >>= 1)
      if (n + step <= units && lo[n + step - 1] < x) n += step;
    return n;
  };
  Pieces front, back;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {  // (once: the code is short for the instruction cache)
    if (which == 0 && prefix < 0) continue;
    const Seg g = make_seg(p, which ? own : prefix, which ? own_bounds : bounds, &bad);
    if (g.tiles == 0) continue;
    const int r = (b * p.q_len - g.t0) * group + row, rt = r / kItemRows;
    const long long start = (which ? own_at : prefix_at) + kvh * g.head + static_cast<long long>(rt) * g.full;
    const long long end = start + (rt == g.row_tiles - 1 ? g.last : g.full);
    Pieces y;
    y.first = shares_below(start + 1) - 1;
    y.count = shares_below(end) - y.first;
    y.slot = lo[y.first] == start ? 0 : 1;
    y.row = r - rt * kItemRows;
    if (y.count == 1) y.o = p.plane_o[which], y.ml = p.plane_ml[which], y.row = at;
    if (which)
      back = y;
    else
      front = y;
  }
  RowSum<kHd, kLanes> sum;
  if (p.list[1].less > 0) {  // the block's keys: every lane looks one up, then they are weighed in turn
    const List& l = p.list[1];
    const int len = seg_len(l, own_bounds.len, &bad);
    float q[kV];
#pragma unroll
    for (int i = 0; i < kV; i += 4) {
      const uint2 x = *reinterpret_cast<const uint2*>(p.q + token * p.q_tok + head * p.q_head + d * kV + i);
      q[i] = bf16_lo(x.x), q[i + 1] = bf16_hi(x.x), q[i + 2] = bf16_lo(x.y), q[i + 3] = bf16_hi(x.y);
    }
    const float c = p.softmax_scale * kLog2e * k_scale;
#pragma unroll 1
    for (int x0 = 0; x0 < p.q_len; x0 += kLanes) {
      const int x = x0 + d, key = len - p.q_len + x;
      bool sees = x < p.q_len && key >= 0;
      if (sees)
        sees = p.spec_mask != nullptr ? p.spec_mask[(static_cast<long long>(b) * p.q_len + tok) * p.q_len + x] != 0
                                      : x <= tok;
      int line = 0;
      float sk = 1.f, sv = 1.f;
      if (sees) {
        int block = __ldg(l.table + static_cast<long long>(b) * l.max_blocks + (key >> p.page_shift));
        if (block < 0 || block >= p.num_blocks) {
          atomicOr(&g_status_ragged, FP8MLA_DEV_BAD_PAGE);
          block = 0;
        }
        line = ((block * p.h_kv + kvh) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
        if (scale_rows) sk = __ldg(p.k_scale + line), sv = __ldg(p.v_scale + line);
      }
      const uint32_t seen = __ballot_sync(0xffffffffu, sees) >> (threadIdx.x % 32 - d);
      const int n = min(kLanes, p.q_len - x0);
#pragma unroll 1
      for (int j0 = 0; j0 < n; j0 += 2)
#pragma unroll
      for (int j = j0; j < j0 + 2; ++j) {
        const long long from = __shfl_sync(0xffffffffu, line, j, kLanes) * static_cast<long long>(kHd);
        uint32_t wk[kV / 2], wv[kV / 2];  // (unseen: the cache's first row)
#pragma unroll
        for (int i = 0; i < kV / 4; ++i) {
          const uint4 h = to_f16(make_uint2(__ldg(reinterpret_cast<const uint32_t*>(p.k + from) + d * (kV / 4) + i),
                                            __ldg(reinterpret_cast<const uint32_t*>(p.v + from) + d * (kV / 4) + i)));
          wk[2 * i] = h.x, wk[2 * i + 1] = h.y, wv[2 * i] = h.z, wv[2 * i + 1] = h.w;
        }
        const float skj = __shfl_sync(0xffffffffu, sk, j, kLanes), svj = __shfl_sync(0xffffffffu, sv, j, kLanes);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kV; i += 2) s += q[i] * f16_lo(wk[i / 2]) + q[i + 1] * f16_hi(wk[i / 2]);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        s *= c * skj;
        const float m = s + kLift, top = s == s ? fmaxf(sum.m, m) : fmaxf(sum.m, 0.f);  // the pieces' sums are lifted
        if (!((seen >> j) & 1) || top == kNegInf) continue;
        const float f = ex2_approx(sum.m - top), w = ex2_approx(m - top);
        sum.m = top;
        sum.l = sum.l * f + w;
#pragma unroll
        for (int i = 0; i < kV; i += 2) {
          sum.acc[i] = sum.acc[i] * f + f16_lo(wv[i / 2]) * (w * svj);
          sum.acc[i + 1] = sum.acc[i + 1] * f + f16_hi(wv[i / 2]) * (w * svj);
        }
      }
    }
  }
  sum.add(p, lo, front, back, d);
  if (mine >= total) return;
  sum.finish(p.out + static_cast<long long>(at) * kHd, p.lse + at, p.sinks ? p.sinks[head] : kNegInf, v_scale, d);
}

// -------------------------------------------------------------------- host --

// The test hook's settings by device (limit 0: the default).
constexpr int kMostDevices = 64;
std::atomic<uint32_t> g_wait_limit[kMostDevices], g_fault_tile[kMostDevices];

void use_wait_test(Params* p) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMostDevices) dev = 0;
  const uint32_t limit = g_wait_limit[dev].load(std::memory_order_relaxed);
  p->wait_limit = limit != 0 ? limit : kWaitLimit;
  p->fault_tile = g_fault_tile[dev].load(std::memory_order_relaxed);
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

struct Space {  // the workspace: offsets, and the grid it is for
  int grid, slot_rows;
  size_t units, lo, seg_at, cuts, slot_ml, slot_o, plane_ml[2], plane_o[2], bytes;
};

// tokens and segments of a list that reads up to max_keys keys a segment
double most_work(long long tokens, long long segs, int h_kv, int group, long long max_keys) {
  const long long tiles = (max_keys + kTile - 1) / kTile;
  return static_cast<double>(h_kv) * (tokens * group / kItemRows + segs) * (100 + 52 * std::max(tiles, 1ll));  // at most
}

Space lay_out(double work, long long tokens, int segs, int h_q, int group, int hd, bool joined) {
  Space s;
  s.grid = static_cast<int>(std::max(1.0, std::min<double>(std::min(device_sms(), kMostUnits), work / kLeast)));
  s.slot_rows = static_cast<int>(std::min<long long>(kItemRows, std::max(1ll, tokens * group)));
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  const size_t slots = s.grid > 1 ? static_cast<size_t>(2) * s.grid * s.slot_rows : 0;
  const size_t rows = joined ? static_cast<size_t>(tokens) * h_q : 0;
  s.units = take(256);
  s.lo = take((s.grid + 1) * sizeof(long long));
  s.seg_at = take(joined ? segs * sizeof(long long) : 0);
  s.cuts = take(joined ? 0 : s.grid * sizeof(Cut));
  s.slot_ml = take(slots * sizeof(float2));
  s.slot_o = take(slots * hd * sizeof(float));
  for (int i = 0; i < 2; ++i) {
    s.plane_ml[i] = take(rows * sizeof(float2));
    s.plane_o[i] = take(rows * hd * sizeof(float));
  }
  s.bytes = at;
  return s;
}

void use(Params* p, const Space& s, void* workspace) {
  char* w = static_cast<char*>(workspace);
  p->units = reinterpret_cast<int*>(w + s.units);
  p->lo = reinterpret_cast<long long*>(w + s.lo);
  p->seg_at = reinterpret_cast<long long*>(w + s.seg_at);
  p->cuts = reinterpret_cast<Cut*>(w + s.cuts);
  p->slot_ml = reinterpret_cast<float2*>(w + s.slot_ml);
  p->slot_o = reinterpret_cast<float*>(w + s.slot_o);
  for (int i = 0; i < 2; ++i) {
    p->plane_ml[i] = reinterpret_cast<float2*>(w + s.plane_ml[i]);
    p->plane_o[i] = reinterpret_cast<float*>(w + s.plane_o[i]);
  }
  p->slot_rows = s.slot_rows;
  p->per_unit = ~0ull / static_cast<unsigned>(s.grid);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// View {hd, rows, 1} of a cache as rows of codes; box = a page's rows, 128 at most.
bool encode_rows(CUtensorMap* map, const void* base, int hd, long long rows, int page) {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(rows), 1};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hd), static_cast<cuuint64_t>(rows) * hd};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(hd), static_cast<cuuint32_t>(std::min(page, kTile)), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kHd, bool kRows>
cudaError_t launch(const Params& p, int grid, cudaStream_t stream) {
  CUtensorMap tk, tv;
  const long long rows = (static_cast<long long>(p.num_blocks) * p.h_kv) << p.page_shift;
  if (!encode_rows(&tk, p.k, kHd, rows, 1 << p.page_shift) || !encode_rows(&tv, p.v, kHd, rows, 1 << p.page_shift))
    return cudaErrorInvalidValue;
  constexpr size_t smem = smem_bytes<kHd, kRows>();
  static_assert(smem <= 232448, "the tiles fit in shared memory");
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = configure_once(configured, [&] {
    cudaFuncAttributes f;
    cudaError_t x = cudaFuncGetAttributes(&f, ragged_kernel<kHd, kRows>);
    // the warpgroups' shares come out of what the launch takes
    if (x == cudaSuccess && f.numRegs * kThreads < 128 * (2 * kSoftmaxRegs + kConvertRegs + kIssueRegs))
      x = cudaErrorInvalidConfiguration;
    return x != cudaSuccess ? x
                            : cudaFuncSetAttribute(ragged_kernel<kHd, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
  });
  if (e != cudaSuccess) return e;
  return launch_dependent(ragged_kernel<kHd, kRows>, dim3(grid), dim3(kThreads), smem, stream, tk, tv, p);
}

cudaError_t launch_any(const Params& p, int hd, int scale_rows, int grid, cudaStream_t stream) {
  if (hd == 64) return scale_rows ? launch<64, true>(p, grid, stream) : launch<64, false>(p, grid, stream);
  return scale_rows ? launch<128, true>(p, grid, stream) : launch<128, false>(p, grid, stream);
}

bool cache_ok(const RaggedCache& c, int h_kv, int* page_shift) {
  int shift = 4;
  while (shift < 9 && (1 << shift) != c.page_size) ++shift;
  if (shift == 9 || c.num_blocks < 1) return false;  // 16, 32, 64, 128 or 256 keys a page
  if (((static_cast<long long>(c.num_blocks) * h_kv) << shift) >= (1ll << 31)) return false;  // rows: copies' coordinates
  *page_shift = shift;
  if (c.k == nullptr || c.v == nullptr || c.k_scale == nullptr || c.v_scale == nullptr) return false;
  const uintptr_t need = c.scale_rows ? 16 : 4;
  return !misaligned(c.k, 16) && !misaligned(c.v, 16) && !misaligned(c.k_scale, need) && !misaligned(c.v_scale, need) &&
         h_kv >= 1;
}

bool heads_ok(int h_q, int h_kv, int head_dim) {
  return (head_dim == 64 || head_dim == 128) && h_q >= 1 && h_kv >= 1 && h_q % h_kv == 0 && h_q <= 65536;
}

void fill_cache(Params* p, const RaggedCache& c, int head_dim) {
  p->k = static_cast<const uint8_t*>(c.k);
  p->v = static_cast<const uint8_t*>(c.v);
  p->k_scale = c.k_scale;
  p->v_scale = c.v_scale;
  p->num_blocks = c.num_blocks;
  p->lengths = kLengths[head_dim == 128][c.scale_rows != 0];
}

// Whether memory that a call writes meets an input of it (the queries are looked at apart: the output may take their place).
bool meets(std::initializer_list<Rows> written, std::initializer_list<Rows> inputs) {
  for (const Rows& w : written)
    for (const Rows& in : inputs)
      if (rows_overlap(w, in)) return true;
  return false;
}
bool meets_cache(std::initializer_list<Rows> written, const RaggedCache& c, int h_kv, int head_dim) {
  const uint64_t rows = static_cast<uint64_t>(c.num_blocks) * h_kv * c.page_size, scales = (c.scale_rows ? rows : 1) * 4;
  return meets(written, {block_of(c.k, rows * head_dim), block_of(c.v, rows * head_dim), block_of(c.k_scale, scales),
                         block_of(c.v_scale, scales)});
}
uint64_t words(long long n, long long m = 1) { return static_cast<uint64_t>(n) * static_cast<uint64_t>(m) * 4; }

constexpr long long kMostKeys = 1ll << 30;  // a segment
constexpr long long kMostRows = 1ll << 30;  // tokens * h_q
// Segments: every CTA counts through them (14 ns each, 0.9 s for as many), and their numbers stay in 32 bits.
constexpr long long kMostSegments = 1ll << 26;

}  // namespace ragged

// A table of no columns has no memory: then all lengths are 0.
static bool table_ok(const int32_t* table, int columns) { return columns > 0 ? table != nullptr : table == nullptr; }

size_t cross_workspace_bytes(int n_tokens, int bs, int h_q, int h_kv, int head_dim, long long max_keys) {
  using namespace ragged;
  if (!heads_ok(h_q, h_kv, head_dim) || n_tokens < 0 || bs < 0 || bs > kMostSegments || max_keys < 0 || max_keys > kMostKeys ||
      static_cast<long long>(n_tokens) * h_q > kMostRows)
    return 0;
  const int group = h_q / h_kv;
  return lay_out(most_work(n_tokens, bs, h_kv, group, max_keys), n_tokens, bs, h_q, group, head_dim, false).bytes;
}

fp8mla_status_t cross_entry(const CrossArgs& a, cudaStream_t stream) {
  using namespace ragged;
  Params p = {};
  if (!heads_ok(a.h_q, a.h_kv, a.head_dim) || a.n_tokens < 0 || a.bs < 0 || a.bs > kMostSegments || a.max_blocks < 0 ||
      !(a.softmax_scale > 0.f) || !cache_ok(a.cache, a.h_kv, &p.page_shift))
    return FP8MLA_ERR_INVALID_ARG;
  const long long max_keys = static_cast<long long>(a.max_blocks) << p.page_shift;
  const long long rows = static_cast<long long>(a.n_tokens) * a.h_q;
  if (max_keys > kMostKeys || rows > kMostRows || (a.q_starts == nullptr && a.n_tokens < a.bs))
    return FP8MLA_ERR_INVALID_ARG;
  if (a.n_tokens == 0 || (a.bs == 0 && !a.fill_out && !a.fill_lse)) return FP8MLA_OK;
  if (a.q == nullptr || a.out == nullptr || a.lse == nullptr || (a.bs > 0 && (!table_ok(a.block_table, a.max_blocks) || a.kv_lens == nullptr)))
    return FP8MLA_ERR_INVALID_ARG;
  if (misaligned(a.q, 16) || misaligned(a.out, 16) || misaligned(a.lse, 4) || misaligned(a.q_starts, 4) ||
      misaligned(a.block_table, 4) || misaligned(a.kv_lens, 4) || ((a.q_token | a.q_head | a.out_token | a.out_head) & 7))
    return FP8MLA_ERR_INVALID_ARG;
  const int group = a.h_q / a.h_kv;
  const Space s =
      lay_out(most_work(a.n_tokens, a.bs, a.h_kv, group, max_keys), a.n_tokens, a.bs, a.h_q, group, a.head_dim, false);
  if (a.workspace == nullptr || misaligned(a.workspace, 256)) return FP8MLA_ERR_INVALID_ARG;
  if (a.workspace_bytes < s.bytes) return FP8MLA_ERR_WORKSPACE_TOO_SMALL;
  // the output may take the queries' place; nothing else is shared
  const Rows q = rows_of(a.q, a.q_token, a.q_head, a.n_tokens, a.h_q, a.head_dim, 2);
  const Rows out = rows_of(a.out, a.out_token, a.out_head, a.n_tokens, a.h_q, a.head_dim, 2);
  const Rows lse = block_of(a.lse, rows * 4), ws = block_of(a.workspace, s.bytes);
  if (clobbers(out, q) || rows_overlap_themselves(out) || rows_overlap(lse, q) || rows_overlap(ws, q) ||
      rows_overlap(out, lse) || rows_overlap(out, ws) || rows_overlap(lse, ws) ||
      meets_cache({out, lse, ws}, a.cache, a.h_kv, a.head_dim) ||
      meets({out, lse, ws}, {block_of(a.q_starts, words(a.bs + 1ll)), block_of(a.block_table, words(a.bs, a.max_blocks)),
                             block_of(a.kv_lens, words(a.bs))}))
    return FP8MLA_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(a.q);
  fill_cache(&p, a.cache, a.head_dim);
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.q_tok = a.q_token, p.q_head = a.q_head, p.o_tok = a.out_token, p.o_head = a.out_head;
  p.list[0] = List{a.q_starts, a.kv_lens, a.block_table, a.bs, a.max_blocks, static_cast<int>(max_keys), 1, a.n_tokens, 0};
  p.list[1] = List{};
  p.group = make_fast_div(group);
  p.softmax_scale = a.softmax_scale;
  p.tokens = a.n_tokens;
  p.h_q = a.h_q;
  p.h_kv = a.h_kv;
  p.fill_out = a.fill_out;
  p.fill_lse = a.fill_lse;
  use(&p, s, a.workspace);
  use_wait_test(&p);
  // Items that are short and no more than the SMs, as far as the table's width shows, are not cut, and the merge's launch
  // is left out.  One token x 16 heads of 64 by 100, 400, 1024, 1280, 2048 keys (lengths 39 to 234): 9.9, 9.9, 12.8, 14.4,
  // 19.3 us whole, 11.5, 12.8, 13.5, 13.7, 14.2 cut; 128 items of up to 640 keys of 128 dims (138) 13.9 and 17.4.  A table
  // that is wider than the keys, as one kept for the longest context, hides that they are short: then they are cut (777 keys
  // of 64 dims 12.7 us, with a table of 16384 keys 13.3; 128 items of up to 600 keys 14.2 and 16.8).
  const long long tiles = (max_keys + kTile - 1) / kTile, all_rows = static_cast<long long>(a.n_tokens) * group;
  const int form = form_of(a.q_starts ? static_cast<int>(std::min<long long>(all_rows, kItemRows)) : group);
  const long long items = a.h_kv * (a.q_starts ? all_rows / kItemRows + a.bs : a.bs);
  p.whole = items <= device_sms() && p.lengths.fixed[form] + tiles * p.lengths.each[form] <= kWhole;
  cudaError_t e = launch_any(p, a.head_dim, a.cache.scale_rows, s.grid, stream);
  if (e == cudaSuccess && s.grid > 1 && !p.whole) {
    const dim3 grid(s.grid, (s.slot_rows + kCrossRows - 1) / kCrossRows);
    e = a.head_dim == 64
            ? launch_dependent(cross_merge_kernel<64>, grid, dim3(kMergeThreads), 0, stream, p, a.cache.scale_rows)
            : launch_dependent(cross_merge_kernel<128>, grid, dim3(kMergeThreads), 0, stream, p, a.cache.scale_rows);
  }
  return e == cudaSuccess ? FP8MLA_OK : FP8MLA_ERR_CUDA;
}

namespace ragged {
double shared_work(int bs, int q_len, int h_kv, int group, int n_prefixes, long long max_prefix_keys,
                      long long max_keys) {
  const long long tokens = static_cast<long long>(bs) * q_len;
  return (n_prefixes > 0 ? most_work(tokens, n_prefixes, h_kv, group, max_prefix_keys) : 0) +
         most_work(tokens, bs, h_kv, group, max_keys);
}
bool shared_sizes_ok(int bs, int q_len, int h_q, int h_kv, int head_dim, int n_prefixes, long long max_prefix_keys,
                     long long max_keys) {
  return heads_ok(h_q, h_kv, head_dim) && bs >= 0 && q_len >= 1 && q_len <= 32 && n_prefixes >= 0 &&
         max_prefix_keys >= 0 && max_prefix_keys <= kMostKeys && max_keys >= 0 && max_keys <= kMostKeys &&
         static_cast<long long>(bs) * q_len * h_q <= kMostRows && static_cast<long long>(bs) * h_kv <= 0x7FFFFFFF &&
         static_cast<long long>(n_prefixes) + bs <= kMostSegments;
}
}  // namespace ragged

size_t shared_workspace_bytes(int bs, int q_len, int h_q, int h_kv, int head_dim, int n_prefixes,
                              long long max_prefix_keys, long long max_keys) {
  using namespace ragged;
  if (!shared_sizes_ok(bs, q_len, h_q, h_kv, head_dim, n_prefixes, max_prefix_keys, max_keys)) return 0;
  const int group = h_q / h_kv;
  return lay_out(shared_work(bs, q_len, h_kv, group, n_prefixes, max_prefix_keys, max_keys),
                 static_cast<long long>(bs) * q_len, n_prefixes + bs, h_q, group, head_dim, true)
      .bytes;
}

fp8mla_status_t shared_entry(const SharedArgs& a, cudaStream_t stream) {
  using namespace ragged;
  Params p = {};
  if (!cache_ok(a.cache, a.h_kv, &p.page_shift) || a.max_blocks < 0 || (a.n_prefixes > 0 && a.prefix_blocks < 0) ||
      !(a.softmax_scale > 0.f))
    return FP8MLA_ERR_INVALID_ARG;
  const long long prefix_keys = a.n_prefixes > 0 ? static_cast<long long>(a.prefix_blocks) << p.page_shift : 0;
  const long long keys = static_cast<long long>(a.max_blocks) << p.page_shift;
  if (!shared_sizes_ok(a.bs, a.q_len, a.h_q, a.h_kv, a.head_dim, a.n_prefixes, prefix_keys, keys))
    return FP8MLA_ERR_INVALID_ARG;
  if (a.bs == 0) return FP8MLA_OK;
  if (a.q == nullptr || a.out == nullptr || a.lse == nullptr || a.seqlens == nullptr ||
      !table_ok(a.block_table, a.max_blocks) ||
      (a.n_prefixes > 0 && (!table_ok(a.prefix_table, a.prefix_blocks) || a.prefix_lens == nullptr || a.prefix_starts == nullptr)))
    return FP8MLA_ERR_INVALID_ARG;
  if (misaligned(a.q, 16) || misaligned(a.out, 16) || misaligned(a.lse, 4) || misaligned(a.block_table, 4) ||
      misaligned(a.seqlens, 4) || misaligned(a.prefix_table, 4) || misaligned(a.prefix_lens, 4) ||
      misaligned(a.prefix_starts, 4) || misaligned(a.sinks, 4))
    return FP8MLA_ERR_INVALID_ARG;
  const int group = a.h_q / a.h_kv;
  const long long tokens = static_cast<long long>(a.bs) * a.q_len;
  const Space s = lay_out(shared_work(a.bs, a.q_len, a.h_kv, group, a.n_prefixes, prefix_keys, keys), tokens,
                          a.n_prefixes + a.bs, a.h_q, group, a.head_dim, true);
  if (a.workspace == nullptr || misaligned(a.workspace, 256)) return FP8MLA_ERR_INVALID_ARG;
  if (a.workspace_bytes < s.bytes) return FP8MLA_ERR_WORKSPACE_TOO_SMALL;
  const uint64_t rows = static_cast<uint64_t>(tokens) * a.h_q;
  const Rows q = block_of(a.q, rows * a.head_dim * 2), out = block_of(a.out, rows * a.head_dim * 2);
  const Rows lse = block_of(a.lse, rows * 4), ws = block_of(a.workspace, s.bytes);
  if (clobbers(out, q) || rows_overlap(lse, q) || rows_overlap(ws, q) || rows_overlap(out, lse) ||
      rows_overlap(out, ws) || rows_overlap(lse, ws) || meets_cache({out, lse, ws}, a.cache, a.h_kv, a.head_dim) ||
      meets({out, lse, ws}, {block_of(a.block_table, words(a.bs, a.max_blocks)), block_of(a.seqlens, words(a.bs)),
                             block_of(a.spec_mask, static_cast<uint64_t>(tokens) * a.q_len),
                             block_of(a.sinks, words(a.h_q))}) ||
      (a.n_prefixes > 0 &&
       meets({out, lse, ws}, {block_of(a.prefix_table, words(a.n_prefixes, a.prefix_blocks)),
                              block_of(a.prefix_lens, words(a.n_prefixes)),
                              block_of(a.prefix_starts, words(a.n_prefixes + 1ll))})))
    return FP8MLA_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(a.q);
  fill_cache(&p, a.cache, a.head_dim);
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.q_tok = p.o_tok = static_cast<long long>(a.h_q) * a.head_dim;
  p.q_head = p.o_head = a.head_dim;
  const bool block = a.q_len > 1 || a.spec_mask != nullptr;
  p.list[0] = List{a.prefix_starts, a.prefix_lens, a.prefix_table, a.n_prefixes, a.prefix_blocks,
                   static_cast<int>(prefix_keys), a.q_len, a.bs, 0};
  p.list[1] = List{nullptr, a.seqlens, a.block_table, a.bs, a.max_blocks, static_cast<int>(keys), a.q_len, a.bs,
                   block ? a.q_len : 0};
  p.spec_mask = a.spec_mask;
  p.sinks = a.sinks;
  p.group = make_fast_div(group);
  p.of_rows = make_fast_div(a.q_len * group);
  p.of_heads = make_fast_div(a.h_kv);
  p.softmax_scale = a.softmax_scale;
  p.joined = 1;
  p.tokens = static_cast<int>(tokens);
  p.h_q = a.h_q;
  p.h_kv = a.h_kv;
  p.q_len = a.q_len;
  use(&p, s, a.workspace);
  use_wait_test(&p);
  cudaError_t e = launch_any(p, a.head_dim, a.cache.scale_rows, s.grid, stream);
  if (e == cudaSuccess) {
    const int total = static_cast<int>(rows);
    auto merge = [&](auto kernel, int each) {
      e = launch_dependent(kernel, dim3((total + each - 1) / each), dim3(kMergeThreads), 0, stream, p, a.cache.scale_rows,
                           s.grid, total);
    };
    const bool many = total > device_sms() * 32 * 128 / a.head_dim;
    if (a.head_dim == 64)
      many ? merge(shared_merge_kernel<64, 8>, kSharedRows<64, 8>) : merge(shared_merge_kernel<64, 4>, kSharedRows<64, 4>);
    else
      many ? merge(shared_merge_kernel<128, 8>, kSharedRows<128, 8>)
           : merge(shared_merge_kernel<128, 4>, kSharedRows<128, 4>);
  }
  return e == cudaSuccess ? FP8MLA_OK : FP8MLA_ERR_CUDA;
}

cudaError_t ragged_set_wait_test(int fault_tile, uint64_t wait_limit_ns) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= ragged::kMostDevices) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
  ragged::g_fault_tile[dev] = static_cast<uint32_t>(fault_tile);
  ragged::g_wait_limit[dev] = static_cast<uint32_t>(std::min<uint64_t>(wait_limit_ns, ragged::kWaitLimit));
  return cudaSuccess;
}

uint32_t ragged_read_and_clear_status() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_status_ragged, sizeof(v));
  cudaMemcpyToSymbol(g_status_ragged, &z, sizeof(z));
  return v;
}

}  // namespace fp8mla
