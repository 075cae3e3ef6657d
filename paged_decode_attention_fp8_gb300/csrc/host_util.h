// Host-side helpers shared by the launchers (no device code, no CUDA types).
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstdlib>
#include <utility>

namespace fp8mla {

// Runs `set` for device `dev` unless it already succeeded there: one-time,
// per-device setup such as a kernel's shared-memory limit, which CUDA keeps
// per device.  Bit d of `done` records device d; a device index outside
// [0, 64) runs `set` on every call.  `set` returns a status whose
// value-initialised form ({} : 0 / cudaSuccess) means success; a failure is
// returned and retried on the next call.  Concurrent first calls on one
// device may both run `set`, so it must be idempotent.
template <typename F>
inline auto once_per_device(std::atomic<uint64_t>& done, int dev, F&& set) -> decltype(set()) {
  using Status = decltype(set());
  const uint64_t bit = (dev >= 0 && dev < 64) ? (uint64_t{1} << dev) : uint64_t{0};
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return Status{};
  const Status r = std::forward<F>(set)();
  if (r == Status{} && bit != 0) done.fetch_or(bit, std::memory_order_acq_rel);
  return r;
}

inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Where the rows of a tensor [n, heads, width] lie, in bytes: row (i, h) is [at + i token + h head, ... + width).
// A plain block of memory is one row.
struct Rows {
  int64_t at, token, head, n, heads, width;
  bool empty() const { return n < 1 || heads < 1 || width < 1; }
};
inline Rows block_of(const void* p, uint64_t bytes) {
  return {static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)), 0, 0, 1, p == nullptr || bytes == 0 ? 0 : 1,
          static_cast<int64_t>(bytes)};
}
inline Rows rows_of(const void* p, int64_t token, int64_t head, int64_t n, int64_t heads, int64_t width, int64_t size) {
  Rows r{static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)), 0, 0, p == nullptr ? 0 : n, heads, width * size};
  if (__builtin_mul_overflow(token, size, &r.token) || __builtin_mul_overflow(head, size, &r.head))
    r.token = r.head = INT64_MAX;  // no memory is that large (see extent)
  return r;
}

// The first byte of all rows and the one behind their last; false where that leaves 62 bits, as no memory does.
inline bool extent(const Rows& r, int64_t* lo, int64_t* hi) {
  constexpr int64_t kMost = int64_t{1} << 62;
  int64_t t, h;
  if (__builtin_mul_overflow(r.n - 1, r.token, &t) || __builtin_mul_overflow(r.heads - 1, r.head, &h) ||
      std::abs(t) > kMost / 4 || std::abs(h) > kMost / 4 || r.at > kMost / 4 || r.width > kMost / 4)
    return false;
  *lo = r.at + std::min<int64_t>(t, 0) + std::min<int64_t>(h, 0);
  *hi = r.at + std::max<int64_t>(t, 0) + std::max<int64_t>(h, 0) + r.width;
  return true;
}

// Whether lo < step m + c < hi for an integer m in [first, last].
inline bool hits(int64_t step, int64_t c, int64_t first, int64_t last, int64_t lo, int64_t hi) {
  if (first > last) return false;
  if (step == 0) return lo < c && c < hi;
  if (step < 0) return hits(-step, c, -last, -first, lo, hi);
  int64_t m = (lo - c) / step;  // the first m with step m + c > lo
  while (step * m + c > lo) --m;
  while (step * m + c <= lo) ++m;
  m = std::max(m, first);
  return m <= last && step * m + c < hi;
}

// Whether a row of a shares a byte with one of b.  Exact where the strides are the same (a dimension of one has any);
// else, and past 2^16 steps, tensors whose extents meet are taken to.
inline bool rows_overlap(Rows a, Rows b) {
  if (a.empty() || b.empty()) return false;
  int64_t alo, ahi, blo, bhi;
  if (!extent(a, &alo, &ahi) || !extent(b, &blo, &bhi)) return true;
  if (ahi <= blo || bhi <= alo) return false;
  if (a.n == 1) a.token = b.token;
  if (b.n == 1) b.token = a.token;
  if (a.heads == 1) a.head = b.head;
  if (b.heads == 1) b.head = a.head;
  if (a.token != b.token || a.head != b.head) return true;
  // row of b less row of a: d + token m + head k, m in (-a.n, b.n), k in (-a.heads, b.heads)
  const int64_t d = b.at - a.at;
  if (a.token > 0 && a.head >= 0) {  // the usual case: parts of one row of heads, a token's after the other
    const int64_t off = (d % a.token + a.token) % a.token;
    if (off >= (a.heads - 1) * a.head + a.width && off + (b.heads - 1) * b.head + b.width <= a.token) return false;
  }
  const bool few_heads = a.heads + b.heads <= a.n + b.n;
  const int64_t from = few_heads ? 1 - a.heads : 1 - a.n, to = few_heads ? b.heads : b.n;
  if (to - from > (1 << 16)) return true;
  for (int64_t i = from; i < to; ++i)
    if (few_heads ? hits(a.token, d + a.head * i, 1 - a.n, b.n - 1, -b.width, a.width)
                  : hits(a.head, d + a.token * i, 1 - a.heads, b.heads - 1, -b.width, a.width))
      return true;
  return false;
}

// Whether two rows of r share a byte.
inline bool rows_overlap_themselves(const Rows& r) {
  if (r.empty()) return false;
  int64_t lo, hi;
  if (!extent(r, &lo, &hi)) return true;
  const bool few_heads = r.heads <= r.n;
  const int64_t outer = few_heads ? r.head : r.token, inner = few_heads ? r.token : r.head;
  const int64_t outers = few_heads ? r.heads : r.n, inners = few_heads ? r.n : r.heads;
  if (hits(inner, 0, 1, inners - 1, -r.width, r.width)) return true;
  // the usual cases: each set of rows behind the one before, or between its rows
  if (inner >= 0 && outer >= inner * (inners - 1) + r.width) return false;
  if (outer >= r.width && inner >= outer * (outers - 1) + r.width) return false;
  if (outers > (1 << 16)) return true;
  for (int64_t i = 1; i < outers; ++i)
    if (hits(inner, outer * i, 1 - inners, inners - 1, -r.width, r.width)) return true;
  return false;
}

inline bool same_rows(const Rows& a, const Rows& b) {
  return a.at == b.at && a.n == b.n && a.heads == b.heads && a.width == b.width && (a.n <= 1 || a.token == b.token) &&
         (a.heads <= 1 || a.head == b.head);
}

// Whether `out` shares memory with an input that it does not replace row by row.
inline bool clobbers(const Rows& out, const Rows& in) { return !same_rows(out, in) && rows_overlap(out, in); }

}  // namespace fp8mla
