// Shared constants and the bounded mbarrier wait used by every kernel.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <mutex>
#include <utility>

#include "fp8mla.h"
#include "host_util.h"
#include "ptx.cuh"

namespace fp8mla {

// The last N tensor maps an entry point encoded, by (base pointer, extent,
// device): a map depends on nothing else (its boxes and strides are fixed per
// entry point), so a call on the same cache skips the host-side encoding.
template <int N>
class TensorMapCache {
 public:
  template <typename Encode>
  bool get(const void* base, long long extent, CUtensorMap* out, Encode&& encode) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lock(mu_);
    for (const Entry& e : entries_)
      if (e.used && e.base == base && e.extent == extent && e.device == dev) {
        *out = e.map;
        return true;
      }
    CUtensorMap m;
    if (!encode(&m)) return false;
    entries_[next_] = Entry{base, extent, dev, true, m};
    next_ = (next_ + 1) % N;
    *out = m;
    return true;
  }

 private:
  struct Entry {
    const void* base;
    long long extent;
    int device;
    bool used;
    CUtensorMap map;
  };
  std::mutex mu_;
  Entry entries_[N] = {};
  int next_ = 0;
};

// A wait that has not completed after this long is treated as a hang: the
// kernel records FP8MLA_DEV_WAIT_TIMEOUT and stops instead of spinning on.
// The limit lives in device memory (one copy per translation unit) so that a
// test can shorten it for the kernels of one file (fp8mla_test_fault_injection).
constexpr uint64_t kWaitLimitNs = 4000000000ull;
constexpr uint32_t kWaitMinPolls = 1u << 16;
static __device__ uint64_t g_wait_limit_ns = kWaitLimitNs;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_huge_valf();

// The first bounded wait of this translation unit's kernels that ran out:
// {site (a source line), block, thread, recorded}; read and cleared by the host.
static __device__ uint32_t g_timeout_where[4];

__device__ __forceinline__ void record_timeout_site(uint32_t site) {
  if (atomicCAS(&g_timeout_where[3], 0u, 1u) == 0u) {
    g_timeout_where[0] = site;
    g_timeout_where[1] = blockIdx.x;
    g_timeout_where[2] = threadIdx.x;
  }
}

// Bounded wait on an mbarrier phase.  Returns false (without waiting further)
// once *abort_flag is set by any thread of the CTA, or after the limit, in
// which case it sets the flag and the status bit itself.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                             uint32_t* status, uint32_t site = 0) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 31u) == 0) {
      if (abort_flag != nullptr && *abort_flag) return false;
      if (it > kWaitMinPolls && globaltimer_ns() - t0 > *(volatile uint64_t*)&g_wait_limit_ns) {
        if (abort_flag != nullptr) *abort_flag = 1u;
        atomicOr(status, FP8MLA_DEV_WAIT_TIMEOUT);
        record_timeout_site(site);
        return false;
      }
    }
  }
}

// The same contract as wait_bounded, but polling with the non-blocking probe:
// for waits on the critical path, where a suspended thread wakes up late.
__device__ __forceinline__ bool wait_spin(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag,
                                          uint32_t* status, uint32_t site = 0) {
  if (mbar_test_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_test_wait(bar, parity)) return true;
    if ((it & 255u) == 0) {
      if (abort_flag != nullptr && *abort_flag) return false;
      if (it > kWaitMinPolls && globaltimer_ns() - t0 > *(volatile uint64_t*)&g_wait_limit_ns) {
        if (abort_flag != nullptr) *abort_flag = 1u;
        atomicOr(status, FP8MLA_DEV_WAIT_TIMEOUT);
        record_timeout_site(site);
        return false;
      }
    }
  }
}

// Pages of a sequence; 0 (and a status bit) for a length the block table cannot hold.
__device__ __forceinline__ int seq_pages(int s_k, int page, int max_pages, uint32_t* status) {
  if (s_k <= 0) {
    if (s_k < 0) atomicOr(status, FP8MLA_DEV_BAD_SEQLEN);
    return 0;
  }
  const int n = (s_k + page - 1) / page;
  if (n > max_pages) {
    atomicOr(status, FP8MLA_DEV_BAD_SEQLEN);
    return 0;
  }
  return n;
}

// One arrival per warp: every lane's earlier work (shared-memory writes,
// completed tcgen05 loads/stores followed by tcgen05.fence::before_thread_sync)
// is ordered before lane 0's release-arrive by the warp barrier.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// once_per_device on the current device; a failing cudaGetDevice is returned.
template <typename F>
inline cudaError_t configure_once(std::atomic<uint64_t>& done, F&& set) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  return once_per_device(done, dev, std::forward<F>(set));
}

// Launches `kernel` on `stream` as a programmatic dependent of the previous
// work in the stream: its CTAs may start while that work finishes, so the
// kernel must call griddep_wait() before touching memory the predecessor
// writes or reads.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                             Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The same in thread-block clusters of `cluster` neighbouring CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent_clusters(unsigned cluster, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                      cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The end of one output row: key weights summed to l against reference m (log2
// units of the scaled scores), an optional sink logit `sink` (natural units,
// -inf = none) joining the denominator once.  Returns the output factor f
// (times the accumulated P.V) and the row's LSE (natural log).  No key and no
// sink: f = 0, LSE -inf; no key with a sink: f = 0, LSE = sink.
__device__ __forceinline__ void finish_row(float m, float l, float sink, float v_scale, float* f, float* lse) {
  if (sink == kNegInf) {
    *f = l > 0.f ? v_scale / l : 0.f;
    *lse = l > 0.f ? (m + lg2_approx(l)) * kLn2 : kNegInf;
    return;
  }
  const float sk2 = sink * kLog2e;
  if (!(l > 0.f)) {
    *f = 0.f;
    *lse = sink;
    return;
  }
  const float mm = fmaxf(m, sk2);
  const float wk = ex2_approx(m - mm);
  const float den = l * wk + ex2_approx(sk2 - mm);
  *f = v_scale * wk / den;
  *lse = (mm + lg2_approx(den)) * kLn2;
}

// A V row's scale whose log2 goes into the row's weight and whose inverse takes it out of the sum: below 2^-126 the first
// is -inf and the second past float32, and the sum of many keys is before that.  From 2^-110 down it counts as 2^-110, which
// keeps the sum right (up to 2^17 keys that are all so small) and puts a row's values off by 2^-101 at most.  (A NaN stays
// one.)
__device__ __forceinline__ float v_row_scale(float s) { return s < 0x1p-110f ? 0x1p-110f : s; }

// n / d by a multiply-high (see make_fast_div)
struct FastDiv {
  uint32_t d, m, s;
};

__device__ __forceinline__ uint32_t fast_div(uint32_t n, const FastDiv& f) {
  return f.d == 1 ? n : (__umulhi(n, f.m) >> f.s);
}

// Constants of fast_div for divisor d (numerators below 2^31): with
// l = ceil(log2 d), m = floor(2^(31 + l) / d) + 1 < 2^32 gives
// n / d = (n * m) >> (31 + l) for every n < 2^31 (d = 1 is passed through).
inline FastDiv make_fast_div(int d) {
  FastDiv f;
  f.d = static_cast<uint32_t>(d);
  f.m = 0;
  f.s = 0;
  if (d <= 1) return f;
  uint32_t l = 0;
  while ((1ull << l) < static_cast<uint64_t>(d)) ++l;
  f.m = static_cast<uint32_t>((1ull << (31 + l)) / static_cast<uint64_t>(d) + 1);
  f.s = l - 1;
  return f;
}

// SM count of the current device, queried once per device (152 if unknown).
inline int device_sms() {
  static std::atomic<int> sms[64];  // zero-initialised: static storage
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  int n = sms[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 152;
    sms[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace fp8mla
