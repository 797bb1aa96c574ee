// kda_cache_attention.cuh -- what the two attention kernels over the cache share:
// requests as their planners see them, softmax constants, row output.
#pragma once

#include "kda_cache.cuh"
#include "kda_launch.h"
#include "tc_ptx.cuh"

namespace kda {
namespace cache {

constexpr float kSlack = 8.f;  // log2 head room of a weight over the reference maximum
constexpr long long kWaitCycles = 2000000000ll;  // about a second: a wait gives up after it
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Waits for a phase of the barrier; false when it took kWaitCycles or `*failed` (another
// warp's wait that gave up; may be null) was set.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* failed) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const long long start = clock64();
  for (uint32_t i = 1;; ++i) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((i & 15) == 0 && ((failed && *failed) || clock64() - start > kWaitCycles)) return false;
  }
}

// Which requests a launch takes: those whose rows per kv head (new tokens x query
// heads of the group) lie in (above, up_to].
struct RowRange {
  int64_t above, up_to;
};

// A request of the launch.
struct Request {
  int kv, n, bos;
  int64_t rows;  // per kv head; 0: not of this launch
};

__device__ __forceinline__ bool load_request(const View& c, const AttentionArgs& a, int b,
                                             const RowRange& range, bool report, Request& r) {
  int eos;
  // a decreasing offset takes both of its neighbours out: their tokens may overlap others'
  const bool ok = seq_range(a.cu_new, b, a.total_tokens, report ? a.err : nullptr, r.bos, eos) &&
                  (b == 0 || __ldg(a.cu_new + b - 1) <= r.bos);
  r.kv = __ldg(a.kv_lens + b);
  r.rows = 0;
  r.n = 0;
  if (!ok) return false;
  if (r.kv < 0 || r.kv > (int64_t)a.max_blocks * c.page_size) {
    if (report) report_error(a.err, kErrDeviceCheck);
    return false;
  }
  r.n = eos - r.bos;
  const int64_t rows = (int64_t)r.n * (a.num_heads / c.kv_heads);
  if (rows > range.above && rows <= range.up_to) r.rows = rows;
  return r.rows > 0;
}

// The last index i with plan[i] <= x (plan[0] <= x < plan[n]).
template <typename P>
__device__ __forceinline__ int find_last(const P* plan, int n, unsigned long long x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((unsigned long long)plan[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Power of two that brings a row with this largest magnitude into [1, 2): the row's
// factors down (applied to it, with the sign of the score factor) and f (of its raw
// scores, log2 units; kept positive and finite, so that a masked score stays -infinity).
struct RowScale {
  float down, f;
};
__device__ __forceinline__ RowScale row_scale(float top, float scale, float k_factor) {
  // e held to the normal range, 0 where top is not finite
  int e = ((__float_as_int(top) >> 23) & 255) - 127;
  e = e == 128 ? 0 : max(-126, min(e, 126));
  RowScale r;
  r.down = copysignf(__int_as_float((127 - e) << 23), scale);
  r.f = fminf(fmaxf(fabsf(scale) * kLog2e * k_factor * __int_as_float((127 + e) << 23), 1.2e-38f),
              3.e38f);
  return r;
}

}  // namespace cache
}  // namespace kda
