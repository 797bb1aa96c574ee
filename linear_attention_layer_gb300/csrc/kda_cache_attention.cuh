// kda_cache_attention.cuh -- what the two attention kernels over both forms of the cache share:
// requests as their planners see them, softmax constants, row output.
#pragma once

#include <type_traits>

#include "kda_byte_cache.cuh"
#include "kda_cache.cuh"
#include "kda_launch.h"
#include "tc_ptx.cuh"

namespace kda {
namespace cache {

// Weights are 2^(s - m) with a reference m below the largest score seen by kLift at least and
// kLift + kSlack at most: up to 2^15, within a half's range, and as far from the end of its
// small numbers as that allows.
constexpr float kSlack = 8.f, kLift = 7.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int BITS, int D>
using FormLayout = std::conditional_t<BITS == 4, Layout<D>, Layout8<D>>;

// -m of a row that has seen nothing yet, 8 bits: any score passes it.
constexpr float kUnset = 1e30f;

// 2^d for d <= 0; 0 where fp32 has no normal number for it.
__device__ __forceinline__ float power_below(int d) {
  return d < -126 ? 0.f : __int_as_float((127 + d) << 23);
}

// Waits for a phase of the barrier; false when it took `limit` cycles or `*failed` (another wait
// that gave up; may be null) was set.  Each thread has its own answer: before code that needs a
// whole warp the answers have to be brought together by a vote, or some of its threads could
// leave and the others wait for them.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, uint32_t limit,
                                           volatile int* failed) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const uint32_t start = (uint32_t)clock();  // 32 bits: 2 s, and a register less
  for (uint32_t i = 1;; ++i) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    if ((i & 15) == 0 && ((failed && *failed) || (uint32_t)clock() - start > limit)) return false;
  }
}

// Which requests a launch takes: those whose rows per kv head (new tokens x query
// heads of the group) lie in (above, up_to].
struct RowRange {
  int64_t above, up_to;
};

// Longest request: key numbers are rounded up to whole tiles in 31 bits.
constexpr int kMostKeys = INT32_MAX - 127;

// A request of the launch.
struct Request {
  int kv, n, bos;
  int64_t rows;  // per kv head; 0: not of this launch
};

// What a kernel ahead may still be writing when this one's CTAs start (launch_after) is not read by
// the path for data that does not change while a kernel runs.
template <bool AFTER, typename T>
__device__ __forceinline__ T fetch(const T* p) {
  if constexpr (AFTER)
    return *p;
  else
    return __ldg(p);
}

template <bool AFTER = false>
__device__ __forceinline__ bool load_request(const View& c, const AttentionArgs& a, int b,
                                             const RowRange& range, bool report, Request& r) {
  int eos;
  // a decreasing offset takes both of its neighbours out: their tokens may overlap others'
  const bool ok = seq_range(a.cu_new, b, a.total_tokens, report ? a.err : nullptr, r.bos, eos) &&
                  (b == 0 || fetch<AFTER>(a.cu_new + b - 1) <= r.bos);
  r.kv = fetch<AFTER>(a.kv_lens + b);
  r.rows = 0;
  r.n = 0;
  if (!ok) return false;
  if (r.kv < 0 || r.kv > (int64_t)a.max_blocks * c.page_size || r.kv > kMostKeys) {
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
    const int mid = lo + ((hi - lo) >> 1);
    if ((unsigned long long)plan[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Power of two that brings a row with this largest magnitude into [2^10, 2^11) -- again
// far from a half's smallest numbers, where its second half would lose bits: the row's
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
  e = max(e - 10, -126);
  r.down = copysignf(__int_as_float((127 - e) << 23), scale);
  r.f = fminf(fmaxf(fabsf(scale) * kLog2e * k_factor * __int_as_float((127 + e) << 23), 1.2e-38f),
              3.e38f);
  return r;
}

// The raw score up to which a weight 2^(s f - m) stays within 2^(kLift + kSlack): rounded down, or
// beside a reference of 2^24 and more a weight could pass a half's largest value.
__device__ __forceinline__ float score_limit(float m, float f) {
  return __fdiv_rd(__fadd_rd(m, kLift + kSlack), f);
}

// One row of a unit put together from parts i = first .. last, whose (m, l, o[D]) lie at
// index at(i) of ml and o: by one warp, each lane with D / 32 neighbouring channels.  The
// loads do not wait for one another.
template <int D>
struct RowSum {
  float top = -INFINITY, sum = 0.f, x[D / 32] = {};

  template <typename At>
  __device__ __forceinline__ void add(const float* o, const float2* ml, int first, int last,
                                      At at) {
    const int lane = threadIdx.x & 31;
    for (int base = first; base <= last; base += 32) {
      const int n = min(32, last - base + 1);
      const float2 mine = lane < n ? ml[at(base + lane)] : make_float2(-INFINITY, 0.f);
      float next = fmaxf(top, mine.x);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) next = fmaxf(next, __shfl_xor_sync(0xffffffffu, next, s));
      const float keep = next == -INFINITY ? 1.f : ex2_approx(top - next);
      const float k = next == -INFINITY ? 1.f : ex2_approx(mine.x - next);
      top = next;
      sum = fmaf(sum, keep, warp_sum(k * mine.y));
#pragma unroll
      for (int j = 0; j < D / 32; ++j) x[j] *= keep;
#pragma unroll 8
      for (int i = 0; i < n; ++i) {
        const float w = __shfl_sync(0xffffffffu, k, i);
        float y[D / 32];
        load(o + at(base + i) * D, y);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) x[j] = fmaf(y[j], w, x[j]);
      }
    }
  }
  __device__ __forceinline__ static void load(const float* p, float (&y)[D / 32]) {
    const int lane = threadIdx.x & 31;
    if constexpr (D == 128) {
      const float4 v = *reinterpret_cast<const float4*>(p + 4 * lane);
      y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
    } else {
      const float2 v = *reinterpret_cast<const float2*>(p + 2 * lane);
      y[0] = v.x, y[1] = v.y;
    }
  }
  __device__ __forceinline__ void store_part(float* o, float2* ml, int64_t at) const {
    const int lane = threadIdx.x & 31;
    if constexpr (D == 128)
      *reinterpret_cast<float4*>(o + at * D + 4 * lane) = make_float4(x[0], x[1], x[2], x[3]);
    else
      *reinterpret_cast<float2*>(o + at * D + 2 * lane) = make_float2(x[0], x[1]);
    if (lane == 0) ml[at] = make_float2(top, sum);
  }
  // The finished row; v_factor is the head's power of two of the values.
  template <typename T>
  __device__ __forceinline__ void store(T* out, float* lse, int64_t at, float v_factor) const {
    const int lane = threadIdx.x & 31;
    const float inv = sum == 0.f ? 0.f : v_factor / sum;
    T* p = out + at * D + lane * (D / 32);
    if constexpr (sizeof(T) == 2) {
      uint32_t w[D / 64];
#pragma unroll
      for (int j = 0; j < D / 64; ++j) w[j] = tc::pack_bf16(x[2 * j] * inv, x[2 * j + 1] * inv);
      if constexpr (D == 128)
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      if constexpr (D == 128)
        *reinterpret_cast<float4*>(p) = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
      else
        *reinterpret_cast<float2*>(p) = make_float2(x[0] * inv, x[1] * inv);
    }
    if (lse && lane == 0) lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
  }
};

// A unit that the CTA of this index starts and that CTAs up to `last` carry on (-1: none).
struct OpenUnit {
  int bos;   // first new token of its request
  int row0;  // its first row among the request's (fits: rows of one request < 2^31, checked)
  int rows;
  int head;  // kv head
  int last;
};

// Joins open units: a CTA has PER rows of one, WPR warps a row.
template <typename T, int D, int PER, int WPR>
__global__ void __launch_bounds__(32 * PER * WPR)
    join_kernel(View c, AttentionArgs a, const OpenUnit* units, const float* o, const float2* ml,
                int slot0, int unit_rows) {
  constexpr int kFields = 2 + D / 32;
  __shared__ float shared_sum[WPR > 1 ? PER * WPR : 1][kFields][32];
  wait_for_previous();
  const int first = blockIdx.x;
  const OpenUnit u = units[first];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (u.last < 0 || blockIdx.y * PER >= u.rows) return;
  const int row = blockIdx.y * PER + warp / WPR, part = warp % WPR;
  const int per = (u.last - first + WPR) / WPR;
  const int p0 = first + part * per, p1 = min(u.last, p0 + per - 1);
  RowSum<D> r;
  if (row < u.rows)
    r.add(o, ml, p0, p1, [&](int i) {
      return (int64_t)(slot0 + 2 * i + (i == first ? 1 : 0)) * unit_rows + row;
    });
  if constexpr (WPR > 1) {
    shared_sum[warp][0][lane] = r.top;
    shared_sum[warp][1][lane] = r.sum;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) shared_sum[warp][2 + j][lane] = r.x[j];
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int w = 1; w < WPR; ++w) {
      const float(*s)[32] = shared_sum[warp + w];
      const float next = fmaxf(r.top, s[0][lane]);
      const float k0 = next == -INFINITY ? 1.f : ex2_approx(r.top - next);
      const float k1 = next == -INFINITY ? 1.f : ex2_approx(s[0][lane] - next);
      r.top = next;
      r.sum = r.sum * k0 + s[1][lane] * k1;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) r.x[j] = r.x[j] * k0 + s[2 + j][lane] * k1;
    }
  }
  if (row >= u.rows) return;
  const int group = a.num_heads / c.kv_heads;
  const int rr = u.row0 + row;
  const int64_t at = (int64_t)(u.bos + rr / group) * a.num_heads + u.head * group + rr % group;
  r.store(static_cast<T*>(a.out), a.lse, at, exponent_scale(c.v_exp, u.head, 1));
}

// Launches it right behind the kernel whose units it joins.
template <typename T, int D, int PER, int WPR>
cudaError_t launch_join(const View& c, const AttentionArgs& a, const OpenUnit* units,
                        const float* o, const float2* ml, int slot0, int unit_rows, int ctas,
                        cudaStream_t st) {
  return launch_after(join_kernel<T, D, PER, WPR>, dim3(ctas, unit_rows / PER), 32 * PER * WPR, 0, st,
                      c, a, units, o, ml, slot0, unit_rows);
}

inline int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

}  // namespace cache
}  // namespace kda
