// kda_cache_tables.cu -- kda_cache_tables: block tables, slots and the ring of
// free pages from the requests' lengths.
//
// Everything follows from exclusive prefix sums over the requests, of the new
// tokens, of the pages taken and of the pages given back.  They are few (a
// thousand requests is one pass of one CTA), so one CTA does the sums and moves
// the pages: what bounds it is the chain of dependent loads (lengths, ring,
// table), not their number.  The slots, one per new token, are written by the
// same CTA when they are few and by a second kernel over the whole GPU otherwise.
#include <algorithm>

#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ int pages_of(int64_t tokens, int page) {
  return (int)((tokens + page - 1) / page);
}

// Inclusive sum over the CTA's threads; `total` gets the CTA's sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* warp_sums, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  if (warp > 0) x += warp_sums[warp - 1];
  total = warp_sums[kWarps - 1];
  __syncthreads();
  return x;
}

// The request whose tokens hold packed token i (cu[0] = 0 <= i < cu[n]).
__device__ __forceinline__ int request_of(const int32_t* cu, int n, int i) {
  int lo = 0, hi = n;  // cu[lo] <= i < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Slot of packed token i, whose request's first slot is in place (-1: refused).
__device__ __forceinline__ int64_t slot_of(const TableArgs& a, int i) {
  const int b = request_of(a.cu_new, a.num_seqs, i);
  const int first = a.cu_new[b], n = a.cu_new[b + 1] - first;
  if (a.slots[first] < 0) return -1;
  const int pos = a.kv_lens[b] - n + (i - first);
  return (int64_t)a.block_table[(int64_t)b * a.max_blocks + pos / a.page_size] * a.page_size +
         pos % a.page_size;
}

// Requests of one pass of the CTA, for the page moves that follow their sums.
struct Pass {
  int32_t taken_at[kThreads + 1];  // pages taken before each request of the pass
  int32_t freed_at[kThreads + 1];
  int32_t from[kThreads];          // first column that changes
};

// The request of the pass that page i belongs to.
__device__ __forceinline__ int owner(const int32_t* at, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (at[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) tables_kernel(TableArgs a, int write_slots) {
  __shared__ int64_t warp_sums[kWarps];
  __shared__ Pass ps;
  const int P = a.page_size;
  int64_t head = a.free_range[0], tail = a.free_range[1];
  const bool ring_ok = head >= 0 && tail >= head && tail - head <= a.ring_size;
  if (!ring_ok) {
    head = tail = 0;
    if (threadIdx.x == 0) report_error(a.err, kErrDeviceCheck);
  }
  const int64_t avail = tail - head;
  int64_t tokens = 0, asked = 0, taken = 0, freed = 0;  // of the requests before this pass
  for (int base = 0; base < a.num_seqs; base += kThreads) {
    const int b = base + threadIdx.x;
    const bool in = b < a.num_seqs;
    const int64_t held = in ? a.held_lens[b] : 0, seq = in ? a.seq_lens[b] : 0;
    const int64_t fresh = in ? a.new_lens[b] : 0;
    const bool sound = held >= 0 && seq >= 0 && seq <= held && fresh >= -1 &&
                       pages_of(held, P) <= a.max_blocks;
    const int64_t add = fresh > 0 ? fresh : 0;
    const int64_t keep = sound && fresh >= 0 ? seq : 0;
    const int have = sound ? pages_of(held, P) : 0;
    int64_t target = sound ? keep + add : 0;
    bool refused = !sound || pages_of(target, P) > a.max_blocks || target > INT32_MAX;
    int grow = refused ? 0 : max(0, pages_of(target, P) - have);
    int64_t sum, pass_taken, pass_freed;
    int64_t taken_at = block_scan(grow, warp_sums, sum) - grow;
    pass_taken = sum;
    if (asked + sum > avail) {  // the ring runs dry in this pass or before
      if (grow > 0 && asked + taken_at + grow > avail) {
        refused = true;
        grow = 0;
      }
      taken_at = block_scan(grow, warp_sums, pass_taken) - grow;
    }
    asked += sum;
    if (refused) target = keep;
    if (in && refused && (add > 0 || !sound)) report_error(a.err, kErrDeviceCheck);
    const int want = pages_of(target, P);
    const int shrink = max(0, have - want);
    const int64_t freed_at = block_scan(shrink, warp_sums, pass_freed) - shrink;
    const int64_t first = tokens + block_scan(add, warp_sums, sum) - add;
    tokens += sum;
    ps.taken_at[threadIdx.x] = (int32_t)taken_at;
    ps.freed_at[threadIdx.x] = (int32_t)freed_at;
    ps.from[threadIdx.x] = grow > 0 ? have : want;
    if (in) {
      a.kv_lens[b] = (int32_t)target;
      a.cu_new[b] = (int32_t)min(first, (int64_t)INT32_MAX);
    }
    __syncthreads();
    // pages change hands, a thread each: what a request gives back may be thousands
    for (int i = threadIdx.x; i < pass_freed; i += kThreads) {
      const int o = owner(ps.freed_at, kThreads, i);
      a.free_pages[(tail + freed + i) % a.ring_size] =
          a.block_table[(int64_t)(base + o) * a.max_blocks + ps.from[o] + i - ps.freed_at[o]];
    }
    for (int i = threadIdx.x; i < pass_taken; i += kThreads) {
      const int o = owner(ps.taken_at, kThreads, i);
      a.block_table[(int64_t)(base + o) * a.max_blocks + ps.from[o] + i - ps.taken_at[o]] =
          a.free_pages[(head + taken + i) % a.ring_size];
    }
    taken += pass_taken;
    freed += pass_freed;
    __syncthreads();
    if (in && add > 0 && first < a.max_tokens)
      a.slots[first] =
          refused ? -1
                  : (int64_t)a.block_table[(int64_t)b * a.max_blocks + keep / P] * P + keep % P;
  }
  if (threadIdx.x == 0) {
    a.cu_new[a.num_seqs] = (int32_t)min(tokens, (int64_t)INT32_MAX);
    a.free_range_out[0] = head + taken;
    a.free_range_out[1] = tail + freed;
    if (tokens > a.max_tokens || avail - taken + freed > a.ring_size)
      report_error(a.err, kErrDeviceCheck);
  }
  if (!write_slots) return;
  __syncthreads();  // cu_new, kv_lens, block_table and the first slots are in place
  for (int i = threadIdx.x; i < a.max_tokens; i += kThreads) {
    if (i >= tokens)
      a.slots[i] = -1;
    else if (a.cu_new[request_of(a.cu_new, a.num_seqs, i)] != i)
      a.slots[i] = slot_of(a, i);
  }
}

__global__ void __launch_bounds__(256) slots_kernel(TableArgs a) {
  const int tokens = a.cu_new[a.num_seqs];
  for (int i = blockIdx.x * 256 + threadIdx.x; i < a.max_tokens; i += gridDim.x * 256) {
    if (i >= tokens)
      a.slots[i] = -1;
    else if (a.cu_new[request_of(a.cu_new, a.num_seqs, i)] != i)
      a.slots[i] = slot_of(a, i);
  }
}

// Up to this many slots are written by the first kernel.
constexpr int kOneLaunchTokens = 4096;

}  // namespace

cudaError_t launch_cache_tables(const TableArgs& a, cudaStream_t st) {
  const bool one = a.max_tokens <= kOneLaunchTokens;
  tables_kernel<<<1, kThreads, 0, st>>>(a, one ? 1 : 0);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || one) return e;
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  slots_kernel<<<std::min((a.max_tokens + 255) / 256, 8 * sms), 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
