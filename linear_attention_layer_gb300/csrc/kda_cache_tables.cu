// kda_cache_tables.cu -- kda_cache_tables: block tables, slots and the ring of
// free pages from the requests' lengths.
//
// Everything follows from exclusive prefix sums over the requests, of the new
// tokens, of the pages taken and of the pages given back.  They are few (a
// thousand requests is one pass of one CTA), so one CTA does the sums and moves
// the pages: what bounds it is the chain of dependent loads (lengths, ring,
// table) and the barriers, not their number, so the three sums go together.  The
// slots, one per new token, are written by the same CTA when they are few and by a
// second kernel over the whole GPU otherwise.
#include <algorithm>

#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

// Counters that step through the caller's sizes (each below 2^31) are unsigned: the step past the
// last one does not fit 31 bits.

// 256 requests' decode step / 37 with up to 1800 pages given back / 64 prompts, host included:
// 9.6 / 12.3 / 14.3 us; with 256 threads 10.2 / 13.7 / 16.4, with 1024 10.3 / 12.3 / 14.5.
constexpr int kThreads = 512;

__device__ __forceinline__ int pages_of(int64_t tokens, int page) {
  return (int)((tokens + page - 1) / page);
}

// Pages taken, pages given back and new tokens of a request, or their sums.
struct Counts {
  int64_t pages;   // taken in the low 32 bits, given back in the high ones: fewer than
                   // 2^31 each, a pass moves no more than the tables have entries
  int64_t tokens;
  Counts() = default;
  __device__ __forceinline__ Counts(int taken, int freed, int64_t t)
      : pages((int64_t)((uint64_t)(uint32_t)freed << 32 | (uint32_t)taken)), tokens(t) {}
  __device__ __forceinline__ int taken() const { return (int)(pages & 0xffffffff); }
  __device__ __forceinline__ int freed() const { return (int)(pages >> 32); }
};

// Sums of the CTA's threads before this one; `total` gets the sum of all.
__device__ __forceinline__ Counts block_scan(Counts x, Counts* warp_sums, Counts& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Counts mine = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t p = __shfl_up_sync(0xffffffffu, x.pages, o);
    const int64_t t = __shfl_up_sync(0xffffffffu, x.tokens, o);
    if (lane >= o) x.pages += p, x.tokens += t;
  }
  __syncthreads();  // the sums of the call before are read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  Counts before(0, 0, 0);
  total = before;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const Counts s = warp_sums[w];
    if (w < warp) before.pages += s.pages, before.tokens += s.tokens;
    total.pages += s.pages, total.tokens += s.tokens;
  }
  before.pages += x.pages - mine.pages;
  before.tokens += x.tokens - mine.tokens;
  return before;
}

// The last index i < n with at[i] <= x (at[0] <= x).
__device__ __forceinline__ int owner(const int32_t* at, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = lo + ((hi - lo) >> 1);
    if (at[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Slot of packed token i of request b, whose first slot is in place (-1: refused).
__device__ __forceinline__ int64_t slot_of(const TableArgs& a, int b, int i, int first, int n) {
  if (a.slots[first] < 0) return -1;
  const int pos = a.kv_lens[b] - n + (i - first);
  return (int64_t)a.block_table[(int64_t)b * a.max_blocks + pos / a.page_size] * a.page_size +
         pos % a.page_size;
}

// Requests of one pass of the CTA, for the page moves that follow their sums.
struct Pass {
  int32_t taken_at[kThreads];  // pages taken before each request of the pass
  int32_t freed_at[kThreads];
  int32_t from[kThreads];      // first column that changes
};

constexpr int kFew = 8;  // new tokens whose slots the request's own thread writes

__global__ void __launch_bounds__(kThreads) tables_kernel(TableArgs a, int write_slots) {
  __shared__ Counts warp_sums[kThreads / 32];
  __shared__ Pass ps;
  const int P = a.page_size;
  int64_t head = a.free_range[0], tail = a.free_range[1];
  const bool ring_ok = head >= 0 && tail >= head && tail - head <= a.ring_size;
  if (!ring_ok) {
    head = tail = 0;
    if (threadIdx.x == 0) report_error(a.err, kErrDeviceCheck);
  }
  const int64_t avail = tail - head;
  const int64_t head0 = head % a.ring_size, tail0 = tail % a.ring_size;
  auto in_ring = [&](int64_t at) {  // at < 2 ring_size as long as the ring does not run over
    return at < a.ring_size ? at : at % a.ring_size;
  };
  int64_t tokens = 0, asked = 0, taken = 0, freed = 0;  // of the requests before this pass
  bool long_ones = false;
  for (uint32_t base = 0; base < (uint32_t)a.num_seqs; base += kThreads) {
    const uint32_t b = base + threadIdx.x;
    const bool in = b < (uint32_t)a.num_seqs;
    const int held = in ? a.held_lens[b] : 0, seq = in ? a.seq_lens[b] : 0;
    const int fresh = in ? a.new_lens[b] : 0;
    const bool sound = held >= 0 && seq >= 0 && seq <= held && fresh >= -1 &&
                       pages_of(held, P) <= a.max_blocks;
    const int64_t add = fresh > 0 ? fresh : 0;
    const int keep = sound && fresh >= 0 ? seq : 0;
    const int have = sound ? pages_of(held, P) : 0;
    int64_t target = sound ? keep + add : 0;
    bool refused = !sound || pages_of(target, P) > a.max_blocks || target > INT32_MAX;
    if (refused) target = keep;
    Counts sum;
    Counts at = block_scan(Counts(max(0, pages_of(target, P) - have),
                                           max(0, have - pages_of(target, P)), add),
                                    warp_sums, sum);
    const int64_t all_asked = asked + sum.taken();
    if (all_asked > avail) {  // the ring runs dry in this pass or before
      const int grow = max(0, pages_of(target, P) - have);
      if (grow > 0 && asked + at.taken() + grow > avail) {
        refused = true;
        target = keep;
      }
      at = block_scan(Counts(max(0, pages_of(target, P) - have),
                                      max(0, have - pages_of(target, P)), add),
                               warp_sums, sum);
    }
    asked = all_asked;
    if (in && refused && (add > 0 || !sound)) report_error(a.err, kErrDeviceCheck);
    const int want = pages_of(target, P);
    const int64_t first = tokens + at.tokens;
    ps.taken_at[threadIdx.x] = at.taken();
    ps.freed_at[threadIdx.x] = at.freed();
    ps.from[threadIdx.x] = min(have, want);
    if (in) {
      a.kv_lens[b] = (int32_t)target;
      a.cu_new[b] = (int32_t)min(first, (int64_t)INT32_MAX);
    }
    __syncthreads();
    // pages change hands, a thread each: what a request gives back may be thousands
    for (uint32_t i = threadIdx.x; i < (uint32_t)sum.freed(); i += kThreads) {
      const int o = owner(ps.freed_at, kThreads, i);
      a.free_pages[in_ring(tail0 + freed + i)] =
          a.block_table[(int64_t)(base + o) * a.max_blocks + ps.from[o] + i - ps.freed_at[o]];
    }
    for (uint32_t i = threadIdx.x; i < (uint32_t)sum.taken(); i += kThreads) {
      const int o = owner(ps.taken_at, kThreads, i);
      a.block_table[(int64_t)(base + o) * a.max_blocks + ps.from[o] + i - ps.taken_at[o]] =
          a.free_pages[in_ring(head0 + taken + i)];
    }
    taken += sum.taken();
    freed += sum.freed();
    tokens += sum.tokens;
    long_ones |= __syncthreads_or(in && add > kFew) != 0;
    // a request's first slot, or all of few, by its own thread
    if (in && add > 0) {
      const int n = add <= kFew && write_slots ? (int)add : 1;
      const int32_t* row = a.block_table + (int64_t)b * a.max_blocks;
      for (int t = 0; t < n; ++t) {
        const int64_t i = first + t;
        const int pos = keep + t;
        if (i < a.max_tokens) a.slots[i] = refused ? -1 : (int64_t)row[pos / P] * P + pos % P;
      }
    }
  }
  if (threadIdx.x == 0) {
    a.cu_new[a.num_seqs] = (int32_t)min(tokens, (int64_t)INT32_MAX);
    a.free_range_out[0] = head + taken;
    a.free_range_out[1] = tail + freed;
    if (tokens > a.max_tokens || avail - taken + freed > a.ring_size)
      report_error(a.err, kErrDeviceCheck);
  }
  if (!write_slots) return;
  const int live = (int)min(tokens, (int64_t)a.max_tokens);
  if (long_ones) {
    __syncthreads();  // cu_new, kv_lens, block_table and the first slots are in place
    for (int i = threadIdx.x; i < live; i += kThreads) {
      const int b = owner(a.cu_new, a.num_seqs, i);
      const int first = a.cu_new[b], n = a.cu_new[b + 1] - first;
      if (n > kFew && i != first) a.slots[i] = slot_of(a, b, i, first, n);
    }
  }
  for (int i = live + threadIdx.x; i < a.max_tokens; i += kThreads) a.slots[i] = -1;
}

constexpr int kOffsets = 4096;  // offsets that the slot kernel keeps in shared memory

__global__ void __launch_bounds__(256) slots_kernel(TableArgs a) {
  __shared__ int32_t cu[kOffsets + 1];
  const bool here = a.num_seqs <= kOffsets;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // of the kernel before
  if (here)
    for (int i = threadIdx.x; i <= a.num_seqs; i += 256) cu[i] = a.cu_new[i];
  __syncthreads();
  const int32_t* offsets = here ? cu : a.cu_new;
  const int tokens = offsets[a.num_seqs];
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < (uint32_t)a.max_tokens;
       i += gridDim.x * 256) {
    if (i >= (uint32_t)tokens) {
      a.slots[i] = -1;
      continue;
    }
    const int b = owner(offsets, a.num_seqs, i);
    const int first = offsets[b];
    if (i != (uint32_t)first) a.slots[i] = slot_of(a, b, i, first, offsets[b + 1] - first);
  }
}

// Up to this many slots are written by the first kernel: a few passes of its CTA, which
// cost less than a second launch (2 to 3 us).
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
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min((a.max_tokens - 1) / 256 + 1, 4 * sms));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, slots_kernel, a);
}

}  // namespace kda
