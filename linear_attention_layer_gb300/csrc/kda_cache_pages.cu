// kda_cache_pages.cu -- pages that several requests hold: kda_cache_fork (rows of a block
// table made from rows of another, pages nobody holds any more given back), kda_cache_compact
// (pages in use moved to the lowest numbers) and kda_cache_copy (the bytes).
//
// Who holds a page is not kept anywhere: it follows from the tables, so these calls and
// kda_cache_tables cannot disagree about it.  Each call marks the pages of a table's rows in a
// bitmap (a bit a page, set by an atomic OR: the order does not matter), and everything else
// follows from sums over the bitmap's words in the pages' order, which one CTA takes: 32 pages
// a word, so 131072 pages are four words a thread.
//
// What bounds the calls is the chain of dependent loads, and launches: the steps of a call (rows
// settled, pages marked, sums, new rows) run in one CTA or one cluster of them, with the bitmaps in
// shared memory and barriers between the steps, or, for large tables, as a kernel each over the
// whole GPU.  The copies are bound by HBM.
//
// Measured (GB300): a fork of one prompt of 2000 tokens into 8 rows 7 us and its 7 copies 2.5 us
// (the host takes 6 and 3); of 256 beams over 4096 tokens at most 10.4 us and 73
// copies in two caches 7 us; a compaction of 4096 pages 9.6 us and its 930 moves of 128 KB, 245 MB in
// and out, 41 us (37 in the kernel, a fifth of the bytes still in L2 at its end).  8192 copies of
// 128 KB, 2.16 GB: 367 us, 357 in the kernel, 0.89 of the measured HBM rate, DRAM 76% busy.
#include <algorithm>

#include "kda_cache.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

using cache::launch_after;
using cache::wait_for_previous;

constexpr int kThreads = 1024;  // of the CTA that sums
constexpr int kBatch = 4;       // entries of a table that a thread has under way

__device__ __forceinline__ int pages_of(int64_t tokens, int page) {
  return (int)((tokens + page - 1) / page);
}

// All CTAs of the cluster, and their memory.
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\t"
      "barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}

// A word of shared memory of another CTA of the cluster, at this CTA's address of it.
__device__ __forceinline__ uint32_t of_cta(const uint32_t* p, int cta) {
  uint32_t at = (uint32_t)__cvta_generic_to_shared(p), x;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(cta));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}

// The CTAs that share a step: this one's number and how many they are.
struct Crew {
  uint32_t cta, ctas;
  __device__ __forceinline__ uint32_t thread() const { return cta * blockDim.x + threadIdx.x; }
  __device__ __forceinline__ uint32_t threads() const { return ctas * blockDim.x; }
};
__device__ __forceinline__ Crew grid_crew() { return Crew{blockIdx.x, gridDim.x}; }

__device__ __forceinline__ void set_bit(uint32_t* map, int page) {
  atomicOr(map + (page >> 5), 1u << (page & 31));
}
__device__ __forceinline__ bool bit_of(const uint32_t* map, int page) {
  return map[page >> 5] >> (page & 31) & 1;
}

// Marks the pages of a batch; shared ones are marked by many rows, so their words are looked at
// first (a stale one only costs the atomic).  A page of -1 is none.
__device__ __forceinline__ void set_bits(uint32_t* map, const int (&page)[kBatch]) {
  uint32_t w[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    w[j] = page[j] >= 0 ? *(volatile uint32_t*)(map + (page[j] >> 5)) : ~0u;
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    if (!(w[j] >> (page[j] & 31) & 1)) set_bit(map, page[j]);
}

// Whether a row of a table makes sense.
__device__ __forceinline__ bool sound(int held, int page_size, int max_blocks) {
  return held >= 0 && pages_of(held, page_size) <= max_blocks;
}

// Marks the pages that rows hold.
__device__ __forceinline__ void mark_rows(uint32_t* map, const int32_t* table, const int32_t* lens,
                                          int rows, int columns, int page_size, int num_pages,
                                          int* err, Crew crew) {
  const uint64_t total = (uint64_t)(uint32_t)rows * (uint32_t)columns, step = crew.threads();
  for (uint64_t i = crew.thread(); i < total; i += kBatch * step) {
    int held[kBatch], page[kBatch];
    uint32_t col[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint64_t e = i + j * step;
      held[j] = 0;
      col[j] = 0;
      if (e < total) {
        const uint32_t row = (uint32_t)e / (uint32_t)columns;
        col[j] = (uint32_t)e - row * (uint32_t)columns;
        held[j] = lens[row];
      }
    }
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      page[j] = -1;
      if (sound(held[j], page_size, columns) && col[j] < (uint32_t)pages_of(held[j], page_size))
        page[j] = table[i + j * step];
      else
        col[j] = ~0u;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (col[j] != ~0u && (page[j] < 0 || page[j] >= num_pages)) page[j] = -1, bad = true;
    if (bad) report_error(err, kErrDeviceCheck);
    set_bits(map, page);
  }
}

// Sums of the CTA's threads before this one; `total` gets the sum of all.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();  // the sums of the call before are read
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  const int mine = lane < kThreads / 32 ? warp_sums[lane] : 0;
  int s = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  return incl - x + __shfl_sync(0xffffffffu, s - mine, warp);
}

// ------------------------------------------------------------------ fork ----

// A new row: what it keeps and its unfinished last page (-1: none).
struct Row {
  int32_t keep, tail;
};

// Rows that make no sense: their pages stay where they are.
__device__ __forceinline__ void check_rows(const int32_t* lens, int rows, int columns,
                                           int page_size, int* err) {
  const Crew crew = grid_crew();
  for (uint32_t r = crew.thread(); r < (uint32_t)rows; r += crew.threads())
    if (!sound(lens[r], page_size, columns)) report_error(err, kErrDeviceCheck);
}

struct ForkScratch {
  uint32_t *old_map, *whole_map, *tail_map;  // pages of old rows, of new rows whole, kept tails
  int32_t* first;                            // [num_pages] lowest row with the page as its tail
  Row* rows;                                 // [num_seqs]
};

// Zeroes the bitmaps and settles each new row: a row whose parent or length does not make sense
// keeps nothing.  Of crews that do the same, the lead speaks for all.
__device__ __forceinline__ void fork_rows(const ForkArgs& a, const ForkScratch& s, int words,
                                          Crew crew, bool lead) {
  const uint32_t i = crew.thread(), n = crew.threads();
  for (uint32_t w = i; w < (uint32_t)words; w += n)
    s.old_map[w] = s.whole_map[w] = s.tail_map[w] = 0;
  const int P = a.page_size;
  for (uint32_t b = i; b < (uint32_t)a.num_seqs; b += n) {
    const int parent = a.parents[b];
    Row r{0, -1};
    if (parent >= 0 && parent < a.old_seqs) {
      const int held = a.held_lens[parent], keep = a.keep_lens[b];
      if (sound(held, P, a.max_blocks) && keep >= 0 && keep <= held) {
        r.keep = keep;
        if (keep % P) {
          const int page = a.block_table[(int64_t)parent * a.max_blocks + keep / P];
          if (page >= 0 && page < a.num_pages) {
            r.tail = page;
            if (lead) s.first[page] = INT32_MAX;
          }
        }
      } else if (lead) {
        report_error(a.err, kErrDeviceCheck);
      }
    } else if (lead && parent != -1) {
      report_error(a.err, kErrDeviceCheck);
    }
    s.rows[b] = r;
  }
}

__device__ __forceinline__ void fork_mark_old(const ForkArgs& a, const ForkScratch& s, Crew crew) {
  mark_rows(s.old_map, a.block_table, a.held_lens, a.old_seqs, a.max_blocks, a.page_size,
            a.num_pages, a.err, crew);
}

// The lowest row that ends inside each page.
__device__ __forceinline__ void fork_first(const ForkArgs& a, const ForkScratch& s, Crew crew) {
  for (uint32_t b = crew.thread(); b < (uint32_t)a.num_seqs; b += crew.threads()) {
    const int tail = s.rows[b].tail;
    if (tail >= 0) atomicMin(s.first + tail, (int)b);
  }
}

// Writes the new rows and marks their pages.
__device__ __forceinline__ void fork_mark_new(const ForkArgs& a, const ForkScratch& s, Crew crew) {
  const int P = a.page_size;
  const uint64_t total = (uint64_t)a.num_seqs * a.max_blocks, step = crew.threads();
  for (uint64_t i = crew.thread(); i < total; i += kBatch * step) {
    int keep[kBatch], parent[kBatch], page[kBatch];
    uint32_t col[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint64_t e = i + j * step;
      keep[j] = parent[j] = 0;
      col[j] = 0;
      if (e < total) {
        const uint32_t row = (uint32_t)e / (uint32_t)a.max_blocks;
        col[j] = (uint32_t)e - row * (uint32_t)a.max_blocks;
        keep[j] = s.rows[row].keep;
        parent[j] = a.parents[row];
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      page[j] = col[j] < (uint32_t)pages_of(keep[j], P)
                    ? a.block_table[(int64_t)parent[j] * a.max_blocks + col[j]]
                    : -1;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint64_t e = i + j * step;
      if (e < total) a.block_table_out[e] = page[j];
      if (col[j] >= (uint32_t)(keep[j] / P) || page[j] >= a.num_pages) page[j] = -1;
    }
    set_bits(s.whole_map, page);
  }
}

// The ring of free pages as a call finds it; empty if its range makes no sense.  It runs on from
// head0 and tail0 without a division.
struct FreeRing {
  int64_t head, tail, head0, tail0;
};
__device__ __forceinline__ FreeRing load_ring(const ForkArgs& a, bool lead) {
  FreeRing r{a.free_range[0], a.free_range[1], 0, 0};
  if (!(r.head >= 0 && r.tail >= r.head && r.tail - r.head <= a.ring_size)) {
    r.head = r.tail = 0;
    if (lead && threadIdx.x == 0) report_error(a.err, kErrDeviceCheck);
  }
  r.head0 = r.head % a.ring_size;
  r.tail0 = r.tail % a.ring_size;
  return r;
}

// Settles the unfinished last pages and gives back what nobody holds: one CTA.
__device__ __forceinline__ void fork_settle(const ForkArgs& a, const ForkScratch& s,
                                            const FreeRing& ring, int words, int* warp_sums) {
  const int P = a.page_size;
  const int64_t avail = ring.tail - ring.head;
  auto in_ring = [&](int64_t at) { return at < a.ring_size ? at : at % a.ring_size; };
  int64_t asked = 0;
  for (uint32_t base = 0; base < (uint32_t)a.num_seqs; base += kThreads) {
    const uint32_t b = base + threadIdx.x;
    Row r{0, -1};
    bool move = false;
    if (b < (uint32_t)a.num_seqs) {
      r = s.rows[b];
      if (r.tail >= 0) {
        move = bit_of(s.whole_map, r.tail) || s.first[r.tail] != (int)b;
        if (!move) set_bit(s.tail_map, r.tail);
      }
    }
    int total;
    const int64_t at = asked + block_scan(move, warp_sums, total);
    if (b < (uint32_t)a.num_seqs) {
      int32_t copy[3] = {-1, -1, 0};
      if (move) {
        int32_t* entry = a.block_table_out + (int64_t)b * a.max_blocks + r.keep / P;
        if (at < avail) {
          copy[0] = r.tail;
          copy[1] = a.free_pages[in_ring(ring.head0 + at)];
          copy[2] = r.keep % P;
          *entry = copy[1];
        } else {  // no page is left: the row ends with its last whole one
          report_error(a.err, kErrDeviceCheck);
          *entry = -1;
          r.keep -= r.keep % P;
        }
      }
      a.kv_lens[b] = r.keep;
#pragma unroll
      for (int i = 0; i < 3; ++i) a.copies[3 * (int64_t)b + i] = copy[i];
    }
    asked += total;
  }
  const int64_t taken = min(asked, avail);
  __syncthreads();  // tail_map
  const int per = (words + kThreads - 1) / kThreads;
  const int w0 = min(words, per * (int)threadIdx.x), w1 = min(words, w0 + per);
  int count = 0, freed;
  for (int w = w0; w < w1; ++w)
    count += __popc(s.old_map[w] & ~(s.whole_map[w] | *(volatile uint32_t*)(s.tail_map + w)));
  int64_t at = block_scan(count, warp_sums, freed) + ring.tail0;
  for (int w = w0; w < w1; ++w) {
    uint32_t gone = s.old_map[w] & ~(s.whole_map[w] | *(volatile uint32_t*)(s.tail_map + w));
    for (; gone; gone &= gone - 1) a.free_pages[in_ring(at++)] = w * 32 + __ffs(gone) - 1;
  }
  if (threadIdx.x == 0) {
    a.free_range_out[0] = ring.head + taken;
    a.free_range_out[1] = ring.tail + freed;
    if (avail - taken + freed > a.ring_size) report_error(a.err, kErrDeviceCheck);
  }
}

// A call in one launch: CTAs CTAs, one or a cluster, with their bitmaps and rows in shared memory.
// Each settles all rows for itself; marks its part of the entries in its own bitmap, half of the
// CTAs the old rows', half the new ones'; and the first one puts the bitmaps together.
constexpr int kCluster = 8;
constexpr int kMapWords = 2048, kMostRows = 1024;

template <int CTAS>
__global__ void __launch_bounds__(kThreads) fork_kernel(ForkArgs a, int32_t* first, int words) {
  __shared__ uint32_t maps[3][kMapWords];
  __shared__ Row rows[kMostRows];
  __shared__ int warp_sums[32];
  const ForkScratch s{maps[0], maps[1], maps[2], first, rows};
  const bool lead = blockIdx.x == 0;
  const Crew alone{0, 1};
  wait_for_previous();
  const FreeRing ring = load_ring(a, lead);
  check_rows(a.held_lens, a.old_seqs, a.max_blocks, a.page_size, a.err);
  fork_rows(a, s, words, alone, lead);
  __syncthreads();
  if (lead) fork_first(a, s, alone);
  if constexpr (CTAS == 1) {
    fork_mark_old(a, s, alone);
    fork_mark_new(a, s, alone);
    __syncthreads();
  } else {
    const Crew half{blockIdx.x % (CTAS / 2), CTAS / 2};
    if (blockIdx.x < CTAS / 2)
      fork_mark_old(a, s, half);
    else
      fork_mark_new(a, s, half);
    cluster_sync();
    if (lead)
      for (int w = threadIdx.x; w < words; w += kThreads) {
        uint32_t held = maps[0][w], whole = 0;
#pragma unroll
        for (int i = 1; i < CTAS / 2; ++i) held |= of_cta(&maps[0][w], i);
#pragma unroll
        for (int i = CTAS / 2; i < CTAS; ++i) whole |= of_cta(&maps[1][w], i);
        maps[0][w] = held;
        maps[1][w] = whole;
      }
    cluster_sync();  // before the others leave
  }
  if (lead) fork_settle(a, s, ring, words, warp_sums);
}
// The same as a kernel each.
__global__ void __launch_bounds__(256) fork_rows_kernel(ForkArgs a, ForkScratch s, int words) {
  check_rows(a.held_lens, a.old_seqs, a.max_blocks, a.page_size, a.err);
  fork_rows(a, s, words, grid_crew(), true);
}
__global__ void __launch_bounds__(256) fork_mark_kernel(ForkArgs a, ForkScratch s) {
  wait_for_previous();
  fork_first(a, s, grid_crew());
  fork_mark_old(a, s, grid_crew());
  fork_mark_new(a, s, grid_crew());
}
__global__ void __launch_bounds__(kThreads) fork_settle_kernel(ForkArgs a, ForkScratch s,
                                                               int words) {
  __shared__ int warp_sums[32];
  wait_for_previous();
  fork_settle(a, s, load_ring(a, true), words, warp_sums);
}

// --------------------------------------------------------------- compact ----

struct CompactScratch {
  uint32_t* live;    // bitmap
  int32_t* before;   // [words] pages in use before each word's first
  int32_t* count;    // pages in use
};

__device__ __forceinline__ void compact_clear(const CompactArgs& a, uint32_t* live, int words,
                                              Crew crew) {
  for (uint32_t w = crew.thread(); w < (uint32_t)words; w += crew.threads()) live[w] = 0;
  check_rows(a.held_lens, a.num_seqs, a.max_blocks, a.page_size, a.err);
}

__device__ __forceinline__ void compact_mark(const CompactArgs& a, uint32_t* live, Crew crew) {
  mark_rows(live, a.block_table, a.held_lens, a.num_seqs, a.max_blocks, a.page_size, a.num_pages,
            a.err, crew);
}

// Pages in use before each word, and the list of moves: the i-th page in use at or past their
// number L goes to the i-th free one below it.
// One CTA, or several that do the same, of which the lead writes.
__device__ __forceinline__ void compact_plan(const CompactArgs& a, const CompactScratch& s,
                                             int words, int* warp_sums, int& before_l, bool lead) {
  const int per = (words + kThreads - 1) / kThreads;
  const int w0 = min(words, per * (int)threadIdx.x), w1 = min(words, w0 + per);
  int count = 0, L;
  for (int w = w0; w < w1; ++w) count += __popc(s.live[w]);
  const int at0 = block_scan(count, warp_sums, L);
  int at = at0;
  for (int w = w0; w < w1; ++w) {
    const uint32_t bits = s.live[w];
    s.before[w] = at;
    if (L >> 5 == w) before_l = at + __popc(bits & ((1u << (L & 31)) - 1));
    at += __popc(bits);
  }
  if (threadIdx.x == 0) {
    s.count[0] = L;
    if (lead) {
      a.free_range_out[0] = 0;
      a.free_range_out[1] = a.num_pages - L;
    }
    if (L >> 5 >= words) before_l = L;  // L == num_pages, the words full
  }
  __syncthreads();
  if (!lead) return;
  const int stay = before_l, moves = L - stay;
  at = at0;
  for (int w = w0; w < w1; ++w) {
    const uint32_t bits = s.live[w];
    const int page0 = w * 32;
    // pages of this word below L and the others
    const uint32_t low = page0 + 32 <= L ? ~0u : page0 >= L ? 0u : (1u << (L & 31)) - 1;
    int hole = page0 - at;  // free pages before this word (all below L while it matters)
    for (uint32_t x = ~bits & low; x; x &= x - 1, ++hole)
      a.copies[3 * (int64_t)hole + 1] = page0 + __ffs(x) - 1;
    int mover = at + __popc(bits & low) - stay;
    for (uint32_t x = bits & ~low; x; x &= x - 1, ++mover) {
      a.copies[3 * (int64_t)mover] = page0 + __ffs(x) - 1;
      a.copies[3 * (int64_t)mover + 2] = a.page_size;
    }
    at += __popc(bits);
  }
  for (int i = moves + threadIdx.x; i < a.num_pages / 2; i += kThreads) {
    a.copies[3 * (int64_t)i] = a.copies[3 * (int64_t)i + 1] = -1;
    a.copies[3 * (int64_t)i + 2] = 0;
  }
}

// The rows with the pages' new numbers, and the ring.
__device__ __forceinline__ void compact_rows(const CompactArgs& a, const CompactScratch& s,
                                             Crew crew) {
  const int L = s.count[0];
  // pages in use below L: those that stay
  const int stay = L < a.num_pages
                       ? s.before[L >> 5] + __popc(s.live[L >> 5] & ((1u << (L & 31)) - 1))
                       : L;
  const uint64_t total = (uint64_t)a.num_seqs * a.max_blocks, step = crew.threads();
  for (uint64_t i = crew.thread(); i < total; i += kBatch * step) {
    int held[kBatch], page[kBatch];
    uint32_t col[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint64_t e = i + j * step;
      held[j] = 0;
      col[j] = 0;
      if (e < total) {
        const uint32_t row = (uint32_t)e / (uint32_t)a.max_blocks;
        col[j] = (uint32_t)e - row * (uint32_t)a.max_blocks;
        held[j] = a.held_lens[row];
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      page[j] = sound(held[j], a.page_size, a.max_blocks) &&
                        col[j] < (uint32_t)pages_of(held[j], a.page_size)
                    ? a.block_table[i + j * step]
                    : -1;
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (page[j] >= L && page[j] < a.num_pages) {
        const int w = page[j] >> 5;
        const int rank =
            s.before[w] + __popc(s.live[w] & ((1u << (page[j] & 31)) - 1)) - stay;
        page[j] = a.copies[3 * (int64_t)rank + 1];
      }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (i + j * step < total) a.block_table_out[i + j * step] = page[j];
  }
  for (int64_t i = crew.thread(); i < a.num_pages - L; i += crew.threads())
    a.free_pages[i] = L + (int)i;
}

// A call in one launch, as fork_kernel; every CTA puts the bitmaps together for itself.
template <int CTAS>
__global__ void __launch_bounds__(kThreads) compact_kernel(CompactArgs a, int words) {
  __shared__ uint32_t mine[kMapWords], live[CTAS == 1 ? 1 : kMapWords];
  __shared__ int before[kMapWords], warp_sums[32], before_l, count;
  const CompactScratch s{CTAS == 1 ? mine : live, before, &count};
  const bool lead = blockIdx.x == 0;
  wait_for_previous();
  compact_clear(a, mine, words, Crew{0, 1});
  __syncthreads();
  compact_mark(a, mine, grid_crew());
  if constexpr (CTAS == 1) {
    __syncthreads();
  } else {
    cluster_sync();
    for (int w = threadIdx.x; w < words; w += kThreads) {
      uint32_t x = 0;
#pragma unroll
      for (int i = 0; i < CTAS; ++i) x |= of_cta(&mine[w], i);
      live[w] = x;
    }
    __syncthreads();
  }
  compact_plan(a, s, words, warp_sums, before_l, lead);
  if constexpr (CTAS == 1)
    __syncthreads();
  else
    cluster_sync();  // the moves; and before a CTA leaves, whose bitmap the others read
  compact_rows(a, s, grid_crew());
}
// The same as a kernel each.
__global__ void __launch_bounds__(256) compact_clear_kernel(CompactArgs a, CompactScratch s,
                                                            int words) {
  compact_clear(a, s.live, words, grid_crew());
}
__global__ void __launch_bounds__(256) compact_mark_kernel(CompactArgs a, CompactScratch s) {
  wait_for_previous();
  compact_mark(a, s.live, grid_crew());
}
__global__ void __launch_bounds__(kThreads) compact_plan_kernel(CompactArgs a, CompactScratch s,
                                                                int words) {
  __shared__ int warp_sums[32];
  __shared__ int before_l;
  wait_for_previous();
  compact_plan(a, s, words, warp_sums, before_l, true);
}
__global__ void __launch_bounds__(256) compact_rows_kernel(CompactArgs a, CompactScratch s) {
  wait_for_previous();
  compact_rows(a, s, grid_crew());
}

// ------------------------------------------------------------------ copy ----

struct Layers {
  uint8_t* pages[kCopyLayers];
};

constexpr int kVecs = 8;            // 16-byte words of a thread under way
constexpr int kPart = 256 * kVecs;  // words of a part of a page at most
constexpr int kList = 256;          // items that a CTA looks at in one go

// The items (copy, layer, part of a page) are dealt out to the CTAs in turn.  A list of copies
// may be empty for the most part: a CTA looks at its items together, a thread each, and keeps
// those that ask for something.
__global__ void __launch_bounds__(256, 4) copy_kernel(CopyArgs a, Layers layers, int parts,
                                                      int part_vecs) {
  __shared__ int4 list[kList];  // from, to, tokens, layer and part
  __shared__ int count;
  wait_for_previous();
  const uint32_t group_vecs = a.group_bytes / 16;
  const uint32_t head_vecs = a.groups * group_vecs, page_vecs = head_vecs * a.runs;
  const uint64_t per_copy = (uint64_t)a.num_layers * parts;
  const uint64_t items = (uint64_t)a.num_copies * per_copy;
  for (uint64_t base = blockIdx.x; base < items; base += (uint64_t)kList * gridDim.x) {
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    const uint64_t item = base + (uint64_t)threadIdx.x * gridDim.x;
    if (item < items) {
      const uint64_t i = item / per_copy;
      const int32_t* copy = a.copies + 3 * i;
      const int from = copy[0], to = copy[1], tokens = copy[2];
      if (from != -1 && tokens != 0 && from != to) {
        if (from >= 0 && from < a.num_pages && to >= 0 && to < a.num_pages && tokens > 0 &&
            tokens <= a.groups * 16)
          list[atomicAdd(&count, 1)] = make_int4(from, to, tokens, (int)(item - i * per_copy));
        else
          report_error(a.err, kErrDeviceCheck);
      }
    }
    __syncthreads();
    const int n = count;
    for (int e = 0; e < n; ++e) {
      const int4 it = list[e];
      const int layer = it.w / parts, part = it.w - layer * parts;
      // the groups in use of each head, one run where that is all of them
      const uint32_t groups = (it.z + 15) / 16;
      const bool all = groups == (uint32_t)a.groups;
      const uint32_t run = all ? page_vecs : groups * group_vecs;
      const uint32_t vecs = all ? run : run * a.runs;
      uint4* const pages = reinterpret_cast<uint4*>(layers.pages[layer]);
      const uint4* const src = pages + (int64_t)it.x * page_vecs;
      uint4* const dst = pages + (int64_t)it.y * page_vecs;
      const uint32_t first = (uint32_t)part * part_vecs + threadIdx.x;
      const uint32_t end = min(vecs, (uint32_t)(part + 1) * part_vecs);
      uint4 x[kVecs];
      uint32_t at[kVecs];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const uint32_t v = first + i * 256, head = v / run;
        at[i] = head * head_vecs + (v - head * run);
        if (v < end) x[i] = __ldcs(src + at[i]);
      }
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (first + i * 256 < end) __stcs(dst + at[i], x[i]);
    }
    __syncthreads();  // the list is read
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// Entries of tables that one CTA takes, and that one cluster does (pages and rows as far as its
// shared memory has room).  In a graph of 20 calls, with one CTA and with the cluster: compactions of
// 600 entries 6.6 and 7.7 us, of 2048 8.3 and 9.3, of 4096 11.3 and 11.2, of 8192 18.9 and 15.1; forks of
// 600 7.2 and 6.7, of 2368 8.6 and 7.7, of 16384 14.5 and 8.2 (a fork alone would take the cluster
// at any size).  Before the launches overlapped: a compaction of 5200 12.4 us with the cluster and
// 14.9 as four kernels, a fork of 35000 12.5 and 15.5 as three.
constexpr int64_t kOneEntries = 1 << 11, kClusterEntries = 1 << 18;
constexpr int kClusterPages = 32 * kMapWords;

// One CTA, or one cluster whose CTAs wait for one another at the barriers between the steps.
template <typename... P, typename... A>
cudaError_t launch_steps(bool one, void (*one_kernel)(P...), void (*kernel)(P...), cudaStream_t st,
                         A... args) {
  if (one) return launch_after(one_kernel, dim3(1), kThreads, 0, st, args...);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// CTAs of a kernel over a table's entries.
unsigned entry_ctas(int64_t entries, int most) {
  const int64_t per = 256 * kBatch;
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>((entries + per - 1) / per, most));
}

int words_of(int pages) { return (int)(((int64_t)pages + 31) / 32); }

size_t fork_layout(const ForkArgs& a, uint8_t* ws, ForkScratch* s) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = ws + at;
    at += up256(bytes);
    return p;
  };
  const size_t map = (size_t)words_of(a.num_pages) * 4;
  ForkScratch r;
  r.old_map = reinterpret_cast<uint32_t*>(take(map));
  r.whole_map = reinterpret_cast<uint32_t*>(take(map));
  r.tail_map = reinterpret_cast<uint32_t*>(take(map));
  r.first = reinterpret_cast<int32_t*>(take((size_t)a.num_pages * 4));
  r.rows = reinterpret_cast<Row*>(take((size_t)a.num_seqs * sizeof(Row)));
  if (s) *s = r;
  return at;
}

size_t compact_layout(const CompactArgs& a, uint8_t* ws, CompactScratch* s) {
  const size_t map = up256((size_t)words_of(a.num_pages) * 4);
  if (s) {
    s->live = reinterpret_cast<uint32_t*>(ws);
    s->before = reinterpret_cast<int32_t*>(ws + map);
    s->count = reinterpret_cast<int32_t*>(ws + 2 * map);
  }
  return 2 * map + 256;
}

}  // namespace

size_t cache_fork_workspace_bytes(const ForkArgs& a) { return fork_layout(a, nullptr, nullptr); }
size_t cache_compact_workspace_bytes(const CompactArgs& a) {
  return compact_layout(a, nullptr, nullptr);
}

cudaError_t launch_cache_fork(const ForkArgs& a, cudaStream_t st) {
  ForkScratch s;
  fork_layout(a, static_cast<uint8_t*>(a.workspace), &s);
  const int words = words_of(a.num_pages);
  const int64_t rows = (int64_t)a.old_seqs + a.num_seqs;
  const int64_t entries = rows * std::max(a.max_blocks, 1);
  if (entries <= kClusterEntries && a.num_pages <= kClusterPages && a.num_seqs <= kMostRows)
    return launch_steps(entries <= kOneEntries, fork_kernel<1>, fork_kernel<kCluster>, st, a, s.first,
                        words);
  const int most = 8 * sm_count();
  fork_rows_kernel<<<(unsigned)std::min<int64_t>(std::max<int64_t>(words, rows) / 256 + 1, most),
                     256, 0, st>>>(
      a, s, words);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_after(fork_mark_kernel, dim3(entry_ctas(rows * a.max_blocks, most)), 256, 0, st, a, s);
  if (e != cudaSuccess) return e;
  return launch_after(fork_settle_kernel, dim3(1), kThreads, 0, st, a, s, words);
}

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t st) {
  CompactScratch s;
  compact_layout(a, static_cast<uint8_t*>(a.workspace), &s);
  const int words = words_of(a.num_pages);
  const int64_t entries = (int64_t)a.num_seqs * std::max(a.max_blocks, 1);
  if (entries <= kClusterEntries && a.num_pages <= kClusterPages)
    return launch_steps(entries <= kOneEntries, compact_kernel<1>, compact_kernel<kCluster>, st, a,
                        words);
  const int most = 8 * sm_count();
  compact_clear_kernel<<<std::min(std::max(words, a.num_seqs) / 256 + 1, most), 256, 0, st>>>(
      a, s, words);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const dim3 ctas(entry_ctas((int64_t)a.num_seqs * a.max_blocks, most));
  e = launch_after(compact_mark_kernel, ctas, 256, 0, st, a, s);
  if (e != cudaSuccess) return e;
  e = launch_after(compact_plan_kernel, dim3(1), kThreads, 0, st, a, s, words);
  if (e != cudaSuccess) return e;
  return launch_after(compact_rows_kernel, ctas, 256, 0, st, a, s);
}

cudaError_t launch_cache_copy(const CopyArgs& a, uint8_t* const* pages, cudaStream_t st) {
  // a page has fewer than 2^27 words; its parts are alike, but for the last
  const int vecs = (int)((int64_t)a.groups * a.group_bytes / 16 * a.runs);
  const int parts = (vecs + kPart - 1) / kPart, part_vecs = (vecs + parts - 1) / parts;
  for (int first = 0; first < a.num_layers; first += kCopyLayers) {
    CopyArgs b = a;
    b.num_layers = std::min(a.num_layers - first, kCopyLayers);
    Layers layers = {};
    for (int i = 0; i < b.num_layers; ++i) layers.pages[i] = pages[first + i];
    const int64_t items = (int64_t)b.num_copies * b.num_layers * parts;
    const cudaError_t e =
        launch_after(copy_kernel, dim3((unsigned)std::min<int64_t>(items, 4ll * sm_count())), 256,
                     0, st, b, layers, parts, part_vecs);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kda
