// kda_cache_pages.cu -- pages that several requests hold: kda_cache_fork (rows of a block
// table made from rows of another, pages nobody holds any more given back), kda_cache_compact
// (pages in use moved to the lowest numbers) and kda_cache_copy (the bytes).
//
// Who holds a page is not kept anywhere: it follows from the tables, so these calls and
// kda_cache_tables cannot disagree about it.  Each call marks the pages of a table's rows in a
// bitmap (a bit a page, set by an atomic OR: the order does not matter), and everything else
// follows from sums over the bitmap's words in the pages' order, which one CTA takes: 32 pages
// a word, so 131072 pages are four words a thread.  What bounds the calls is the chain of
// launches and dependent loads; what bounds the copies is HBM.
#include <algorithm>

#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int kThreads = 1024;  // of the CTA that sums

__device__ __forceinline__ int pages_of(int64_t tokens, int page) {
  return (int)((tokens + page - 1) / page);
}

// Programmatic dependent launch: the kernels of a call wait here for the memory of the one
// before.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void set_bit(uint32_t* map, int page) {
  const uint32_t bit = 1u << (page & 31);
  uint32_t* w = map + (page >> 5);
  // shared pages are marked by many rows; a stale word only costs the atomic
  if (!(*(volatile uint32_t*)w & bit)) atomicOr(w, bit);
}
__device__ __forceinline__ bool bit_of(const uint32_t* map, int page) {
  return map[page >> 5] >> (page & 31) & 1;
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

struct ForkScratch {
  uint32_t *old_map, *whole_map, *tail_map;  // pages of old rows, of new rows whole, kept tails
  int32_t* first;                            // [num_pages] lowest row with the page as its tail
  Row* rows;                                 // [num_seqs]
};

// Zeroes the bitmaps and settles each new row: a row whose parent or length does not make sense
// keeps nothing.
__global__ void __launch_bounds__(256) fork_rows_kernel(ForkArgs a, ForkScratch s, int words) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x, n = gridDim.x * 256;
  for (uint32_t w = i; w < (uint32_t)words; w += n)
    s.old_map[w] = s.whole_map[w] = s.tail_map[w] = 0;
  const int P = a.page_size;
  for (uint32_t b = i; b < (uint32_t)a.num_seqs; b += n) {
    const int parent = a.parents[b];
    Row r{0, -1};
    if (parent >= 0 && parent < a.old_seqs) {
      const int held = a.held_lens[parent], keep = a.keep_lens[b];
      if (held >= 0 && pages_of(held, P) <= a.max_blocks && keep >= 0 && keep <= held) {
        r.keep = keep;
        if (keep % P) {
          const int page = a.block_table[(int64_t)parent * a.max_blocks + keep / P];
          if (page >= 0 && page < a.num_pages) {
            r.tail = page;
            s.first[page] = INT32_MAX;
          }
        }
      } else {
        report_error(a.err, kErrDeviceCheck);
      }
    } else if (parent != -1) {
      report_error(a.err, kErrDeviceCheck);
    }
    s.rows[b] = r;
  }
}

constexpr int kColumns = 1024;  // of a row that one CTA takes
// The first of them (grid_of); columns count up in 32 bits without a sign.
__device__ __forceinline__ int64_t first_column() {
  return ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * kColumns;
}

// Marks the old rows' pages; writes the new rows and marks theirs.
__global__ void __launch_bounds__(256) fork_mark_kernel(ForkArgs a, ForkScratch s) {
  wait_for_previous();
  const int P = a.page_size;
  const int64_t col0 = first_column();
  if (col0 >= a.max_blocks) return;
  const int cols = (int)min((int64_t)a.max_blocks, col0 + kColumns);
  for (uint32_t r = blockIdx.x; r < (uint32_t)a.old_seqs + (uint32_t)a.num_seqs; r += gridDim.x) {
    if (r < (uint32_t)a.old_seqs) {
      const int held = a.held_lens[r];
      if (held < 0 || pages_of(held, P) > a.max_blocks) {  // its pages stay where they are
        if (threadIdx.x == 0 && col0 == 0) report_error(a.err, kErrDeviceCheck);
        continue;
      }
      const int n = min(cols, pages_of(held, P));
      for (uint32_t c = (uint32_t)col0 + threadIdx.x; c < (uint32_t)n; c += 256) {
        const int page = a.block_table[(int64_t)r * a.max_blocks + c];
        if (page >= 0 && page < a.num_pages)
          set_bit(s.old_map, page);
        else
          report_error(a.err, kErrDeviceCheck);
      }
    } else {
      const int b = (int)(r - a.old_seqs);
      const Row row = s.rows[b];
      const int whole = row.keep / P, n = pages_of(row.keep, P);
      const int32_t* from = a.block_table + (int64_t)max(0, a.parents[b]) * a.max_blocks;
      int32_t* to = a.block_table_out + (int64_t)b * a.max_blocks;
      for (uint32_t c = (uint32_t)col0 + threadIdx.x; c < (uint32_t)cols; c += 256) {
        const int page = c < (uint32_t)n ? from[c] : -1;
        to[c] = page;
        if (c < (uint32_t)whole && page >= 0 && page < a.num_pages) set_bit(s.whole_map, page);
      }
      if (threadIdx.x == 0 && col0 == 0 && row.tail >= 0) atomicMin(s.first + row.tail, b);
    }
  }
}

// Settles the unfinished last pages and gives back what nobody holds.
__global__ void __launch_bounds__(kThreads) fork_settle_kernel(ForkArgs a, ForkScratch s,
                                                               int words) {
  __shared__ int warp_sums[32];
  wait_for_previous();
  const int P = a.page_size;
  int64_t head = a.free_range[0], tail = a.free_range[1];
  if (!(head >= 0 && tail >= head && tail - head <= a.ring_size)) {
    head = tail = 0;
    if (threadIdx.x == 0) report_error(a.err, kErrDeviceCheck);
  }
  const int64_t avail = tail - head;
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
          copy[1] = a.free_pages[(head + at) % a.ring_size];
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
  int64_t at = block_scan(count, warp_sums, freed) + tail;
  for (int w = w0; w < w1; ++w) {
    uint32_t gone = s.old_map[w] & ~(s.whole_map[w] | *(volatile uint32_t*)(s.tail_map + w));
    for (; gone; gone &= gone - 1) a.free_pages[at++ % a.ring_size] = w * 32 + __ffs(gone) - 1;
  }
  if (threadIdx.x == 0) {
    a.free_range_out[0] = head + taken;
    a.free_range_out[1] = tail + freed;
    if (avail - taken + freed > a.ring_size) report_error(a.err, kErrDeviceCheck);
  }
}

// --------------------------------------------------------------- compact ----

struct CompactScratch {
  uint32_t* live;    // bitmap
  int32_t* before;   // [words] pages in use before each word's first
  int32_t* count;    // pages in use
};

__global__ void __launch_bounds__(256) compact_clear_kernel(CompactScratch s, int words) {
  for (uint32_t w = blockIdx.x * 256 + threadIdx.x; w < (uint32_t)words; w += gridDim.x * 256)
    s.live[w] = 0;
}

__global__ void __launch_bounds__(256) compact_mark_kernel(CompactArgs a, CompactScratch s) {
  wait_for_previous();
  const int64_t col0 = first_column();
  for (uint32_t r = blockIdx.x; r < (uint32_t)a.num_seqs; r += gridDim.x) {
    const int held = a.held_lens[r];
    const bool sound = held >= 0 && pages_of(held, a.page_size) <= a.max_blocks;
    if (!sound && threadIdx.x == 0 && col0 == 0) report_error(a.err, kErrDeviceCheck);
    const int n = sound ? (int)min(col0 + kColumns, (int64_t)pages_of(held, a.page_size)) : 0;
    for (uint32_t c = (uint32_t)col0 + threadIdx.x; c < (uint32_t)n; c += 256) {
      const int page = a.block_table[(int64_t)r * a.max_blocks + c];
      if (page >= 0 && page < a.num_pages)
        set_bit(s.live, page);
      else
        report_error(a.err, kErrDeviceCheck);
    }
  }
}

// Pages in use before each word, and the list of moves: the i-th page in use at or past their
// number L goes to the i-th free one below it.
__global__ void __launch_bounds__(kThreads) compact_plan_kernel(CompactArgs a, CompactScratch s,
                                                                int words) {
  __shared__ int warp_sums[32];
  __shared__ int before_l;
  wait_for_previous();
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
    a.free_range_out[0] = 0;
    a.free_range_out[1] = a.num_pages - L;
    if (L >> 5 >= words) before_l = L;  // L == num_pages, the words full
  }
  __syncthreads();
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
__global__ void __launch_bounds__(256) compact_rows_kernel(CompactArgs a, CompactScratch s) {
  wait_for_previous();
  const int L = s.count[0];
  // pages in use below L: those that stay
  const int stay = L < a.num_pages
                       ? s.before[L >> 5] + __popc(s.live[L >> 5] & ((1u << (L & 31)) - 1))
                       : L;
  const int64_t col0 = first_column();
  const int cols = (int)min((int64_t)a.max_blocks, col0 + kColumns);
  for (uint32_t r = blockIdx.x; r < (uint32_t)a.num_seqs; r += gridDim.x) {
    const int held = a.held_lens[r];
    const bool sound = held >= 0 && pages_of(held, a.page_size) <= a.max_blocks;
    const int n = sound ? pages_of(held, a.page_size) : 0;
    for (uint32_t c = (uint32_t)col0 + threadIdx.x; c < (uint32_t)cols; c += 256) {
      const int64_t at = (int64_t)r * a.max_blocks + c;
      int page = c < (uint32_t)n ? a.block_table[at] : -1;
      if (page >= L && page < a.num_pages) {
        const int rank = s.before[page >> 5] +
                         __popc(s.live[page >> 5] & ((1u << (page & 31)) - 1)) - stay;
        page = a.copies[3 * (int64_t)rank + 1];
      }
      a.block_table_out[at] = page;
    }
  }
  if (blockIdx.z) return;
  const int64_t n = (int64_t)gridDim.x * gridDim.y * 256;
  for (int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
       i < a.num_pages - L; i += n)
    a.free_pages[i] = L + (int)i;
}

// ------------------------------------------------------------------ copy ----

struct Layers {
  uint8_t* pages[kCopyLayers];
};

constexpr int kVecs = 8;                       // 16-byte words of a thread under way
constexpr int kPart = 256 * kVecs;             // words of a CTA's part of a page

// The items (copy, layer, part of a page) are dealt out to the CTAs in turn.
__global__ void __launch_bounds__(256) copy_kernel(CopyArgs a, Layers layers, int parts) {
  wait_for_previous();
  const int group_vecs = a.group_bytes / 16;
  const int64_t head_vecs = (int64_t)a.groups * group_vecs, page_vecs = head_vecs * a.runs;
  const int64_t items = (int64_t)a.num_copies * a.num_layers * parts;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int part = (int)(item % parts);
    const int64_t rest = item / parts;
    const int layer = (int)(rest % a.num_layers);
    const int32_t* copy = a.copies + 3 * (rest / a.num_layers);
    const int from = __ldg(copy), to = __ldg(copy + 1), tokens = __ldg(copy + 2);
    if (from == -1 || tokens == 0 || from == to) continue;
    if (from < 0 || from >= a.num_pages || to < 0 || to >= a.num_pages || tokens < 0 ||
        tokens > a.groups * 16) {
      if (threadIdx.x == 0) report_error(a.err, kErrDeviceCheck);
      continue;
    }
    // the groups in use of each head, one run where that is all of them
    const int groups = (tokens + 15) / 16;
    const bool all = groups == a.groups;
    const uint32_t run = all ? (uint32_t)page_vecs : (uint32_t)(groups * group_vecs);
    const uint32_t vecs = all ? run : run * (uint32_t)a.runs;
    uint8_t* base = layers.pages[layer];
    const uint4* src = reinterpret_cast<const uint4*>(base) + from * page_vecs;
    uint4* dst = reinterpret_cast<uint4*>(base) + to * page_vecs;
    const uint32_t first = (uint32_t)part * kPart + threadIdx.x;
    uint4 x[kVecs];
    int64_t at[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t v = first + i * 256;
      if (v < vecs) {
        const uint32_t head = v / run;
        at[i] = head * head_vecs + (v - head * run);
        x[i] = __ldcs(src + at[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (first + i * 256 < vecs) __stcs(dst + at[i], x[i]);
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

// Launches a kernel that may start before the one ahead of it in the stream has ended.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Rows in x; parts of a row in y, in z what y has no room for.
dim3 grid_of(int64_t rows, unsigned parts, int most) {
  const unsigned y = std::min(parts, 32768u);
  return dim3((unsigned)std::min<int64_t>(rows, most), y, (parts + y - 1) / y);
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
  const int words = words_of(a.num_pages), most = 8 * sm_count();
  const int64_t work = std::max<int64_t>(std::max(words, a.num_seqs), 1);
  fork_rows_kernel<<<(unsigned)std::min<int64_t>((work + 255) / 256, most), 256, 0, st>>>(a, s,
                                                                                          words);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.old_seqs + a.num_seqs;
  const unsigned parts = (unsigned)(((int64_t)a.max_blocks + kColumns - 1) / kColumns);
  if (rows > 0 && parts > 0) {
    e = launch_after(fork_mark_kernel, grid_of(rows, parts, most), 256, st, a, s);
    if (e != cudaSuccess) return e;
  }
  return launch_after(fork_settle_kernel, dim3(1), kThreads, st, a, s, words);
}

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t st) {
  CompactScratch s;
  compact_layout(a, static_cast<uint8_t*>(a.workspace), &s);
  const int words = words_of(a.num_pages), most = 8 * sm_count();
  compact_clear_kernel<<<std::min((words + 255) / 256 + 1, most), 256, 0, st>>>(s, words);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned parts = (unsigned)(((int64_t)a.max_blocks + kColumns - 1) / kColumns);
  const dim3 grid = grid_of(std::max(a.num_seqs, 1), std::max(parts, 1u), most);
  e = launch_after(compact_mark_kernel, grid, 256, st, a, s);
  if (e != cudaSuccess) return e;
  e = launch_after(compact_plan_kernel, dim3(1), kThreads, st, a, s, words);
  if (e != cudaSuccess) return e;
  return launch_after(compact_rows_kernel, grid, 256, st, a, s);
}

cudaError_t launch_cache_copy(const CopyArgs& a, uint8_t* const* pages, cudaStream_t st) {
  const int64_t vecs = (int64_t)a.groups * a.group_bytes / 16 * a.runs;
  const int parts = (int)((vecs + kPart - 1) / kPart);
  for (int first = 0; first < a.num_layers; first += kCopyLayers) {
    CopyArgs b = a;
    b.num_layers = std::min(a.num_layers - first, kCopyLayers);
    Layers layers = {};
    for (int i = 0; i < b.num_layers; ++i) layers.pages[i] = pages[first + i];
    const int64_t items = (int64_t)b.num_copies * b.num_layers * parts;
    const cudaError_t e =
        launch_after(copy_kernel, dim3((unsigned)std::min<int64_t>(items, 8ll * sm_count())), 256,
                     st, b, layers, parts);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kda
