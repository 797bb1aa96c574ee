// kda_cache_chunk.cu -- kda_cache_attention for many rows per kv head (prefill
// chunks, bf16): causal attention over the 4-bit paged cache on tcgen05.
//
// A unit is a request, a kv head and up to 256 of the rows (new token x query head)
// that share it, as two blocks of 128 rows.  Its keys are walked in tiles of 64,
//     S = q K^T,   P = 2^(S f - m),   l += row sums of P,   O += P V,
// with the running reference m of kda_cache_attention.cu (moved, and O rescaled,
// only when a score passes it by more than 15).  4 * 64 * 128 * D flops a block and
// tile stand against the softmax of 128 x 64 scores and, shared by the blocks, the
// dequantisation of 2 * 64 * D codes: the tensor cores bound it if those two keep
// out of their way.
//
// Operands.  P and q (halves, a power of two per row taken out, see row_scale) are A
// operands in tensor memory; K and V are dequantised to halves in shared memory (code x
// scale is exact), K as a K-major and V as an MN-major B operand -- the same bytes in
// both cases: rows of keys, 64 channels to a 128-byte swizzled row.  With A in tensor
// memory shared memory only feeds B, 64 bytes a cycle of the 128 it has, which leaves room
// for writing the dequantised tiles.  Tensor memory, 512 columns of 32 bits: S 2 x 64,
// P 2 x 32, q 64, O 2 x D: with D = 128 the second block's q has no room there and is an
// A operand in shared memory (its 8 score products then take 48 cycles instead of 32).
// P apart from S is worth that: the next scores are computed while a tile's weights
// are (2048 new tokens at the end of 32768 keys, 32 heads on 8: with P over S, and both
// blocks' q in tensor memory, 822 us; apart, 779).
//
// Warps.  0-3 and 4-7: softmax of the two blocks, a thread a row; 8-11: dequantisation;
// 12 (and 14): issues the matrix products; 13: copies pages into a ring.  Measured slower: two
// threads a row (16 softmax warps of 80 registers, 862 us against 822), eight warps for the
// dequantisation with registers moved to the softmax (876 against 746), and, for up to 128
// rows, the two blocks on alternate tiles of the same rows (no faster than one block).
//
// Work split.  The tiles of all units in one sequence are cut evenly over the CTAs, one
// per SM; parts of a unit are joined by a second kernel.  Units of one chunk differ in
// length (causality), so a planner kernel sums them first.
//
// Measured: the chunk above takes 742 us, 1.44 PFLOP/s, 0.76 of the measured bf16 rate (this
// kernel 722, the launches around it the rest); tensor pipe 63% busy.  A tile of both blocks
// takes about 1600 cycles: 1152 of products, the rest waits for the softmax, whose two
// warps a quadrant take about 1500 (64 exponentials a row and warp alone 256).
#include <math.h>

#include <algorithm>

#include "kda_cache_attention.cuh"

namespace kda {
namespace {

using namespace cache;

constexpr int kBlock = 128;             // rows of a block
constexpr int kRows = 2 * kBlock;       // rows of a unit
constexpr int kKeys = 64;               // keys of a tile
constexpr int kGroups = kKeys / kGroup;
constexpr int kRawStages = 4, kTileStages = 3;
constexpr int kValidRing = 16;          // more tiles than can be under way
// With 8 bits a block of rows has an issuing warp of its own, and the softmax's warps take registers
// from the others (8 bits, the chunk above: 787 us with one issuer and 128 registers for all, 764;
// 4 bits 744 and 756).
template <int BITS>
constexpr int kIssuers = BITS == 8 ? 2 : 1;
template <int BITS>
constexpr int kThreads = 32 * (BITS == 8 ? 16 : 14);
constexpr int kSoftmaxRegs = 160, kDequantRegs = 112, kOtherRegs = 80;
// Whether a launch with this many registers a thread has what the warps take: beyond that the
// softmax's warps would wait without an end.
constexpr bool registers_suffice(int a_thread) {
  return 8 * kSoftmaxRegs + 4 * kDequantRegs + 4 * kOtherRegs <= kThreads<8> / 32 * a_thread;
}
static_assert(registers_suffice(128) && !registers_suffice(127), "the split is that of 128 a thread");
template <int BITS, int REGS>
__device__ __forceinline__ void take_registers() {
  if constexpr (BITS == 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int BITS, int REGS>
__device__ __forceinline__ void leave_registers() {
  if constexpr (BITS == 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
constexpr uint32_t kCols = 512;

struct Plan {
  unsigned long long* tiles;  // [entries + 1] tiles before each entry (request, row unit)
  int2* entry;                // request, row unit
  int* first;                 // [num_seqs + 1] first entry of each request
  OpenUnit* open;             // [ctas]
  float* o;                   // [2 * ctas][kRows][D]
  float2* ml;                 // [2 * ctas][kRows]
};

// Keys that the rows of a unit see at most: those its last row sees.
__device__ __forceinline__ int unit_tiles(const Request& q, int group, int r) {
  const int64_t last = min((int64_t)(r + 1) * kRows, q.rows) - 1;
  const int see = q.kv - q.n + (int)(last / group) + 1;
  return max(1, (see + kKeys - 1) / kKeys);  // rows that see nothing still get their zeros
}

// Sums over the block, inclusive.
__device__ __forceinline__ unsigned long long scan1024(unsigned long long x,
                                                       unsigned long long* sums,
                                                       unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    unsigned long long s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  total = sums[31];
  return warp ? x + sums[warp - 1] : x;
}

__global__ void __launch_bounds__(1024) plan_kernel(View c, AttentionArgs a, RowRange range,
                                                    Plan plan, int max_entries) {
  __shared__ unsigned long long sums[32];
  const int group = a.num_heads / c.kv_heads;
  unsigned long long at = 0, total;
  for (uint32_t base = 0; base < (uint32_t)a.num_seqs; base += 1024) {
    const uint32_t b = base + threadIdx.x;
    const bool in = b < (uint32_t)a.num_seqs;
    Request q;
    const bool live = in && load_request(c, a, b, range, false, q);
    const unsigned long long n = live ? (q.rows + kRows - 1) / kRows : 0;
    const unsigned long long incl = scan1024(n, sums, total);
    if (in) plan.first[b] = (int)min(at + incl - n, (unsigned long long)max_entries);
    at += total;
  }
  // ranges that overlap (malformed offsets) could ask for more entries than there is room for
  const int entries = (int)min(at, (unsigned long long)max_entries);
  if (threadIdx.x == 0) plan.first[a.num_seqs] = entries;
  __syncthreads();
  unsigned long long tiles = 0;
  for (uint32_t base = 0; base < (uint32_t)entries; base += 1024) {
    const uint32_t e = base + threadIdx.x;
    const bool in = e < (uint32_t)entries;
    unsigned long long n = 0;
    if (in) {
      const int b = find_last(plan.first, a.num_seqs, e);
      Request q;
      load_request(c, a, b, range, false, q);
      const int r = e - plan.first[b];
      n = (unsigned long long)unit_tiles(q, group, r) * c.kv_heads;
      plan.entry[e] = make_int2(b, r);
    }
    const unsigned long long incl = scan1024(n, sums, total);
    if (in) plan.tiles[e] = tiles + incl - n;
    tiles += total;
  }
  if (threadIdx.x == 0) plan.tiles[entries] = tiles;
}

// The part of a unit that a CTA works on next.
struct Piece {
  Request q;
  int h, r;
  int b;
  int begin, end;  // tiles
  int tiles;       // of the unit
  int entry;

  // x: first tile of the piece in the sequence of all; stop: the CTA's last + 1.
  __device__ __forceinline__ void set(const View& c, const AttentionArgs& a, const RowRange& range,
                                      const Plan& plan, int entries, unsigned long long x,
                                      unsigned long long stop) {
    entry = find_last(plan.tiles, entries, x);
    const int2 er = plan.entry[entry];
    b = er.x;
    r = er.y;
    load_request(c, a, b, range, false, q);
    tiles = unit_tiles(q, a.num_heads / c.kv_heads, r);
    const unsigned long long off = x - plan.tiles[entry];
    h = (int)(off / tiles);
    begin = (int)(off - (unsigned long long)h * tiles);
    end = (int)min((unsigned long long)tiles, begin + (stop - x));
  }
  __device__ __forceinline__ int rows() const {
    return (int)min(q.rows - (int64_t)r * kRows, (int64_t)kRows);
  }
};

template <int BITS, int D>
struct Smem {
  static constexpr int kTile = kKeys * D * 2;
  static constexpr int kRaw = kGroups * FormLayout<BITS, D>::kGroupBytes;
  alignas(1024) uint8_t k[kTileStages][kTile];
  alignas(1024) uint8_t v[kTileStages][kTile];
  static constexpr bool kQueryHere = D > 64;  // the second block's
  alignas(1024) uint8_t q[kQueryHere ? kBlock * D * 2 : 16];
  alignas(128) uint8_t raw[kRawStages][kRaw];
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];
  uint64_t k_full[kTileStages], k_empty[kTileStages], v_full[kTileStages], v_empty[kTileStages];
  uint64_t q_full[2], s_full[2], s_free[2], p_full[2], o_full[2], issued;
  uint32_t valid[kValidRing];  // groups of a tile that can be read
  uint32_t powers[kValidRing]; // 8 bits: exponent bytes that a tile's K and, times 256, V are under
  uint32_t tmem;
  uint32_t copied;  // tiles whose pages were asked for
  int failed;
};

// A position in a ring of N barriers: index and the parity of the fill being waited for.
template <int N>
struct Ring {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void step() {
    if (++i == N) {
      i = 0;
      parity ^= 1;
    }
  }
};

// Dequantisation of a tile of 8-bit codes, by warp dw of four its group of 16 keys: halves in
// units of the largest power of two that the piece has met, as rows of 128 swizzled bytes: scores
// and O then change their units only where a larger one turns up, in the branch that moves the
// softmax's reference, and a tile costs the softmax what a 4-bit one does (powers of its own for
// each tile, taken into the weights there: 797 us for the chunk above).  A code times 2^-d is
// exact down to 2^-24 of the unit.  Lanes take the 16-byte pieces so that
// eight of them read 128 bytes in a row and write to all banks.
template <int D, bool V>
struct Dequant8 {
  static constexpr int N = D / 32;  // pieces of a lane
  uint4 w[N];

  __device__ __forceinline__ void load(const uint8_t* g) {
    const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if constexpr (V)
        w[n] = *reinterpret_cast<const uint4*>(g + Layout8<D>::kVCodes + sub_of(n) * 512 + lane * 16);
      else  // two keys a time, of channels 32 t + 16 h .. in opposite orders
        w[n] = *reinterpret_cast<const uint4*>(g + half_of(n) * 1024 + key_of(n) * 64 + t * 16);
    }
  }
  // K: the key of piece n, and which 16 of the 32 channels (D = 128)
  __device__ __forceinline__ static int key_of(int n) {
    const int lane = threadIdx.x & 31;
    return 2 * ((lane >> 3) + 4 * (n & 1)) + (lane >> 2 & 1);
  }
  __device__ __forceinline__ static int half_of(int n) {
    return D == 64 ? 0 : (n >> 1) ^ (threadIdx.x >> 1 & 1);
  }
  // V: the sub-block of piece n (D = 128), in opposite orders for neighbouring channels
  __device__ __forceinline__ static int sub_of(int n) {
    return D == 64 ? n : n ^ (threadIdx.x >> 2 & 1);
  }
  // Eight halves of codes x, y to chunk `chunk` of row `row`.
  __device__ __forceinline__ static void put(uint8_t* tile, int row, int chunk, uint32_t x,
                                             uint32_t y, uint32_t f) {
    uint32_t h[4];
    e4m3x4_to_f16(x, h[0], h[1]);
    e4m3x4_to_f16(y, h[2], h[3]);
    if (f != 0x3c003c00u) {
#pragma unroll
      for (int q = 0; q < 4; ++q) h[q] = mul_f16x2(h[q], f);
    }
    *reinterpret_cast<uint4*>(tile + (chunk >> 3) * (kKeys * 128) + row * 128 +
                              (((chunk & 7) ^ (row & 7)) << 4)) =
        make_uint4(h[0], h[1], h[2], h[3]);
  }
  // f: the group's power of two beside the unit, as two halves; left: keys that there are.
  __device__ __forceinline__ void store(uint8_t* tile, int dw, uint32_t f, int left) const {
    const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if constexpr (!V) {
        const int row = dw * kGroup + key_of(n);
        const int chunk = D == 64 ? 2 * t : 4 * t + 2 * half_of(n);  // 8 channels each
        put(tile, row, chunk, w[n].x, w[n].y, f);
        put(tile, row, chunk + 1, w[n].z, w[n].w, f);
      } else if constexpr (D == 128) {
        // tokens 8 (sub / 2) + 2 t + sub % 2, channels 16 (lane / 4) ..
        const int sub = sub_of(n), i = 8 * (sub >> 1) + 2 * t + (sub & 1), g = lane >> 2;
        uint4 x = w[n];
        if (left < kGroup && i >= left) x = make_uint4(0, 0, 0, 0);
        put(tile, dw * kGroup + i, 2 * g, x.x, x.y, f);
        put(tile, dw * kGroup + i, 2 * g + 1, x.z, x.w, f);
      } else {
        // two sub-blocks a time, tokens 2 t and 2 t + 2 of 8 channels a lane
        const int sub = 2 * n + (lane >> 4), g = lane >> 1 & 7;
        const int i = 8 * (sub >> 1) + 4 * (lane & 1) + (sub & 1);
        const uint32_t a = i < left ? ~0u : 0u, b = i + 2 < left ? ~0u : 0u;
        put(tile, dw * kGroup + i, g, w[n].x & a, w[n].y & a, f);
        put(tile, dw * kGroup + i + 2, g, w[n].z & b, w[n].w & b, f);
      }
    }
  }
};

template <int BITS, int D>
__global__ void __launch_bounds__(kThreads<BITS>, 1)
    chunk_kernel(View c, AttentionArgs a, RowRange range, Plan plan, int q_vec) {
  using L = FormLayout<BITS, D>;
  using S = Smem<BITS, D>;
  constexpr uint32_t TS = 0, TP = 128, TQ = 192, TO = 256;  // columns of S, P, q, O
  constexpr bool QS = S::kQueryHere;
  extern __shared__ uint8_t raw_smem[];
  S& sm = *reinterpret_cast<S*>(raw_smem + (-tc::smem_u32(raw_smem) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.num_heads / c.kv_heads;

  if (warp == 12) {
    tc::tmem_alloc(&sm.tmem, kCols);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kRawStages; ++i) {
      tc::mbar_init(&sm.raw_full[i], kGroups + (i == 0 ? a.withheld : 0));
      tc::mbar_init(&sm.raw_empty[i], 4);
    }
    for (int i = 0; i < kTileStages; ++i) {
      tc::mbar_init(&sm.k_full[i], 4);
      tc::mbar_init(&sm.v_full[i], 4);
      tc::mbar_init(&sm.k_empty[i], kIssuers<BITS>);
      tc::mbar_init(&sm.v_empty[i], kIssuers<BITS>);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.q_full[i], 4);
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.s_free[i], 4);
      tc::mbar_init(&sm.p_full[i], 4);
      tc::mbar_init(&sm.o_full[i], 1);
    }
    tc::mbar_init(&sm.issued, kIssuers<BITS>);
    sm.failed = 0;
    tc::mbar_fence_init();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sm.tmem;

  let_next_start();
  if (tid == 0) plan.open[blockIdx.x].last = -1;
  const int entries = plan.first[a.num_seqs];
  const unsigned long long total = entries ? plan.tiles[entries] : 0;
  const unsigned long long per = (total + gridDim.x - 1) / gridDim.x;
  const unsigned long long x0 = min(per * blockIdx.x, total), x1 = min(x0 + per, total);

  // A wait that gives up tells the other warps, who give up as well.  A warp leaves its tiles
  // by a vote, at one place in a tile; until then a thread whose wait gave up goes on with
  // whatever is there (a vote after each wait: 786 us for the chunk above).
  volatile int* failed = &sm.failed;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (wait_phase(bar, parity, a.wait_cycles, failed)) return true;
    *failed = 1;
    report_error(a.err, kErrTimeout);
    return false;
  };
  auto all_ok = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };

  // the warps that issue matrix products, and the blocks of rows that this one is for
  const bool issues = warp == 12 || (kIssuers<BITS> == 2 && warp == 14);
  const int first_blk = kIssuers<BITS> == 2 ? (warp - 12) / 2 : 0;
  if (warp < 8) {
    // ------------------------------------------------------------ softmax ----
    take_registers<BITS, kSoftmaxRegs>();
    const int blk = warp >> 2;
    const int row = tid & (kBlock - 1);
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = lanes + TS + blk * kKeys, tp = lanes + TP + blk * (kKeys / 2),
                   tq = lanes + TQ + blk * (D / 2), to = lanes + TO + blk * D;
    Ring<1> s_full, o_full;
    uint32_t tile_no = 0;  // tiles since the start, over all pieces
    bool ok = true;
    for (unsigned long long x = x0; x < x1 && ok;) {
      Piece p;
      p.set(c, a, range, plan, entries, x, x1);
      x += p.end - p.begin;
      const int rows = p.rows();
      if (blk * kBlock >= rows) {
        tile_no += p.end - p.begin;
        continue;
      }
      const int64_t rr = (int64_t)p.r * kRows + blk * kBlock + row;  // row of the request
      const bool live = blk * kBlock + row < rows;
      const int64_t tok = p.q.bos + rr / group;
      const int head = p.h * group + (int)(rr % group);
      const int see = live ? p.q.kv - p.q.n + (int)(rr / group) + 1 : 0;
      // what every row of the block sees
      const int all_see = p.q.kv - p.q.n + (int)(((int64_t)p.r * kRows + blk * kBlock) / group) + 1;
      // ---- queries: the largest magnitude, then 32 channels at a time ----
      float f;
      {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                   tok * a.q_token_stride + head * a.q_head_stride;
        auto load32 = [&](int i, uint32_t (&w)[16]) {
          if (!live) {
#pragma unroll
            for (int q = 0; q < 16; ++q) w[q] = 0;
          } else if (q_vec) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint4 u = __ldg(reinterpret_cast<const uint4*>(src + i) + q);
              w[4 * q] = u.x, w[4 * q + 1] = u.y, w[4 * q + 2] = u.z, w[4 * q + 3] = u.w;
            }
          } else {
#pragma unroll
            for (int q = 0; q < 16; ++q)
              w[q] = __float_as_uint(IO<__nv_bfloat16>::ld(src + i + 2 * q)) >> 16 |
                     __float_as_uint(IO<__nv_bfloat16>::ld(src + i + 2 * q + 1));
          }
        };
        float top = 0.f;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          uint32_t w[16];
          load32(i, w);
#pragma unroll
          for (int q = 0; q < 16; ++q)
            top = fmaxf(top, fmaxf(fabsf(tc::bf16_lo(w[q])), fabsf(tc::bf16_hi(w[q]))));
        }
        const RowScale rs = row_scale(top, a.scale, exponent_scale(c.k_exp, p.h, 1));
        f = rs.f;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          uint32_t w[16];
          load32(i, w);
#pragma unroll
          for (int q = 0; q < 16; ++q)
            w[q] = tc::pack_f16(tc::bf16_lo(w[q]) * rs.down, tc::bf16_hi(w[q]) * rs.down);
          if (QS && blk == 1) {
            uint8_t* dst = sm.q + (i >> 6) * (kBlock * 128) + row * 128;
            const uint32_t chunk = (i & 63) >> 3;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4*>(dst + (((chunk + q) ^ (row & 7)) << 4)) =
                  make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
          } else {
            tc::tmem_st16u(tq + i / 2, w);
          }
        }
        if (QS && blk == 1)
          tc::fence_proxy_async_smem();
        else
          tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.q_full[blk]);
      }
      float neg = 0.f, thr = -INFINITY;
      // 8 bits: exponent bytes under which the tiles' K and V are (f and O are in their units), and
      // f without K's
      uint32_t powers = 0;
      const float f0 = f;
      uint64_t l2[2] = {0, 0};  // the row's sum, in four parts
      for (int j = p.begin; j < p.end; ++j, ++tile_no) {
        // a wait that gives up lowers the limit, so that the vote below is taken
        if (!wait(&sm.s_full[blk], s_full.parity)) thr = -INFINITY;
        s_full.step();
        tc::tc_fence_after();
        float s[kKeys];
        const int key0 = j * kKeys;
        uint32_t valid, under = 0;
        {
          float h0[32], h1[32];
          tc::tmem_ld32(ts, h0);
          tc::tmem_ld32(ts + 32, h1);
          valid = *(volatile uint32_t*)&sm.valid[tile_no % kValidRing];
          if constexpr (BITS == 8) under = *(volatile uint32_t*)&sm.powers[tile_no % kValidRing];
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = h0[i], s[32 + i] = h1[i];
        }
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.s_free[blk]);
        if (key0 + kKeys > all_see || valid != (1u << kGroups) - 1) {
#pragma unroll
          for (int i = 0; i < kKeys; ++i)
            if (key0 + i >= see || !(valid >> (i / kGroup) & 1)) s[i] = -INFINITY;
        }
        float t4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < kKeys - 4; i += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q) t4[q] = tc::max3(t4[q], s[i + q], s[i + 4 + q]);
        const float top = fmaxf(tc::max3(t4[0], s[kKeys - 4], s[kKeys - 3]),
                                tc::max3(tc::max3(t4[1], t4[2], t4[3]), s[kKeys - 2], s[kKeys - 1]));
        bool waited = false;
        if (__any_sync(0xffffffffu, top > thr || (BITS == 8 && under != powers))) {
          ok = all_ok(!*failed);
          if (!ok) break;
          float keep = 1.f, down = 1.f;
          if (BITS == 8 && under != powers) {  // larger ones from this tile on
            f = fminf(fmaxf(f0 * exponent_factor(under & 255), 1.2e-38f), 3.e38f);
            down = powers ? power_below((int)(powers >> 8) - (int)(under >> 8)) : 0.f;
            powers = under;
            if (thr != -INFINITY) thr = score_limit(-neg, f);
          }
          if (top > -INFINITY) {
            const float before = thr == -INFINITY ? -INFINITY : -neg;
            const float m = fmaxf(before, top * f - kLift);
            keep = ex2_approx(before - m);
            neg = -m;
            thr = score_limit(m, f);
          }
          const uint64_t keep2 = tc::pack2(keep, keep);
          l2[0] = tc::fma2(l2[0], keep2, 0);
          l2[1] = tc::fma2(l2[1], keep2, 0);
          keep *= down;
          if (j > p.begin) {
            // the product of the tile before has to be in O
            if (!wait(&sm.o_full[blk], o_full.parity)) thr = -INFINITY;
            tc::tc_fence_after();
            waited = true;
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
              float o[32];
              uint32_t w[32];
              tc::tmem_ld32(to + i, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 32; ++q) w[q] = __float_as_uint(o[q] * keep);
              tc::tmem_st32(to + i, w);
            }
          }
        }
        const uint64_t f2 = tc::pack2(f, f), neg2 = tc::pack2(neg, neg);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int at = half * 32 + 2 * i;
            float p0, p1;
            tc::unpack2(tc::fma2(tc::pack2(s[at], s[at + 1]), f2, neg2), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            l2[i & 1] = tc::add2(l2[i & 1], tc::pack2(p0, p1));
            w[i] = tc::pack_f16(p0, p1);
          }
          if (half == 0 && j > p.begin) {  // the product before has read its weights
            if (!waited && !wait(&sm.o_full[blk], o_full.parity)) thr = -INFINITY;
            o_full.step();
            tc::tc_fence_after();
          }
          tc::tmem_st16u(tp + half * 16, w);
        }
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.p_full[blk]);
      }
      // ---- end of the piece ----
      ok = all_ok(ok && wait(&sm.o_full[blk], o_full.parity) && !*failed);
      if (!ok) break;
      o_full.step();
      tc::tc_fence_after();
      float l, la, lb;
      tc::unpack2(tc::add2(l2[0], l2[1]), la, lb);
      l = la + lb;
      const bool whole = p.begin == 0 && p.end == p.tiles;
      const float post =
          BITS == 4 ? exponent_scale(c.v_exp, p.h, 1) : exponent_factor((int)(powers >> 8));
      const float inv = !whole ? (BITS == 4 ? 1.f : post) : l == 0.f ? 0.f : post / l;
      const float m = thr == -INFINITY ? -INFINITY : -neg;
      const int64_t out_at = tok * a.num_heads + head;
      const int64_t part_at =
          (int64_t)(2 * blockIdx.x + (p.begin == 0 ? 1 : 0)) * kRows + blk * kBlock + row;
#pragma unroll 1
      for (int i = 0; i < D; i += 32) {
        float o[32];
        tc::tmem_ld32(to + i, o);
        tc::tmem_ld_wait();
        if (!live) continue;
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + out_at * D + i);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            dst[q] = make_uint4(tc::pack_bf16(o[8 * q] * inv, o[8 * q + 1] * inv),
                                tc::pack_bf16(o[8 * q + 2] * inv, o[8 * q + 3] * inv),
                                tc::pack_bf16(o[8 * q + 4] * inv, o[8 * q + 5] * inv),
                                tc::pack_bf16(o[8 * q + 6] * inv, o[8 * q + 7] * inv));
        } else {
          float4* dst = reinterpret_cast<float4*>(plan.o + part_at * D + i);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            dst[q] = BITS == 4 ? make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3])
                               : make_float4(o[4 * q] * inv, o[4 * q + 1] * inv,
                                             o[4 * q + 2] * inv, o[4 * q + 3] * inv);
        }
      }
      if (tid == 0 && p.begin == 0 && !whole)
        plan.open[blockIdx.x] = {p.q.bos, p.r * kRows, rows, p.h,
                                 (int)((x + (p.tiles - p.end) - 1) / per)};
      if (live) {
        if (!whole)
          plan.ml[part_at] = make_float2(m, l);
        else if (a.lse)
          a.lse[out_at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      tc::tc_fence_before();  // the reads of O come before the next piece's products
    }
  } else if (warp < 12) {
    // ----------------------------------------------------- dequantisation ----
    leave_registers<BITS, kDequantRegs>();
    const int dw = warp - 8;
    Ring<kRawStages> raw;
    Ring<kTileStages> st;
    uint32_t empty_parity = 1;  // a fresh barrier passes for the phase before
    uint32_t tile_no = 0;
    bool ok = true;
    for (unsigned long long x = x0; x < x1 && ok;) {
      Piece p;
      p.set(c, a, range, plan, entries, x, x1);
      x += p.end - p.begin;
      int k_top = 0, v_top = 0;  // 8 bits: the largest exponent bytes of the piece so far
      for (int j = p.begin; j < p.end; ++j, ++tile_no) {
        ok = wait(&sm.raw_full[raw.i], raw.parity);
        if constexpr (BITS == 8) {
          const uint8_t* const tile = sm.raw[raw.i];
          const uint32_t valid = sm.valid[tile_no % kValidRing];
          const int left = valid >> dw & 1 ? p.q.kv - j * kKeys - dw * kGroup : 0;
#pragma unroll
          for (int q = 0; q < kGroups; ++q) {
            const uint32_t x =
                *reinterpret_cast<const uint16_t*>(tile + q * L::kGroupBytes + L::kScales);
            if (valid >> q & 1) k_top = max(k_top, x & 255), v_top = max(v_top, x >> 8);
          }
          const uint8_t* const g = tile + dw * L::kGroupBytes;
          const uint32_t mine = *reinterpret_cast<const uint16_t*>(g + L::kScales);
          if (dw == 0 && lane == 0)
            *(volatile uint32_t*)&sm.powers[tile_no % kValidRing] = k_top | v_top << 8;
          Dequant8<D, false> k;
          k.load(g);
          ok &= wait(&sm.k_empty[st.i], empty_parity);
          k.store(sm.k[st.i], dw, half_power(max(0, k_top - (int)(mine & 255))), kGroup);
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.k_full[st.i]);
          Dequant8<D, true> v;
          v.load(g);
          ok &= wait(&sm.v_empty[st.i], empty_parity);
          v.store(sm.v[st.i], dw, half_power(max(0, v_top - (int)(mine >> 8))), left);
        } else {
          const int t8 = lane & 7, b4 = lane >> 3;
          const int kc = L::k_codes(t8, b4), vc = L::v_codes(t8, b4) - L::v_codes(0, 0);
          const int ks_at = L::k_scale(t8, b4), vs_at = L::v_scale(t8 & 6, b4);
          // bytes of the scale words that belong to tokens t8 and t8 + 8
          const uint32_t ks_pick = (ks_at & 3) | (((ks_at & 3) + L::kPer) << 4) | 0x4400;
          const uint32_t vs_pick = (t8 & 1) | (((t8 & 1) + 2) << 4) | 0x4400;
          const uint32_t row0 = (dw * kGroup + t8) * 128, chunk0 = ((b4 * 2) ^ t8) << 4;
          // Warp dw takes group dw of the tile; a lane the tokens t8 and t8 + 8 of it and block
          // b4 of every four.  The scales of both tokens lie in one word.
          const uint8_t* g = sm.raw[raw.i] + dw * L::kGroupBytes;
          const bool here = sm.valid[tile_no % kValidRing] >> dw & 1;
          const int left = here ? p.q.kv - j * kKeys - dw * kGroup : 0;  // tokens of the group
          auto put = [&](uint8_t* at, uint2 codes, uint32_t s2) {
            uint32_t lo[4], hi[4];
            e2m1x8_to_f16(codes.x, lo);
            e2m1x8_to_f16(codes.y, hi);
#pragma unroll
            for (int q = 0; q < 4; ++q) lo[q] = mul_f16x2(lo[q], s2), hi[q] = mul_f16x2(hi[q], s2);
            *reinterpret_cast<uint4*>(at + chunk0) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            *reinterpret_cast<uint4*>(at + (chunk0 ^ 16)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          };
          uint2 codes[2][D / 64];
          uint32_t scales[D / 64];
#pragma unroll
          for (int bb = 0; bb < D / 64; ++bb) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
              codes[half][bb] = *reinterpret_cast<const uint2*>(g + L::k_codes(half * 8, bb * 4) + kc);
            scales[bb] = *reinterpret_cast<const uint32_t*>(g + (ks_at & ~3) + bb * 8);
          }
          ok &= wait(&sm.k_empty[st.i], empty_parity);
#pragma unroll
          for (int bb = 0; bb < D / 64; ++bb) {
            const uint32_t h = e4m3x2_to_f16x2(__byte_perm(scales[bb], 0, ks_pick));
#pragma unroll
            for (int half = 0; half < 2; ++half)
              put(sm.k[st.i] + row0 + half * 1024 + bb * (kKeys * 128), codes[half][bb],
                  __byte_perm(h, 0, half ? 0x3232 : 0x1010));
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.k_full[st.i]);
#pragma unroll
          for (int bb = 0; bb < D / 64; ++bb) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
              codes[half][bb] = *reinterpret_cast<const uint2*>(g + L::v_codes(half * 8, bb * 4) + vc);
            scales[bb] = *reinterpret_cast<const uint32_t*>(g + vs_at + bb * 64);
          }
          ok &= wait(&sm.v_empty[st.i], empty_parity);
          // what lies past the request's length may be anything: its scale becomes 0
          const uint32_t keep = (t8 < left ? 0x00ffu : 0u) | (t8 + 8 < left ? 0xff00u : 0u);
#pragma unroll
          for (int bb = 0; bb < D / 64; ++bb) {
            const uint32_t h = e4m3x2_to_f16x2(__byte_perm(scales[bb], 0, vs_pick) & keep);
#pragma unroll
            for (int half = 0; half < 2; ++half)
              put(sm.v[st.i] + row0 + half * 1024 + bb * (kKeys * 128), codes[half][bb],
                  __byte_perm(h, 0, half ? 0x3232 : 0x1010));
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::mbar_arrive(&sm.v_full[st.i]);
          tc::mbar_arrive(&sm.raw_empty[raw.i]);
        }
        ok = all_ok(ok);
        if (!ok) break;
        raw.step();
        st.step();
        if (st.i == 0) empty_parity ^= 1;
      }
    }
  } else {
    leave_registers<BITS, kOtherRegs>();
    if (issues) {
      // ------------------------------------------------------ matrix products ----
      constexpr int kMine = 2 / kIssuers<BITS>;  // blocks
      if (tc::elect_one()) {  // (2048-token chunk over 32768 keys: 869 us; by lane == 0: 1392)
        const uint64_t kd = tc::make_sdesc(tc::smem_u32(sm.k), 0, 1024, tc::kSwizzle128);
        const uint64_t vd = tc::make_sdesc(tc::smem_u32(sm.v), kKeys * 128, 1024, tc::kSwizzle128);
        const uint64_t qd = tc::make_sdesc(tc::smem_u32(sm.q), 0, 1024, tc::kSwizzle128);
        const uint32_t id_s = tc::make_idesc_f16(128, kKeys, false, false);
        const uint32_t id_o = tc::make_idesc_f16(128, D, false, true);
        Ring<kTileStages> ks, vs;
        Ring<1> q_full[kMine], p_full[kMine];
        uint32_t free_parity[2] = {1, 1};
        bool ok = true;
        for (unsigned long long x = x0; x < x1 && ok;) {
          Piece p;
          p.set(c, a, range, plan, entries, x, x1);
          x += p.end - p.begin;
          const int blocks = min((p.rows() > kBlock ? 2 : 1) - first_blk, kMine);  // of this warp
          const int n = p.end - p.begin;
          // scores of the next tile, as soon as the softmax has the tile before in registers
          auto scores = [&]() {
            ok = wait(&sm.k_full[ks.i], ks.parity);
            const uint64_t b0 = kd + (uint64_t)(ks.i * S::kTile >> 4);
            for (int i = 0; i < blocks && ok; ++i) {
              const int blk = first_blk + i;
              ok = wait(&sm.s_free[blk], free_parity[i]);
              if (!ok) break;
              free_parity[i] ^= 1;
              tc::tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t b1 =
                    b0 + (uint64_t)(((kk >> 2) * (kKeys * 128) + (kk & 3) * 32) >> 4);
                if (QS && blk == 1)
                  tc::mma_bf16_ss(tmem + TS + kKeys,
                                  qd + (uint64_t)(((kk >> 2) * (kBlock * 128) + (kk & 3) * 32) >> 4),
                                  b1, id_s, kk > 0);
                else
                  tc::mma_ts(tmem + TS + blk * kKeys, tmem + TQ + blk * (D / 2) + kk * 8, b1, id_s,
                             kk > 0);
              }
              tc::mma_commit(&sm.s_full[blk]);
            }
            tc::mma_commit(&sm.k_empty[ks.i]);
            ks.step();
          };
          for (int i = 0; i < blocks && ok; ++i) {
            ok = wait(&sm.q_full[first_blk + i], q_full[i].parity);
            q_full[i].step();
          }
          if (ok) scores();
          for (int j = 0; j < n && ok; ++j) {
            if (j + 1 < n) scores();
            if (ok) ok = wait(&sm.v_full[vs.i], vs.parity);
            const uint64_t b0 = vd + (uint64_t)(vs.i * S::kTile >> 4);
            for (int i = 0; i < blocks && ok; ++i) {
              const int blk = first_blk + i;
              ok = wait(&sm.p_full[blk], p_full[i].parity);
              if (!ok) break;
              p_full[i].step();
              tc::tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                tc::mma_ts(tmem + TO + blk * D, tmem + TP + blk * (kKeys / 2) + kk * 8,
                           b0 + (uint64_t)(kk * 2048 >> 4), id_o, j > 0 || kk > 0);
              tc::mma_commit(&sm.o_full[blk]);
            }
            tc::mma_commit(&sm.v_empty[vs.i]);
            vs.step();
          }
        }
      }
      __syncwarp();
    } else if (warp == 13) {
      // ---------------------------------------------------------------- pages ----
      const int GP = c.page_size / kGroup;
      Ring<kRawStages> raw;
      uint32_t empty_parity = 1, tile_no = 0;
      bool ok = true;
      for (unsigned long long x = x0; x < x1 && ok;) {
        Piece p;
        p.set(c, a, range, plan, entries, x, x1);
        x += p.end - p.begin;
        const uint8_t* src = nullptr;
        uint32_t present = 0;  // of the 32 groups from 32 n on, for the n being loaded
        for (int j = p.begin; j < p.end; ++j, ++tile_no) {
          const int first = j * kGroups & 31;
          if (first == 0 || j == p.begin) {
            const int gi = (j * kGroups & ~31) + lane;
            const bool in = gi < (p.q.kv + kGroup - 1) / kGroup;
            const int page =
                in ? __ldg(a.block_table + (int64_t)p.b * a.max_blocks + gi / GP) : 0;
            const bool sound = page >= 0 && page < c.num_pages;
            if (in && !sound) report_error(a.err, kErrDeviceCheck);
            src = c.pages + (((int64_t)page * c.kv_heads + p.h) * GP + gi % GP) * L::kGroupBytes;
            present = __ballot_sync(0xffffffffu, in && sound);
          }
          ok = all_ok(wait(&sm.raw_empty[raw.i], empty_parity));
          if (!ok) break;
          if ((lane ^ first) < kGroups) {
            const int u = lane ^ first;
            if (u == 0)
              *(volatile uint32_t*)&sm.valid[tile_no % kValidRing] =
                  present >> first & ((1u << kGroups) - 1);
            if (present >> lane & 1) {
              tc::mbar_arrive_expect_tx(&sm.raw_full[raw.i], L::kGroupBytes);
              tc::bulk_load(sm.raw[raw.i] + u * L::kGroupBytes, src, L::kGroupBytes,
                            &sm.raw_full[raw.i]);
            } else {
              tc::mbar_arrive(&sm.raw_full[raw.i]);
            }
          }
          __syncwarp();
          raw.step();
          if (raw.i == 0) empty_parity ^= 1;
        }
      }
      if (lane == 0) sm.copied = tile_no;
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  // After a wait gave up, what is under way ends before its memory goes away: the products (of
  // the thread that elect.sync elects each time) and the copies of the last tiles.
  if (*failed && issues && tc::elect_one()) {
    tc::mma_commit(&sm.issued);
    wait_phase(&sm.issued, 0, a.wait_cycles, nullptr);
  }
  if (*failed && warp == 13) {
    if (lane < a.withheld) tc::mbar_arrive(&sm.raw_full[0]);
    const uint32_t n = sm.copied;
    for (uint32_t i = n - min(n, (uint32_t)kRawStages); i < n; ++i)
      wait_phase(&sm.raw_full[i % kRawStages], i / kRawStages & 1, a.wait_cycles, nullptr);
  }
  __syncwarp();
  if (warp == 12) tc::tmem_dealloc(tmem, kCols);
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Entries that well-formed offsets can ask for: a unit of rows each, one more per request.
int64_t max_entries(const View& c, const AttentionArgs& a) {
  const int64_t rows = (int64_t)a.total_tokens * (a.num_heads / c.kv_heads);
  return std::min<int64_t>(rows / kRows + a.num_seqs, INT32_MAX - 1);
}

template <int D>
size_t layout(const View& c, const AttentionArgs& a, uint8_t* ws, Plan* plan) {
  const size_t n = (size_t)max_entries(c, a), slots = 2 * (size_t)sm_count();
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* p = ws + at;
    at += up256(bytes);
    return p;
  };
  Plan p;
  p.tiles = reinterpret_cast<unsigned long long*>(take((n + 1) * 8));
  p.entry = reinterpret_cast<int2*>(take((n + 1) * 8));
  p.first = reinterpret_cast<int*>(take(((size_t)a.num_seqs + 1) * 4));
  p.open = reinterpret_cast<OpenUnit*>(take(slots / 2 * sizeof(OpenUnit)));
  p.o = reinterpret_cast<float*>(take(slots * kRows * D * 4));
  p.ml = reinterpret_cast<float2*>(take(slots * kRows * 8));
  if (plan) *plan = p;
  return at;
}

template <int BITS, int D>
cudaError_t run(const View& c, const AttentionArgs& a, const RowRange& range, cudaStream_t st) {
  static PerDeviceInit init;
  constexpr int kSmem = (int)sizeof(Smem<BITS, D>) + 1024;
  static_assert(kSmem <= 227 * 1024, "more shared memory than a CTA has");
  cudaError_t e = init.run([&] {
    if (BITS == 8) {  // the launch bounds are an upper limit only
      cudaFuncAttributes f;
      const cudaError_t err = cudaFuncGetAttributes(&f, chunk_kernel<BITS, D>);
      if (err != cudaSuccess) return err;
      if (!registers_suffice(f.numRegs)) return cudaErrorLaunchOutOfResources;
    }
    return cudaFuncSetAttribute(chunk_kernel<BITS, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmem);
  });
  if (e != cudaSuccess) return e;
  Plan plan;
  layout<D>(c, a, static_cast<uint8_t*>(a.workspace), &plan);
  const int ctas = sm_count();
  const int q_vec = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.q_token_stride % 8 == 0 &&
                    a.q_head_stride % 8 == 0;
  plan_kernel<<<1, 1024, 0, st>>>(c, a, range, plan, (int)max_entries(c, a));
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  chunk_kernel<BITS, D><<<ctas, kThreads<BITS>, kSmem, st>>>(c, a, range, plan, q_vec);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_join<__nv_bfloat16, D, 4, 1>(c, a, plan.open, plan.o, plan.ml, 0, kRows, ctas, st);
}

}  // namespace

size_t cache_chunk_workspace_bytes(const View& c, const AttentionArgs& a) {
  return a.head_dim == 128 ? layout<128>(c, a, nullptr, nullptr)
                           : layout<64>(c, a, nullptr, nullptr);
}

cudaError_t launch_cache_chunk(int bits, const View& c, const AttentionArgs& a,
                               const RowRange& range, cudaStream_t st) {
  if (bits == 8) return a.head_dim == 128 ? run<8, 128>(c, a, range, st) : run<8, 64>(c, a, range, st);
  return a.head_dim == 128 ? run<4, 128>(c, a, range, st) : run<4, 64>(c, a, range, st);
}

}  // namespace kda
