// kda_cache_attention.cu -- kda_cache_attention for few rows per kv head (decode
// steps, drafted windows): causal attention over the 4-bit paged cache.
//
// Mathematics.  A unit is a request, a kv head and up to 8 NT of the rows (new
// token x query head) that share it.  Its keys are walked in tiles of 32 with the
// usual running maximum m and sum l of a softmax,
//     p_j = 2^(s_j - m),  l = sum p_j,  o = sum p_j v_j,   s = scale log2(e) q . k,
// partial (m, l, o) of parts of a unit's keys being joined by rescaling to the
// common maximum.  m is moved (and o, l rescaled) only when some score passes it
// by more than 8, so p <= 2^8: any reference gives the same quotient o / l.
//
// Products.  mma.sync m16n8k16 on halves with the cache as the 16-row operand:
// scores^T = K q^T (16 keys x 8 rows), o^T += V^T p^T (16 channels x 8 rows).
// The call is bound by HBM -- 9/8 byte a key channel pair for 4 G flops of a group
// of G query heads -- so what counts is the issue slots it takes to turn the codes
// into operands.  A lane's A fragment of K^T or V takes its codes straight from
// the bytes of a group (the layout in include/kda.h is the fragments' order), a
// conversion instruction makes two halves of each byte, and one half2 product
// applies the E4M3 scale: code x scale has 6 significant bits, exact in a half.
// q is scaled to [1/2, 1] by a power of two per row and rounded to halves: bf16
// fits exactly, fp32 goes in as two halves.  p is rounded to a half (2^-11, below
// the output's own 2^-8), for fp32 outputs to two.  All sums are fp32.
//
// Work split.  The tiles of all units in one sequence are cut evenly over the
// warps of the whole GPU, wherever that falls in a unit: lengths of any mix fill
// the machine, one long request included.  A warp streams its tiles through its
// own ring of bulk copies (no CTA-wide synchronisation while it runs).  Parts of a
// unit are joined inside their CTA through the workspace, and across CTAs by a
// second kernel.
#include <math.h>

#include <algorithm>

#include "kda_cache.cuh"
#include "kda_launch.h"
#include "tc_ptx.cuh"

namespace kda {
namespace {

using namespace cache;

constexpr int kTileGroups = 2;                   // groups of 16 keys in a tile
constexpr int kTileKeys = kTileGroups * kGroup;  // 32
constexpr int kMaxSeqs = 2048;                   // requests of one launch (their plan is in smem)
constexpr float kSlack = 8.f;                    // log2 head room of p over the reference m
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What a launch leaves in the workspace.
struct Parts {
  unsigned long long* plan;  // [nseq + 1] tiles before each request, then tiles per warp
  float* o;                  // [slots][rows][D]
  float2* ml;                // [slots][rows]
};

// Slots: two per warp (part that starts inside its unit, part that starts it but
// does not end it), then two per CTA.
struct Shape {
  int ctas, warps;  // warps per CTA
  __host__ __device__ int warp_slots() const { return 2 * ctas * warps; }
  __host__ __device__ int slots() const { return warp_slots() + 2 * ctas; }
};

// A request of the launch, as the split sees it.
struct Request {
  int kv, n, bos;
  int tiles;   // of one unit
  int64_t rt;  // row tiles
};

__device__ __forceinline__ bool load_request(const View& c, const AttentionArgs& a, int b,
                                             int rows_per_tile, bool report, Request& r) {
  const int group = a.num_heads / c.kv_heads;
  int eos;
  // a decreasing offset takes both of its neighbours out: their tokens may overlap others'
  const bool ok = seq_range(a.cu_new, b, a.total_tokens, report ? a.err : nullptr, r.bos, eos) &&
                  (b == 0 || __ldg(a.cu_new + b - 1) <= r.bos);
  r.kv = __ldg(a.kv_lens + b);
  if (!ok || r.kv < 0 || r.kv > (int64_t)a.max_blocks * c.page_size) {
    if (report) report_error(a.err, kErrDeviceCheck);
    r.n = 0;
    r.rt = 0;
    r.tiles = 1;
    return false;
  }
  r.n = eos - r.bos;
  r.rt = ((int64_t)r.n * group + rows_per_tile - 1) / rows_per_tile;
  r.tiles = max(1, (r.kv + kTileKeys - 1) / kTileKeys);  // a unit without keys still writes zeros
  return r.rt > 0;
}

// The last index i with plan[i] <= x.
template <typename P>
__device__ __forceinline__ int find_request(const P* plan, int n, unsigned long long x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (plan[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// A place in the sequence of all tiles.
struct Cursor {
  int b;  // request (relative to the launch)
  int h;  // kv head
  int r;  // row tile
  int tile;
  Request q;

  __device__ __forceinline__ void seek(const View& c, const AttentionArgs& a, int seq0, int nseq,
                                       int rows_per_tile, const unsigned long long* plan,
                                       unsigned long long x) {
    b = find_request(plan, nseq, x);
    load_request(c, a, seq0 + b, rows_per_tile, false, q);
    const unsigned long long off = x - plan[b];
    const unsigned long long u = off / q.tiles;
    tile = (int)(off - u * q.tiles);
    h = (int)(u / q.rt);
    r = (int)(u - (unsigned long long)h * q.rt);
  }
  // The next tile; returns true when it starts a new unit.  Not past the last one.
  __device__ __forceinline__ bool next(const View& c, const AttentionArgs& a, int seq0, int nseq,
                                       int rows_per_tile) {
    if (++tile < q.tiles) return false;
    tile = 0;
    if (++r < q.rt) return true;
    r = 0;
    if (++h < c.kv_heads) return true;
    h = 0;
    while (++b < nseq && !load_request(c, a, seq0 + b, rows_per_tile, false, q)) {
    }
    return true;
  }
};

// (m, l, o) of rows 2t, 2t+1 of each row tile's n8 block, written by the lanes that hold them.
template <typename T, int D>
__device__ __forceinline__ void store_row(T* p, const float (&x)[D / 8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      *reinterpret_cast<float4*>(p + 4 * i) =
          make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
      *reinterpret_cast<uint4*>(p + 8 * i) =
          make_uint4(tc::pack_bf16(x[8 * i], x[8 * i + 1]), tc::pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                     tc::pack_bf16(x[8 * i + 4], x[8 * i + 5]),
                     tc::pack_bf16(x[8 * i + 6], x[8 * i + 7]));
  }
}

template <typename T>
constexpr int kTerms = sizeof(T) == 4 ? 2 : 1;  // halves of a query or weight

template <typename T, int D, int NT, int WARPS, int STAGES>
struct Smem {
  static constexpr int kStage = kTileGroups * Layout<D>::kGroupBytes;
  alignas(128) uint8_t ring[WARPS][STAGES][kStage];
  unsigned long long plan[kMaxSeqs + 1];
  uint64_t full[WARPS][STAGES];
  uint32_t valid[WARPS][STAGES];
  unsigned long long sums[WARPS];
};

template <typename T, int D, int NT, int WARPS, int STAGES, int CTAS>
__global__ void __launch_bounds__(WARPS * 32, CTAS)
    split_kernel(View c, AttentionArgs a, int seq0, int nseq, Parts parts, int q_vec) {
  using L = Layout<D>;
  using S = Smem<T, D, NT, WARPS, STAGES>;
  constexpr int ROWS = 8 * NT;
  constexpr int TERMS = kTerms<T>;
  constexpr int QC = D / 4;       // channels of a query row per lane
  constexpr int KM = D / 16;      // products along the channels of K, and 16-channel tiles of V
  constexpr int VC = D / 8;       // channels of V per lane
  extern __shared__ uint8_t raw[];
  S& sm = *reinterpret_cast<S*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int group = a.num_heads / c.kv_heads;
  const int GP = c.page_size / kGroup;

  // ---- the plan: tiles before each request ----
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s) tc::mbar_init(&sm.full[warp][s], 1);
    tc::mbar_fence_init();
  }
  {
    constexpr int N = WARPS * 32;
    const int per = (nseq + N - 1) / N;
    const int b0 = tid * per;
    unsigned long long mine = 0;
    for (int i = 0; i < per; ++i) {
      const int b = b0 + i;
      if (b >= nseq) break;
      Request r;
      const bool live = load_request(c, a, seq0 + b, ROWS, blockIdx.x == 0, r);
      sm.plan[b] = mine;
      if (live) mine += (unsigned long long)r.rt * r.tiles * c.kv_heads;
    }
    unsigned long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sm.sums[warp] = incl;
    __syncthreads();
    unsigned long long before = incl - mine;
    for (int w = 0; w < warp; ++w) before += sm.sums[w];
    for (int i = 0; i < per; ++i)
      if (b0 + i < nseq) sm.plan[b0 + i] += before;
    if (tid == N - 1) sm.plan[nseq] = before + mine;
    __syncthreads();
  }
  const unsigned long long total = sm.plan[nseq];
  const unsigned long long workers = (unsigned long long)gridDim.x * WARPS;
  const unsigned long long per = (total + workers - 1) / workers;
  if (blockIdx.x == 0) {
    for (int i = tid; i <= nseq; i += WARPS * 32) parts.plan[i] = sm.plan[i];
    if (tid == 0) parts.plan[nseq + 1] = per;
  }
  const int worker = blockIdx.x * WARPS + warp;
  const unsigned long long x0 = min(per * worker, total), x1 = min(x0 + per, total);
  const Shape shape{(int)gridDim.x, WARPS};

  if (x0 < x1) {
    Cursor ld, cp;
    cp.seek(c, a, seq0, nseq, ROWS, sm.plan, x0);
    ld = cp;
    const int count = (int)min(x1 - x0, (unsigned long long)INT32_MAX);
    int issued = 0;
    int pages = -1, pages_of = -1;  // lane l: page of group 32 pages_of + l of ld's request
    int pages_b = -1;

    auto issue = [&](int stage) {
      const int g0 = ld.tile * kTileGroups;
      if (pages_b != ld.b || pages_of != (g0 >> 5)) {
        pages_b = ld.b;
        pages_of = g0 >> 5;
        const int gi = pages_of * 32 + lane;
        pages = gi * (int64_t)kGroup < ld.q.kv
                    ? __ldg(a.block_table + (int64_t)(seq0 + ld.b) * a.max_blocks + gi / GP)
                    : 0;
        if (pages < 0 || pages >= c.num_pages) {
          report_error(a.err, kErrDeviceCheck);
          pages = -1;
        }
      }
      const int p0 = __shfl_sync(0xffffffffu, pages, g0 & 31);
      const int p1 = __shfl_sync(0xffffffffu, pages, (g0 + 1) & 31);
      if (lane == 0) {
        const bool v0 = p0 >= 0 && g0 * kGroup < ld.q.kv;
        const bool v1 = p1 >= 0 && (g0 + 1) * kGroup < ld.q.kv;
        uint64_t* bar = &sm.full[warp][stage];
        uint8_t* dst = sm.ring[warp][stage];
        sm.valid[warp][stage] = (v0 ? 1u : 0u) | (v1 ? 2u : 0u);
        const int i0 = g0 % GP;
        const uint8_t* s0 =
            c.pages + (((int64_t)p0 * c.kv_heads + ld.h) * GP + i0) * L::kGroupBytes;
        if (v0 && v1 && i0 + 1 < GP) {
          tc::mbar_arrive_expect_tx(bar, 2 * L::kGroupBytes);
          tc::bulk_load(dst, s0, 2 * L::kGroupBytes, bar);
        } else if (v0 || v1) {
          tc::mbar_arrive_expect_tx(bar, (v0 && v1 ? 2 : 1) * L::kGroupBytes);
          if (v0) tc::bulk_load(dst, s0, L::kGroupBytes, bar);
          if (v1)
            tc::bulk_load(dst + L::kGroupBytes,
                          c.pages + (((int64_t)p1 * c.kv_heads + ld.h) * GP + (g0 + 1) % GP) *
                                        L::kGroupBytes,
                          L::kGroupBytes, bar);
        } else {
          tc::mbar_arrive(bar);
        }
      }
      ++issued;
      if (issued < count) ld.next(c, a, seq0, nseq, ROWS);
    };

    for (int s = 0; s < STAGES && s < count; ++s) issue(s);

    uint32_t qf[NT][KM][TERMS][2];
    float o[KM][NT][4];
    float m[NT][2], l[NT][2], sf[NT][2];
    int see[NT][2];  // keys that the lane's rows see
    int all_see = 0;  // keys that every row of the unit sees
    int seg_tile = 0;

    auto start_unit = [&]() {
      const int rows = (int)min((int64_t)cp.q.n * group - (int64_t)cp.r * ROWS, (int64_t)ROWS);
      const int64_t row0 = (int64_t)cp.r * ROWS;
      all_see = cp.q.kv - cp.q.n + (int)(row0 / group) + 1;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int64_t row = row0 + n * 8 + g;
        float x[QC], top = 0.f;
        if (n * 8 + g < rows) {
          const int64_t tok = cp.q.bos + row / group;
          const T* p = static_cast<const T*>(a.q) + tok * a.q_token_stride +
                       (cp.h * group + (int)(row % group)) * a.q_head_stride + t * QC;
          if (q_vec) {
#pragma unroll
            for (int i = 0; i < QC * (int)sizeof(T) / 16; ++i) {
              const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) {
                  x[4 * i + j] = __uint_as_float(w[j]);
                } else {
                  x[8 * i + 2 * j] = tc::bf16_lo(w[j]);
                  x[8 * i + 2 * j + 1] = tc::bf16_hi(w[j]);
                }
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < QC; ++i) x[i] = IO<T>::ld(p + i);
          }
        } else {
#pragma unroll
          for (int i = 0; i < QC; ++i) x[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < QC; ++i) top = fmaxf(top, fabsf(x[i]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e with top 2^-e in [1, 2); e held to the normal range, 0 where top is not finite
        int e = ((__float_as_int(top) >> 23) & 255) - 127;
        e = e == 128 ? 0 : max(-126, min(e, 126));
        const float down = __int_as_float((127 - e) << 23);
        const float up = __int_as_float((127 + e) << 23);
        const float f = a.scale * kLog2e * exponent_scale(c.k_exp, cp.h, 1) * up;
        sf[n][0] = __shfl_sync(0xffffffffu, f, t * 8);
        sf[n][1] = __shfl_sync(0xffffffffu, f, t * 8 + 4);
#pragma unroll
        for (int i = 0; i < QC / 2; ++i) {
          const float y0 = x[2 * i] * down, y1 = x[2 * i + 1] * down;
          const uint32_t hi = tc::pack_f16(y0, y1);
          qf[n][i / 2][0][i % 2] = hi;
          if constexpr (TERMS == 2) {
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            qf[n][i / 2][1][i % 2] = tc::pack_f16(y0 - b.x, y1 - b.y);
          }
        }
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          m[n][e2] = -INFINITY;
          l[n][e2] = 0.f;
          const int64_t rr = row0 + n * 8 + 2 * t + e2;
          see[n][e2] = n * 8 + 2 * t + e2 < rows
                           ? cp.q.kv - cp.q.n + (int)(rr / group) + 1
                           : 0;
        }
      }
#pragma unroll
      for (int i = 0; i < KM; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][n][j] = 0.f;
      seg_tile = cp.tile;
    };

    // Ends the part of the unit that this warp had; `last` tile of the unit or not.
    auto end_part = [&](bool ends_unit) {
      const bool whole = ends_unit && seg_tile == 0;
      const int64_t row0 = (int64_t)cp.r * ROWS;
      const int rows = (int)min((int64_t)cp.q.n * group - row0, (int64_t)ROWS);
      const int slot = 2 * worker + (seg_tile == 0 ? 1 : 0);
      const float post = exponent_scale(c.v_exp, cp.h, 1);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[n][e];
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
          const int row = n * 8 + 2 * t + e;
          float x[VC];
          if (row < rows) {
            if (whole) {
              const float inv = sum == 0.f ? 0.f : post / sum;
#pragma unroll
              for (int i = 0; i < KM; ++i) {
                x[2 * i] = o[i][n][e] * inv;
                x[2 * i + 1] = o[i][n][2 + e] * inv;
              }
              const int64_t rr = row0 + row;
              const int64_t at =
                  (cp.q.bos + rr / group) * a.num_heads + cp.h * group + rr % group;
              store_row<T, D>(static_cast<T*>(a.out) + at * D + g * VC, x);
              if (a.lse && g == 0)
                a.lse[at] = sum == 0.f ? -INFINITY : (m[n][e] + log2f(sum)) * kLn2;
            } else {
#pragma unroll
              for (int i = 0; i < KM; ++i) {
                x[2 * i] = o[i][n][e];
                x[2 * i + 1] = o[i][n][2 + e];
              }
              const int64_t at = (int64_t)slot * ROWS + row;
              store_row<float, D>(parts.o + at * D + g * VC, x);
              if (g == 0) parts.ml[at] = make_float2(m[n][e], sum);
            }
          }
        }
    };

    start_unit();
    bool alive = true;
    for (int i = 0; i < count && alive; ++i) {
      const int stage = i % STAGES;
      if (!tc::mbar_wait(&sm.full[warp][stage], (i / STAGES) & 1, kWaitLimit)) {
        if (lane == 0) report_error(a.err, kErrTimeout);
        alive = false;
        break;
      }
      const uint32_t valid = sm.valid[warp][stage];
      const int key0 = cp.tile * kTileKeys;
      float s[kTileGroups][NT][4];
      // ---- scores ----
#pragma unroll
      for (int u = 0; u < kTileGroups; ++u) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[u][n][j] = 0.f;
        if (!(valid >> u & 1)) continue;
        const uint8_t* base = sm.ring[warp][stage] + u * L::kGroupBytes;
        uint32_t ka[D / 32], kb[D / 32];  // codes of keys g and g + 8
        uint32_t sc[2][L::kPer];          // their scales, twice in a word
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(base + g * 64 + t * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(base + (g + 8) * 64 + t * 16);
          ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
          kb[0] = y.x, kb[1] = y.y, kb[2] = y.z, kb[3] = y.w;
          const uint32_t w =
              *reinterpret_cast<const uint32_t*>(base + L::kKScales + g * 16 + t * 4);
          const uint32_t wa = e4m3x2_to_f16x2(w), wb = e4m3x2_to_f16x2(w >> 16);
          sc[0][0] = __byte_perm(wa, 0, 0x1010), sc[0][1] = __byte_perm(wa, 0, 0x3232);
          sc[1][0] = __byte_perm(wb, 0, 0x1010), sc[1][1] = __byte_perm(wb, 0, 0x3232);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(base + g * 32 + t * 8);
          const uint2 y = *reinterpret_cast<const uint2*>(base + (g + 8) * 32 + t * 8);
          ka[0] = x.x, ka[1] = x.y;
          kb[0] = y.x, kb[1] = y.y;
          const uint32_t w = e4m3x2_to_f16x2(
              *reinterpret_cast<const uint16_t*>(base + L::kKScales + g * 8 + t * 2));
          sc[0][0] = __byte_perm(w, 0, 0x1010);
          sc[1][0] = __byte_perm(w, 0, 0x3232);
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t xa[4], xb[4];
          e2m1x8_to_f16(ka[w], xa);
          e2m1x8_to_f16(kb[w], xb);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            xa[j] = mul_f16x2(xa[j], sc[0][w / 2]);
            xb[j] = mul_f16x2(xb[j], sc[1][w / 2]);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t af[4] = {xa[2 * j], xb[2 * j], xa[2 * j + 1], xb[2 * j + 1]};
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < TERMS; ++e)
                tc::mma_16816_f16(s[u][n], af, qf[n][2 * w + j][e][0], qf[n][2 * w + j][e][1]);
          }
        }
      }
      // ---- softmax ----
      bool move = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < kTileGroups; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[u][n][j] *= sf[n][j & 1];
            if (key0 + kTileKeys > all_see || valid != 3u) {
              const int key = key0 + u * kGroup + g + 8 * (j >> 1);
              if (key >= see[n][j & 1] || !(valid >> u & 1)) s[u][n][j] = -INFINITY;
            }
            move |= s[u][n][j] > m[n][j & 1] + kSlack;
          }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = m[n][e];
#pragma unroll
            for (int u = 0; u < kTileGroups; ++u)
              top = fmaxf(top, fmaxf(s[u][n][e], s[u][n][2 + e]));
#pragma unroll
            for (int x = 4; x < 32; x <<= 1)
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float keep = top == -INFINITY ? 1.f : ex2_approx(m[n][e] - top);
            m[n][e] = top;
            l[n][e] *= keep;
#pragma unroll
            for (int i2 = 0; i2 < KM; ++i2) {
              o[i2][n][e] *= keep;
              o[i2][n][2 + e] *= keep;
            }
          }
      }
      uint32_t pf[kTileGroups][NT][TERMS][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float ref[2] = {m[n][0] == -INFINITY ? 0.f : m[n][0],
                              m[n][1] == -INFINITY ? 0.f : m[n][1]};
#pragma unroll
        for (int u = 0; u < kTileGroups; ++u) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[u][n][j] = ex2_approx(s[u][n][j] - ref[j & 1]);
            l[n][j & 1] += s[u][n][j];
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t hi = tc::pack_f16(s[u][n][2 * j], s[u][n][2 * j + 1]);
            pf[u][n][0][j] = tc::movmatrix_trans(hi);
            if constexpr (TERMS == 2) {
              const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              pf[u][n][1][j] =
                  tc::movmatrix_trans(tc::pack_f16(s[u][n][2 * j] - b.x, s[u][n][2 * j + 1] - b.y));
            }
          }
        }
      }
      // ---- values ----
#pragma unroll
      for (int u = 0; u < kTileGroups; ++u) {
        if (!(valid >> u & 1)) continue;
        const uint8_t* base = sm.ring[warp][stage] + u * L::kGroupBytes;
        const int blk = D == 128 ? g : g >> 1;
        uint32_t w = *reinterpret_cast<const uint32_t*>(base + L::kVScales + blk * 16 + t * 4);
        const int left = cp.q.kv - key0 - u * kGroup;
        if (left < kGroup) {  // bytes past the request's length: scale 0
          if (2 * t >= left) w &= 0xffffff00u;
          if (2 * t + 1 >= left) w &= 0xffff00ffu;
          if (2 * t + 8 >= left) w &= 0xff00ffffu;
          if (2 * t + 9 >= left) w &= 0x00ffffffu;
        }
        const uint32_t s0 = e4m3x2_to_f16x2(w), s1 = e4m3x2_to_f16x2(w >> 16);
        uint32_t c0[2][D / 64], c1[2][D / 64];  // [token][word] of tokens 2t.., 2t+8..
        const uint8_t* vb = base + L::kVCodes;
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(vb + g * 64 + t * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(vb + 4 * D + g * 64 + t * 16);
          c0[0][0] = x.x, c0[0][1] = x.y, c0[1][0] = x.z, c0[1][1] = x.w;
          c1[0][0] = y.x, c1[0][1] = y.y, c1[1][0] = y.z, c1[1][1] = y.w;
        } else {
          const uint8_t* p = vb + blk * 64 + t * 16 + (g & 1) * 4;
          c0[0][0] = *reinterpret_cast<const uint32_t*>(p);
          c0[1][0] = *reinterpret_cast<const uint32_t*>(p + 8);
          c1[0][0] = *reinterpret_cast<const uint32_t*>(p + 4 * D);
          c1[1][0] = *reinterpret_cast<const uint32_t*>(p + 4 * D + 8);
        }
#pragma unroll
        for (int wd = 0; wd < D / 64; ++wd) {
          // bytes of (even channel of the first token, of the second), then the odd channels
          uint32_t e0[4], d0[4], e1[4], d1[4];
          e2m1x8_to_f16((c0[0][wd] & 0x0f0f0f0fu) | ((c0[1][wd] << 4) & 0xf0f0f0f0u), e0);
          e2m1x8_to_f16(((c0[0][wd] >> 4) & 0x0f0f0f0fu) | (c0[1][wd] & 0xf0f0f0f0u), d0);
          e2m1x8_to_f16((c1[0][wd] & 0x0f0f0f0fu) | ((c1[1][wd] << 4) & 0xf0f0f0f0u), e1);
          e2m1x8_to_f16(((c1[0][wd] >> 4) & 0x0f0f0f0fu) | (c1[1][wd] & 0xf0f0f0f0u), d1);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t af[4] = {mul_f16x2(e0[j], s0), mul_f16x2(d0[j], s0),
                                    mul_f16x2(e1[j], s1), mul_f16x2(d1[j], s1)};
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < TERMS; ++e)
                tc::mma_16816_f16(o[wd * 4 + j][n], af, pf[u][n][e][0], pf[u][n][e][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (issued < count) issue(stage);
      const bool ends_unit = cp.tile + 1 == cp.q.tiles;
      if (ends_unit || i + 1 == count) {
        end_part(ends_unit);
        if (i + 1 < count) {
          cp.next(c, a, seq0, nseq, ROWS);
          start_unit();
        }
      } else {
        ++cp.tile;
      }
    }
  }

  // ---- join the parts of units that several warps of this CTA had ----
  __syncthreads();
  const unsigned long long c0 = min(per * WARPS * blockIdx.x, total),
                           c1 = min(c0 + per * WARPS, total);
  // Warp w takes the unit that its own tail starts; warp 0 also the one that enters the CTA.
  for (int job = warp == 0 ? 0 : 1; job < 2; ++job) {
    const unsigned long long w0 = min(c0 + per * warp, total), w1 = min(w0 + per, total);
    if (w0 >= w1) break;
    Cursor cu;
    unsigned long long u0, u1;
    cu.seek(c, a, seq0, nseq, ROWS, sm.plan, job == 0 ? w0 : w1 - 1);
    u0 = (job == 0 ? w0 : w1 - 1) - cu.tile;
    u1 = u0 + cu.q.tiles;
    if (job == 0 ? u0 == w0 : (u0 < w0 || u1 <= w1)) continue;  // no such unit
    const bool starts = u0 >= c0, ends = u1 <= c1;
    const unsigned long long p0 = max(u0, c0), p1 = min(u1, c1);
    const int first = (int)((p0 - c0) / per), last = (int)((p1 - 1 - c0) / per);
    const int64_t row0 = (int64_t)cu.r * ROWS;
    const int rows = (int)min((int64_t)cu.q.n * group - row0, (int64_t)ROWS);
    const float post = exponent_scale(c.v_exp, cu.h, 1);
    for (int row = 0; row < rows; ++row) {
      float top = -INFINITY;
      for (int w = first; w <= last; ++w) {
        const int slot = 2 * (blockIdx.x * WARPS + w) + (w == first && starts ? 1 : 0);
        top = fmaxf(top, parts.ml[(int64_t)slot * ROWS + row].x);
      }
      float sum = 0.f, x[D / 32] = {};
      for (int w = first; w <= last; ++w) {
        const int slot = 2 * (blockIdx.x * WARPS + w) + (w == first && starts ? 1 : 0);
        const int64_t at = (int64_t)slot * ROWS + row;
        const float2 ml = parts.ml[at];
        const float k = top == -INFINITY ? 1.f : ex2_approx(ml.x - top);
        sum = fmaf(ml.y, k, sum);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) x[i] = fmaf(parts.o[at * D + i * 32 + lane], k, x[i]);
      }
      if (starts && ends) {
        const float inv = sum == 0.f ? 0.f : post / sum;
        const int64_t rr = row0 + row;
        const int64_t at = (cu.q.bos + rr / group) * a.num_heads + cu.h * group + rr % group;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          IO<T>::st(static_cast<T*>(a.out) + at * D + i * 32 + lane, x[i] * inv);
        if (a.lse && lane == 0)
          a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
      } else {
        const int slot = shape.warp_slots() + 2 * blockIdx.x + (starts ? 1 : 0);
        const int64_t at = (int64_t)slot * ROWS + row;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) parts.o[at * D + i * 32 + lane] = x[i];
        if (lane == 0) parts.ml[at] = make_float2(top, sum);
      }
    }
  }
}

// Joins the parts of units that several CTAs had: one warp per row.
template <typename T, int D, int ROWS, int WARPS>
__global__ void __launch_bounds__(128)
    join_kernel(View c, AttentionArgs a, int seq0, int nseq, Parts parts, Shape shape) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int group = a.num_heads / c.kv_heads;
  const int64_t tok = w / a.num_heads;
  const int hq = (int)(w - tok * a.num_heads);
  const int32_t* cu = a.cu_new + seq0;
  if (tok >= a.total_tokens || tok < cu[0] || tok >= cu[nseq]) return;
  const int b = find_request(cu, nseq, (unsigned long long)tok);
  Request q;
  if (!load_request(c, a, seq0 + b, ROWS, false, q) || tok < q.bos || tok >= q.bos + q.n) return;
  const unsigned long long per = parts.plan[nseq + 1] * WARPS;
  const int h = hq / group;
  const int64_t rr = (tok - q.bos) * group + hq % group;
  const unsigned long long u0 =
      parts.plan[b] + (unsigned long long)(h * q.rt + rr / ROWS) * q.tiles;
  const int first = (int)(u0 / per), last = (int)((u0 + q.tiles - 1) / per);
  if (first == last) return;
  const int row = (int)(rr % ROWS);
  auto at_of = [&](int cta) {
    return (int64_t)(shape.warp_slots() + 2 * cta + (cta == first ? 1 : 0)) * ROWS + row;
  };
  float top = -INFINITY;
  for (int i = first + lane; i <= last; i += 32) top = fmaxf(top, parts.ml[at_of(i)].x);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
  float sum = 0.f, x[D / 32] = {};
#pragma unroll 4
  for (int i = first; i <= last; ++i) {
    const int64_t at = at_of(i);
    const float2 ml = parts.ml[at];
    const float k = top == -INFINITY ? 1.f : ex2_approx(ml.x - top);
    sum = fmaf(ml.y, k, sum);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) x[j] = fmaf(parts.o[at * D + j * 32 + lane], k, x[j]);
  }
  const float inv = sum == 0.f ? 0.f : exponent_scale(c.v_exp, h, 1) / sum;
  T* out = static_cast<T*>(a.out) + w * D;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) IO<T>::st(out + j * 32 + lane, x[j] * inv);
  if (a.lse && lane == 0) a.lse[w] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

int sm_count() {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

constexpr size_t kPlanBytes = ((kMaxSeqs + 2) * 8 + 255) / 256 * 256;

// One CTA of `WARPS` warps with `STAGES` tiles in flight each, `CTAS` per SM.
template <typename T, int D, int NT, int WARPS, int STAGES, int CTAS>
struct Split {
  static constexpr int ROWS = 8 * NT;
  static Shape shape() { return Shape{sm_count() * CTAS, WARPS}; }
  static size_t workspace() {
    const size_t slots = shape().slots();
    return kPlanBytes + slots * ROWS * (D * 4 + 8);
  }
  static cudaError_t launch(const View& c, const AttentionArgs& a, cudaStream_t st) {
    static PerDeviceInit init;
    using S = Smem<T, D, NT, WARPS, STAGES>;
    auto* kernel = split_kernel<T, D, NT, WARPS, STAGES, CTAS>;
    cudaError_t e = init.run([&] {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)sizeof(S));
    });
    if (e != cudaSuccess) return e;
    const Shape sh = shape();
    Parts parts;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    parts.plan = reinterpret_cast<unsigned long long*>(ws);
    parts.o = reinterpret_cast<float*>(ws + kPlanBytes);
    parts.ml = reinterpret_cast<float2*>(parts.o + (size_t)sh.slots() * ROWS * D);
    const int64_t es = sizeof(T);
    const int q_vec = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 &&
                      a.q_token_stride * es % 16 == 0 && a.q_head_stride * es % 16 == 0;
    const int64_t rows = (int64_t)a.total_tokens * a.num_heads;
    for (int seq0 = 0; seq0 < a.num_seqs; seq0 += kMaxSeqs) {
      const int nseq = std::min(kMaxSeqs, a.num_seqs - seq0);
      kernel<<<sh.ctas, WARPS * 32, sizeof(S), st>>>(c, a, seq0, nseq, parts, q_vec);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      join_kernel<T, D, ROWS, WARPS>
          <<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(c, a, seq0, nseq, parts, sh);
      e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
};

// Calls f with the variant for the call's types and expected rows per kv head.
template <typename F>
auto dispatch(const View& c, const AttentionArgs& a, F&& f) {
  const int64_t rows = (int64_t)a.max_new * (a.num_heads / c.kv_heads);
  if (a.bf16) {
    using T = __nv_bfloat16;
    if (a.head_dim == 128) {
      if (rows <= 8) return f(Split<T, 128, 1, 8, 2, 2>{});
      if (rows <= 16) return f(Split<T, 128, 2, 8, 4, 1>{});
      return f(Split<T, 128, 4, 8, 4, 1>{});
    }
    if (rows <= 8) return f(Split<T, 64, 1, 8, 4, 2>{});
    if (rows <= 16) return f(Split<T, 64, 2, 8, 4, 2>{});
    return f(Split<T, 64, 4, 8, 4, 1>{});
  }
  if (a.head_dim == 128) {
    if (rows <= 8) return f(Split<float, 128, 1, 8, 4, 1>{});
    return f(Split<float, 128, 2, 8, 4, 1>{});
  }
  if (rows <= 8) return f(Split<float, 64, 1, 8, 4, 2>{});
  return f(Split<float, 64, 2, 8, 4, 1>{});
}

}  // namespace

size_t cache_attention_workspace_bytes(const View& c, const AttentionArgs& a) {
  return dispatch(c, a, [&](auto v) { return decltype(v)::workspace(); });
}

cudaError_t launch_cache_attention(const View& c, const AttentionArgs& a, cudaStream_t st) {
  return dispatch(c, a, [&](auto v) { return decltype(v)::launch(c, a, st); });
}

}  // namespace kda
