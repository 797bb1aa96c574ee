// kda_cache_split.cuh -- the attention kernel for few rows per kv head (decode steps, drafted
// windows), for both forms of the cache: what it computes and why it is built like this stands
// in kda_cache_attention.cu, what is different for 8 bits in kda_byte_cache_attention.cu.
#pragma once

#include <math.h>

#include <algorithm>

#include "kda_cache_attention.cuh"

namespace kda {
namespace {

using namespace cache;

constexpr int kTileGroups = 2;                   // groups of 16 keys in a tile
constexpr int kTileKeys = kTileGroups * kGroup;  // 32
constexpr int kMaxSeqs = 1024;                   // requests of one launch (their plan is in smem)

// Requests with more rows per kv head than this go to the chunk kernel, whose work for a
// key is that of 128 rows, or 256, whatever their number.  67 windows with up to 40 rows,
// three passes here: 172 us, with the requests of more than 32 rows over there 203 (they
// are a fifth of the keys, and the second set of launches costs 15 us); a pass over all of
// these keys takes 95 us here, the chunk kernel's only one 200, so four passes lose.  Measured
// with 8 query heads on a kv head, 128 channels and 4 bits; other shapes go by the same number.
// 8 bits, here and over there (4 or 8 query heads a kv head alike):
//     requests x keys, channels    16 rows    32 rows    48 rows    64 rows
//     67 x 8000, 128               192  340   358  344   508  348   668  350
//     67 x 8000,  64               117  332   221  332   326  334   425  336
//     67 x 2000, 128                70  124   105  127   150  131   196  133
//     67 x 2000,  64                44  116    73  117    96  118   128  120
//      1 x 4000, 128                20   29    22   30    23   31    25   32
//      1 x 32000, 128               29   46    36   47    42   48    52   49
// so with 64 channels and for single requests 48 is about the border; batches of windows with
// 128 channels would be served better by 32.
constexpr int64_t kSplitRows = 48;

// What a launch leaves in the workspace.
struct Parts {
  OpenUnit* open;  // [ctas]
  float* o;        // [slots][rows][D]
  float2* ml;      // [slots][rows]
};

// Slots: two per warp (part that starts inside its unit, part that starts it but
// does not end it), then two per CTA.
struct Shape {
  int ctas, warps;  // warps per CTA
  __host__ __device__ int warp_slots() const { return 2 * ctas * warps; }
  __host__ __device__ int slots() const { return warp_slots() + 2 * ctas; }
};

// Tiles of one unit: one at least, since a unit without keys still writes its zeros.
__device__ __forceinline__ int tiles_of(const Request& r) {
  return max(1, (r.kv + kTileKeys - 1) / kTileKeys);
}

// A place in the sequence of all tiles.
template <bool AFTER>
struct Cursor {
  int b;  // request (relative to the launch)
  int h;  // kv head
  int r;  // row tile
  int tile;
  int tiles;  // of the unit
  int rt;     // row tiles of the request
  Request q;

  __device__ __forceinline__ bool load(const View& c, const AttentionArgs& a, int seq0,
                                       const RowRange& range, int rows_per_tile) {
    const bool live = load_request<AFTER>(c, a, seq0 + b, range, false, q);
    tiles = tiles_of(q);
    rt = (int)((q.rows + rows_per_tile - 1) / rows_per_tile);
    return live;
  }
  __device__ __forceinline__ void seek(const View& c, const AttentionArgs& a, int seq0, int nseq,
                                       const RowRange& range, int rows_per_tile,
                                       const unsigned long long* plan, unsigned long long x) {
    b = find_last(plan, nseq, x);
    load(c, a, seq0, range, rows_per_tile);
    const unsigned long long off = x - plan[b];
    if (off >> 32 == 0) {
      const uint32_t u = (uint32_t)off / (uint32_t)tiles;
      tile = (int)((uint32_t)off - u * tiles);
      h = (int)(u / (uint32_t)rt);
      r = (int)(u - (uint32_t)h * (uint32_t)rt);
    } else {
      const unsigned long long u = off / tiles;
      tile = (int)(off - u * tiles);
      h = (int)(u / rt);
      r = (int)(u - (unsigned long long)h * rt);
    }
  }
  // The next tile; returns true when it starts a new unit.  Not past the last one.
  __device__ __forceinline__ bool next(const View& c, const AttentionArgs& a, int seq0, int nseq,
                                       const RowRange& range, int rows_per_tile) {
    if (++tile < tiles) return false;
    tile = 0;
    if (++r < rt) return true;
    r = 0;
    if (++h < c.kv_heads) return true;
    h = 0;
    while (++b < nseq && !load(c, a, seq0, range, rows_per_tile)) {
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

// Halves of a query or weight: two for fp32 outputs, one for bf16.
template <typename T>
constexpr int kTerms = sizeof(T) == 4 ? 2 : 1;

// The second half of a weight is held 2^11 times larger: 2^15 at most, and where the first half
// has run out of exponent the second still has 2^-36, 2^-43 of the row's largest weight (held as
// it is it ended at 2^-25: 40000 weights of 2^-33 behind one large one were lost).
constexpr float kSecond = 2048.f;

template <int BITS, typename T, int D, int NT, int WARPS, int STAGES>
struct Smem {
  static constexpr int kStage = kTileGroups * FormLayout<BITS, D>::kGroupBytes;
  static constexpr bool kQueriesHere = NT * kTerms<T> > 2;  // else they stay in registers
  alignas(128) uint8_t ring[WARPS][STAGES][kStage];
  uint2 q[kQueriesHere ? WARPS : 1][kQueriesHere ? NT * kTerms<T> * (D / 16) * 32 : 1];
  unsigned long long plan[kMaxSeqs + 1];
  uint64_t full[WARPS][STAGES];
  uint32_t valid[WARPS][STAGES];
  unsigned long long sums[WARPS];
  // Units that several warps have: [0] the one that enters the CTA, [1 + w] the one that
  // warp w starts and does not end.  last: the last warp of the launch that has some of it.
  struct Job {
    int bos, row0, rows, head;
    unsigned long long last;
  } job[WARPS + 1];
};

template <int BITS, typename T, int D, int NT, int WARPS, int STAGES, int CTAS>
__global__ void __launch_bounds__(WARPS * 32, CTAS)
    split_kernel(View c, AttentionArgs a, int seq0, int nseq, RowRange range, Parts parts,
                 int q_vec) {
  using L = FormLayout<BITS, D>;
  using S = Smem<BITS, T, D, NT, WARPS, STAGES>;
  constexpr int ROWS = 8 * NT;
  constexpr int TERMS = kTerms<T>;
  constexpr int QC = D / 4;       // channels of a query row per lane
  constexpr int KM = D / 16;      // products along the channels of K, and 16-channel tiles of V
  constexpr int VC = D / 8;       // channels of V per lane
  constexpr bool QREG = !S::kQueriesHere;
  constexpr bool AFTER = BITS == 8;  // launched after
  // A lane's words of a key that are loaded at a time (a word is two products with 4 bits, one
  // with 8), loads of a key, and words of a value.
  constexpr int KW = BITS == 4 ? D / 32 : 4, KLOADS = BITS == 4 ? 1 : D / 64;
  constexpr int VW = BITS == 4 ? D / 64 : D / 32;
  extern __shared__ uint8_t raw[];
  S& sm = *reinterpret_cast<S*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int group = a.num_heads / c.kv_heads;
  const int GP = c.page_size / kGroup;

  if constexpr (AFTER) wait_for_previous();
  // ---- the plan: tiles before each request ----
  if (tid <= WARPS) sm.job[tid].rows = 0;
  if (lane == 0) {
    for (int s = 0; s < STAGES; ++s)
      tc::mbar_init(&sm.full[warp][s], kTileGroups + (s == 0 ? a.withheld : 0));
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
      const bool live = load_request<AFTER>(c, a, seq0 + b, range, blockIdx.x == 0, r);
      sm.plan[b] = mine;
      if (live)
        mine += (unsigned long long)((r.rows + ROWS - 1) / ROWS) * tiles_of(r) * c.kv_heads;
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
  let_next_start();
  const int worker = blockIdx.x * WARPS + warp;
  const unsigned long long x0 = min(per * worker, total), x1 = min(x0 + per, total);
  const Shape shape{(int)gridDim.x, WARPS};

  if (x0 < x1) {
    Cursor<AFTER> ld, cp;
    cp.seek(c, a, seq0, nseq, range, ROWS, sm.plan, x0);
    ld = cp;
    auto open_job = [&](int i, unsigned long long end) {
      const int64_t row0 = (int64_t)cp.r * ROWS;
      if (lane == 0)
        sm.job[i] = {cp.q.bos, (int)row0, (int)min(cp.q.rows - row0, (int64_t)ROWS), cp.h,
                     (end - 1) / per};
    };
    if (warp == 0 && cp.tile > 0) open_job(0, x0 + (cp.tiles - cp.tile));
    const int count = (int)min(x1 - x0, (unsigned long long)INT32_MAX);
    int issued = 0;
    // Lane i holds the place of group 32 n + i of ld's unit, for the n being loaded, and issues
    // that group's copy itself.
    const uint8_t* src = nullptr;
    uint32_t present = 0;  // groups of the 32 that can be read
    auto find_pages = [&]() {
      const int gi = (ld.tile * kTileGroups & ~31) + lane;
      const bool in = gi < (ld.q.kv + kGroup - 1) / kGroup;
      const int page =
          in ? fetch<AFTER>(a.block_table + (int64_t)(seq0 + ld.b) * a.max_blocks + gi / GP) : 0;
      const bool sound = page >= 0 && page < c.num_pages;
      if (in && !sound) report_error(a.err, kErrDeviceCheck);
      src = c.pages + (((int64_t)page * c.kv_heads + ld.h) * GP + gi % GP) * L::kGroupBytes;
      present = __ballot_sync(0xffffffffu, in && sound);
    };
    auto issue = [&](int stage) {
      const int first = ld.tile * kTileGroups & 31;
      if ((lane ^ first) < kTileGroups) {
        uint64_t* bar = &sm.full[warp][stage];
        const int u = lane ^ first;
        if (u == 0) sm.valid[warp][stage] = present >> first & ((1u << kTileGroups) - 1);
        if (present >> lane & 1) {
          tc::mbar_arrive_expect_tx(bar, L::kGroupBytes);
          tc::bulk_load(sm.ring[warp][stage] + u * L::kGroupBytes, src, L::kGroupBytes, bar);
        } else {
          tc::mbar_arrive(bar);
        }
      }
      if (++issued < count) {
        const bool turn = ld.next(c, a, seq0, nseq, range, ROWS);
        if (turn || (ld.tile * kTileGroups & 31) == 0) find_pages();
      }
    };

    uint2 qf[QREG ? NT : 1][QREG ? KM : 1][QREG ? TERMS : 1] = {};
    uint2* const qs = sm.q[QREG ? 0 : warp];
    auto query = [&](int n, int i, int e) {
      if constexpr (QREG)
        return qf[n][i][e];
      else
        return qs[((n * KM + i) * TERMS + e) * 32 + lane];
    };
    float o[KM][NT][4];
    float l[NT][2];                          // the lane's sums of the weights
    float sf[NT][2], neg[NT][2], thr[NT][2]; // score factor, -m, raw score that moves m
    int see[NT][2];                          // keys that the lane's rows see
    int all_see = 0;                         // keys that every row of the unit sees
    int v_ref = 0;  // 8 bits: o holds sums times 2^(127 - v_ref); the largest exponent byte met
    int seg_tile = 0;

    // The unit's queries as they lie in memory.  They are asked for before the first keys: behind
    // every warp's copies they would wait for those (1 x 262144 tokens: 3.7 us).
    uint32_t raw_q[NT][QC * sizeof(T) / 4];
    auto fetch_queries = [&]() {
      const int64_t row0 = (int64_t)cp.r * ROWS;
      const int rows = (int)min((int64_t)cp.q.n * group - row0, (int64_t)ROWS);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int64_t row = row0 + n * 8 + g;
        const int64_t tok = cp.q.bos + row / group;
        const T* p = static_cast<const T*>(a.q) + tok * a.q_token_stride +
                     (cp.h * group + (int)(row % group)) * a.q_head_stride + t * QC;
        if (n * 8 + g >= rows) {
#pragma unroll
          for (int i = 0; i < QC * (int)sizeof(T) / 4; ++i) raw_q[n][i] = 0;
        } else if (q_vec) {
#pragma unroll
          for (int i = 0; i < QC * (int)sizeof(T) / 16; ++i) {
            const uint4 u = fetch<AFTER>(reinterpret_cast<const uint4*>(p) + i);
            raw_q[n][4 * i] = u.x, raw_q[n][4 * i + 1] = u.y;
            raw_q[n][4 * i + 2] = u.z, raw_q[n][4 * i + 3] = u.w;
          }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int i = 0; i < QC; ++i)
            raw_q[n][i] = fetch<AFTER>(reinterpret_cast<const uint32_t*>(p) + i);
        } else {
#pragma unroll
          for (int i = 0; i < QC / 2; ++i)
            raw_q[n][i] = fetch<AFTER>(reinterpret_cast<const uint16_t*>(p) + 2 * i) |
                          (uint32_t)fetch<AFTER>(reinterpret_cast<const uint16_t*>(p) + 2 * i + 1)
                              << 16;
        }
      }
    };
    auto start_unit = [&]() {
      const int64_t row0 = (int64_t)cp.r * ROWS;
      const int rows = (int)min((int64_t)cp.q.n * group - row0, (int64_t)ROWS);
      all_see = cp.q.kv - cp.q.n + (int)(row0 / group) + 1;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[QC], top = 0.f;
#pragma unroll
        for (int i = 0; i < QC * (int)sizeof(T) / 4; ++i) {
          if constexpr (sizeof(T) == 4) {
            x[i] = __uint_as_float(raw_q[n][i]);
          } else {
            x[2 * i] = tc::bf16_lo(raw_q[n][i]);
            x[2 * i + 1] = tc::bf16_hi(raw_q[n][i]);
          }
        }
#pragma unroll
        for (int i = 0; i < QC; ++i) top = fmaxf(top, fabsf(x[i]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const RowScale rs = row_scale(top, a.scale, exponent_scale(c.k_exp, cp.h, 1));
        const float down = rs.down, f = rs.f;
        sf[n][0] = __shfl_sync(0xffffffffu, f, t * 8);
        sf[n][1] = __shfl_sync(0xffffffffu, f, t * 8 + 4);
#pragma unroll
        for (int i = 0; i < KM; ++i) {
          const float y[4] = {x[4 * i] * down, x[4 * i + 1] * down, x[4 * i + 2] * down,
                              x[4 * i + 3] * down};
          uint2 f2[TERMS];
          f2[0] = make_uint2(tc::pack_f16(y[0], y[1]), tc::pack_f16(y[2], y[3]));
          if constexpr (TERMS == 2) {
            const float2 b0 = __half22float2(*reinterpret_cast<const __half2*>(&f2[0].x));
            const float2 b1 = __half22float2(*reinterpret_cast<const __half2*>(&f2[0].y));
            f2[1] = make_uint2(tc::pack_f16(y[0] - b0.x, y[1] - b0.y),
                               tc::pack_f16(y[2] - b1.x, y[3] - b1.y));
          }
#pragma unroll
          for (int e2 = 0; e2 < TERMS; ++e2) {
            if constexpr (QREG)
              qf[n][i][e2] = f2[e2];
            else
              qs[((n * KM + i) * TERMS + e2) * 32 + lane] = f2[e2];
          }
        }
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          neg[n][e2] = BITS == 4 ? 0.f : kUnset;
          thr[n][e2] = -INFINITY;
          const int r = n * 8 + 2 * t + e2;
          see[n][e2] = r < rows ? cp.q.kv - cp.q.n + (int)((row0 + r) / group) + 1 : 0;
        }
        l[n][0] = l[n][1] = 0.f;
      }
      v_ref = 0;
#pragma unroll
      for (int i = 0; i < KM; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][n][j] = 0.f;
      seg_tile = cp.tile;
    };

    // Ends the part of the unit that this warp had.
    auto end_part = [&](bool ends_unit) {
      const bool whole = ends_unit && seg_tile == 0;
      const int64_t row0 = (int64_t)cp.r * ROWS;
      const int rows = (int)min((int64_t)cp.q.n * group - row0, (int64_t)ROWS);
      const int slot = 2 * worker + (seg_tile == 0 ? 1 : 0);
      const float post = BITS == 4 ? exponent_scale(c.v_exp, cp.h, 1) : exponent_factor(v_ref);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[n][e];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          const bool unset = BITS == 4 ? thr[n][e] == -INFINITY : neg[n][e] == kUnset;
          const float m = unset ? -INFINITY : -neg[n][e];
          const int row = n * 8 + 2 * t + e;
          float x[VC];
          if (row < rows) {
            const float inv = !whole ? (BITS == 4 ? 1.f : post) : sum == 0.f ? 0.f : post / sum;
#pragma unroll
            for (int i = 0; i < KM; ++i) {
              x[2 * i] = o[i][n][e] * inv;
              x[2 * i + 1] = o[i][n][2 + e] * inv;
            }
            if (whole) {
              const int64_t rr = row0 + row;
              const int64_t at =
                  (cp.q.bos + rr / group) * a.num_heads + cp.h * group + rr % group;
              store_row<T, D>(static_cast<T*>(a.out) + at * D + g * VC, x);
              if (a.lse && g == 0) a.lse[at] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
            } else {
              const int64_t at = (int64_t)slot * ROWS + row;
              store_row<float, D>(parts.o + at * D + g * VC, x);
              if (g == 0) parts.ml[at] = make_float2(m, sum);
            }
          }
        }
    };

    // The K side of one tile, or a load of it, in registers as it comes from shared memory.
    struct Keys {
      uint32_t a[kTileGroups][KW], b[kTileGroups][KW];  // codes of keys g and g + 8
      uint32_t sc[kTileGroups][2][D / 64];              // 4 bits: their scales, twice in a word
    };
    float s[kTileGroups][NT][4];
    uint32_t pf[kTileGroups][NT][TERMS][2];
    auto load_keys = [&](const uint8_t* base, Keys& k, int part) {
#pragma unroll
      for (int u = 0; u < kTileGroups; ++u) {
        const uint8_t* p = base + u * L::kGroupBytes;
        if constexpr (BITS == 8) {
          p += part * 1024 + t * 16;
          const uint4 x = *reinterpret_cast<const uint4*>(p + g * 64);
          const uint4 y = *reinterpret_cast<const uint4*>(p + (g + 8) * 64);
          k.a[u][0] = x.x, k.a[u][1] = x.y, k.a[u][2] = x.z, k.a[u][3] = x.w;
          k.b[u][0] = y.x, k.b[u][1] = y.y, k.b[u][2] = y.z, k.b[u][3] = y.w;
        } else if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(p + g * 64 + t * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(p + (g + 8) * 64 + t * 16);
          k.a[u][0] = x.x, k.a[u][1] = x.y, k.a[u][2] = x.z, k.a[u][3] = x.w;
          k.b[u][0] = y.x, k.b[u][1] = y.y, k.b[u][2] = y.z, k.b[u][3] = y.w;
          const uint32_t w = *reinterpret_cast<const uint32_t*>(p + L::kKScales + g * 16 + t * 4);
          const uint32_t wa = e4m3x2_to_f16x2(w), wb = e4m3x2_to_f16x2(w >> 16);
          k.sc[u][0][0] = __byte_perm(wa, 0, 0x1010), k.sc[u][0][1] = __byte_perm(wa, 0, 0x3232);
          k.sc[u][1][0] = __byte_perm(wb, 0, 0x1010), k.sc[u][1][1] = __byte_perm(wb, 0, 0x3232);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(p + g * 32 + t * 8);
          const uint2 y = *reinterpret_cast<const uint2*>(p + (g + 8) * 32 + t * 8);
          k.a[u][0] = x.x, k.a[u][1] = x.y;
          k.b[u][0] = y.x, k.b[u][1] = y.y;
          const uint32_t w = e4m3x2_to_f16x2(
              *reinterpret_cast<const uint16_t*>(p + L::kKScales + g * 8 + t * 2));
          k.sc[u][0][0] = __byte_perm(w, 0, 0x1010);
          k.sc[u][1][0] = __byte_perm(w, 0, 0x3232);
        }
        if (part == 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[u][n][j] = 0.f;
        }
      }
    };
    // 8 bits: 4 channels a lane of every key, one product.
    auto score_word8 = [&](const Keys& k, int w) {
      uint32_t af[kTileGroups][4];
#pragma unroll
      for (int u = 0; u < kTileGroups; ++u) {
        e4m3x4_to_f16(k.a[u][w % KW], af[u][0], af[u][2]);
        e4m3x4_to_f16(k.b[u][w % KW], af[u][1], af[u][3]);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (TERMS == 1) {
          const uint2 q = query(n, w, 0);
#pragma unroll
          for (int u = 0; u < kTileGroups; ++u) tc::mma_16816_f16(s[u][n], af[u], q.x, q.y);
        } else {  // short sums, second halves first: see value_word
          float part[kTileGroups][4] = {};
#pragma unroll
          for (int e = TERMS - 1; e >= 0; --e) {
            const uint2 q = query(n, w, e);
#pragma unroll
            for (int u = 0; u < kTileGroups; ++u) tc::mma_16816_f16(part[u], af[u], q.x, q.y);
          }
#pragma unroll
          for (int u = 0; u < kTileGroups; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][n][i] += part[u][i];
        }
      }
    };
    // 4 bits: 8 channels a lane of every key, two products.
    auto score_word4 = [&](const Keys& k, int w) {
      uint32_t af[kTileGroups][2][4];
#pragma unroll
      for (int u = 0; u < kTileGroups; ++u) {
        uint32_t xa[4], xb[4];
        e2m1x8_to_f16(k.a[u][w], xa);
        e2m1x8_to_f16(k.b[u][w], xb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          af[u][j >> 1][2 * (j & 1)] = mul_f16x2(xa[j], k.sc[u][0][w / 2]);
          af[u][j >> 1][2 * (j & 1) + 1] = mul_f16x2(xb[j], k.sc[u][1][w / 2]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (TERMS == 1) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint2 q = query(n, 2 * w + j, 0);
#pragma unroll
            for (int u = 0; u < kTileGroups; ++u) tc::mma_16816_f16(s[u][n], af[u][j], q.x, q.y);
          }
        } else {  // short sums, second halves first: see value_word
          float part[kTileGroups][4] = {};
#pragma unroll
          for (int e = TERMS - 1; e >= 0; --e)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint2 q = query(n, 2 * w + j, e);
#pragma unroll
              for (int u = 0; u < kTileGroups; ++u)
                tc::mma_16816_f16(part[u], af[u][j], q.x, q.y);
            }
#pragma unroll
          for (int u = 0; u < kTileGroups; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][n][i] += part[u][i];
        }
      }
    };
    auto score_word = [&](const Keys& k, int w) {
      if constexpr (BITS == 8)
        score_word8(k, w);
      else
        score_word4(k, w);
    };
    auto tile_scores = [&](const uint8_t* base) {
      Keys k;
#pragma unroll
      for (int part = 0; part < KLOADS; ++part) {
        load_keys(base, k, part);
#pragma unroll
        for (int w = 0; w < KW; ++w) score_word(k, part * KW + w);
      }
    };
    struct Values {
      uint32_t c0[2][VW], c1[2][VW];  // [token][word] of tokens 2t.., 2t + 8..
    };
    // left (8 bits): tokens of the group that there are; what lies past them may be anything.
    auto load_values = [&](const uint8_t* base, int u, Values& v, int left) {
      const uint8_t* vb = base + u * L::kGroupBytes + L::kVCodes;
      if constexpr (BITS == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t(&w)[VW] = i < 2 ? v.c0[i & 1] : v.c1[i & 1];
          const uint8_t* p = vb + i * 4 * D + g * (D / 2) + t * (D / 8);
          if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(p);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x, w[1] = x.y;
          }
        }
        if (left < kGroup) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t(&w)[VW] = i < 2 ? v.c0[i & 1] : v.c1[i & 1];
            const uint32_t keep = 2 * t + (i & 1) + 8 * (i >> 1) < left ? ~0u : 0u;
#pragma unroll
            for (int j = 0; j < VW; ++j) w[j] &= keep;
          }
        }
      } else if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(vb + g * 64 + t * 16);
        const uint4 y = *reinterpret_cast<const uint4*>(vb + 4 * D + g * 64 + t * 16);
        v.c0[0][0] = x.x, v.c0[0][1] = x.y, v.c0[1][0] = x.z, v.c0[1][1] = x.w;
        v.c1[0][0] = y.x, v.c1[0][1] = y.y, v.c1[1][0] = y.z, v.c1[1][1] = y.w;
      } else {
        const uint8_t* p = vb + (g >> 1) * 64 + t * 16 + (g & 1) * 4;
        v.c0[0][0] = *reinterpret_cast<const uint32_t*>(p);
        v.c0[1][0] = *reinterpret_cast<const uint32_t*>(p + 8);
        v.c1[0][0] = *reinterpret_cast<const uint32_t*>(p + 4 * D);
        v.c1[1][0] = *reinterpret_cast<const uint32_t*>(p + 4 * D + 8);
      }
    };
    // o of channel tile i += values times the weights of group u.
    auto value_product = [&](int i, const uint32_t (&af)[4], int u) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if constexpr (TERMS == 1) {
          tc::mma_16816_f16(o[i][n], af, pf[u][n][0][0], pf[u][n][0][1]);
        } else {
          // The tensor cores cut off what they add up; over a long row that drifts towards
          // zero (9001 keys: 1e-5 of an fp32 output, so 5e-7).  Sums of 16 keys are added here,
          // rounded; the weights' second halves go first, where what is cut off is little.
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          tc::mma_16816_f16(part, af, pf[u][n][1][0], pf[u][n][1][1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) part[j] *= 1.f / kSecond;
          tc::mma_16816_f16(part, af, pf[u][n][0][0], pf[u][n][0][1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][n][j] += part[j];
        }
      }
    };
    // 8 bits: 4 channels a lane of one group's values, two products.  The bytes of two tokens
    // are brought side by side before the conversion.
    auto value_word8 = [&](const Values& v, int u, int wd) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t pick = j ? 0x7362 : 0x5140;
        uint32_t af[4];
        e4m3x4_to_f16(__byte_perm(v.c0[0][wd], v.c0[1][wd], pick), af[0], af[1]);
        e4m3x4_to_f16(__byte_perm(v.c1[0][wd], v.c1[1][wd], pick), af[2], af[3]);
        value_product(2 * wd + j, af, u);
      }
    };
    // 4 bits: 8 channels a lane of one group's values, four products.
    auto value_word4 = [&](const Values& v, uint32_t scales, int u, int wd) {
      const uint32_t s0 = e4m3x2_to_f16x2(scales), s1 = e4m3x2_to_f16x2(scales >> 16);
      // bytes of (even channel of the first token, of the second), then the odd channels
      uint32_t e0[4], d0[4], e1[4], d1[4];
      e2m1x8_to_f16((v.c0[0][wd] & 0x0f0f0f0fu) | ((v.c0[1][wd] << 4) & 0xf0f0f0f0u), e0);
      e2m1x8_to_f16(((v.c0[0][wd] >> 4) & 0x0f0f0f0fu) | (v.c0[1][wd] & 0xf0f0f0f0u), d0);
      e2m1x8_to_f16((v.c1[0][wd] & 0x0f0f0f0fu) | ((v.c1[1][wd] << 4) & 0xf0f0f0f0u), e1);
      e2m1x8_to_f16(((v.c1[0][wd] >> 4) & 0x0f0f0f0fu) | (v.c1[1][wd] & 0xf0f0f0f0u), d1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t af[4] = {mul_f16x2(e0[j], s0), mul_f16x2(d0[j], s0), mul_f16x2(e1[j], s1),
                                mul_f16x2(d1[j], s1)};
        value_product(wd * 4 + j, af, u);
      }
    };
    auto value_word = [&](const Values& v, uint32_t scales, int u, int wd) {
      if constexpr (BITS == 8)
        value_word8(v, u, wd);
      else
        value_word4(v, scales, u, wd);
    };

    int stage = 0;
    uint32_t parity = 0;
    // A lane whose wait gives up goes on with whatever is there, until the vote of the tile
    // that it waited for finds it (a vote after each wait: 265 us instead of 257 for the decode
    // step above).
    auto wait = [&](int st, uint32_t par) {
      const bool ok = wait_phase(&sm.full[warp][st], par, a.wait_cycles, nullptr);
      if (!ok) report_error(a.err, kErrTimeout);
      return ok;
    };
    fetch_queries();
    find_pages();
    for (int s = 0; s < STAGES && s < count; ++s) issue(s);
    start_unit();
    bool fed = wait(0, 0);
    tile_scores(sm.ring[warp][0]);
    int i = 0;
    for (; i < count; ++i) {
      // s holds the raw scores of tile i
      const uint8_t* const base = sm.ring[warp][stage];
      const uint32_t valid = sm.valid[warp][stage];
      const int key0 = cp.tile * kTileKeys;
      // A tile that some row does not see in full, or that is not all there.
      const bool edge = key0 + kTileKeys > all_see || valid != (1u << kTileGroups) - 1;
      uint32_t vs[kTileGroups] = {};  // 4 bits, scales of V: tokens 2t, 2t + 1, 2t + 8, 2t + 9
      float kf[kTileGroups] = {}, vf[kTileGroups];  // 8 bits, factors of the groups' K and V
      int vb[kTileGroups], v_top = 0;          // and the latter's exponent bytes
      int left[kTileGroups];                   // tokens of the groups
#pragma unroll
      for (int u = 0; u < kTileGroups; ++u) {
        left[u] = kGroup;
        if constexpr (BITS == 4) {
          vs[u] = *reinterpret_cast<const uint32_t*>(base + u * L::kGroupBytes + L::kVScales +
                                                     (D == 128 ? g : g >> 1) * 16 + t * 4);
        } else {
          const uint32_t x =
              *reinterpret_cast<const uint16_t*>(base + u * L::kGroupBytes + L::kScales);
          const bool here = valid >> u & 1;
          kf[u] = here ? exponent_factor(x & 255) : 1.f;
          vb[u] = here ? (int)(x >> 8) : 0;
          v_top = max(v_top, vb[u]);
        }
      }
      if (edge) {
#pragma unroll
        for (int u = 0; u < kTileGroups; ++u) {
          const bool here = valid >> u & 1;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (!here || key0 + u * kGroup + g + 8 * (j >> 1) >= see[n][j & 1])
                s[u][n][j] = -INFINITY;
          // what lies past the request's length may be anything: its scales become 0
          left[u] = here ? cp.q.kv - key0 - u * kGroup : 0;
          if constexpr (BITS == 4) {
            if (2 * t >= left[u]) vs[u] &= 0xffffff00u;
            if (2 * t + 1 >= left[u]) vs[u] &= 0xffff00ffu;
            if (2 * t + 8 >= left[u]) vs[u] &= 0xff00ffffu;
            if (2 * t + 9 >= left[u]) vs[u] &= 0x00ffffffu;
          }
        }
      }
      // 8 bits: factor of a raw score (kept positive, so that a masked one stays -infinity) and
      // its weight's exponent beside the reference.
      auto factor = [&](int u, int n, int e) {
        return fminf(fmaxf(sf[n][e] * kf[u], 1.2e-38f), 3.e38f);
      };
      float y[kTileGroups][NT][4];
      auto exponents = [&]() {
#pragma unroll
        for (int u = 0; u < kTileGroups; ++u)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float f[2] = {factor(u, n, 0), factor(u, n, 1)};
#pragma unroll
            for (int j = 0; j < 4; ++j) y[u][n][j] = fmaf(s[u][n][j], f[j & 1], neg[n][j & 1]);
          }
      };
      bool move = false;
      if constexpr (BITS == 8) {
        exponents();
        move = v_top > v_ref;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < kTileGroups; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            move |= BITS == 4 ? s[u][n][j] > thr[n][j & 1] : y[u][n][j] > kLift + kSlack;
      if (__any_sync(0xffffffffu, move || !fed)) {
        fed = __all_sync(0xffffffffu, fed);
        if (!fed) break;
        float down = 1.f;  // 8 bits: what a larger exponent of V takes from the sums
        if (BITS == 8 && v_top > v_ref) {
          down = v_ref ? power_below(v_ref - v_top) : 0.f;
          v_ref = v_top;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < kTileGroups; ++u) {
              const float both = fmaxf(s[u][n][e], s[u][n][2 + e]);
              top = fmaxf(top, BITS == 4 ? both : both * factor(u, n, e));
            }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1)
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            float keep = 1.f;
            if (top > -INFINITY) {
              const bool unset = BITS == 4 ? thr[n][e] == -INFINITY : neg[n][e] == kUnset;
              const float before = unset ? -INFINITY : -neg[n][e];
              const float m = fmaxf(before, (BITS == 4 ? top * sf[n][e] : top) - kLift);
              keep = ex2_approx(before - m);
              neg[n][e] = -m;
              if constexpr (BITS == 4) thr[n][e] = score_limit(m, sf[n][e]);
              l[n][e] *= keep;
            }
            if (BITS == 8 || top > -INFINITY) {
              if constexpr (BITS == 8) keep *= down;
#pragma unroll
              for (int i2 = 0; i2 < KM; ++i2) {
                o[i2][n][e] *= keep;
                o[i2][n][2 + e] *= keep;
              }
            }
          }
        if constexpr (BITS == 8) exponents();
      }
      if constexpr (BITS == 8) {
#pragma unroll
        for (int u = 0; u < kTileGroups; ++u) vf[u] = power_below(vb[u] - v_ref);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int u = 0; u < kTileGroups; ++u) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[u][n][j] = ex2_approx(
                BITS == 4 ? fmaf(s[u][n][j], sf[n][j & 1], neg[n][j & 1]) : y[u][n][j]);
          l[n][0] += s[u][n][0] + s[u][n][2];
          l[n][1] += s[u][n][1] + s[u][n][3];
          if constexpr (BITS == 8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[u][n][j] *= vf[u];
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t hi = tc::pack_f16(s[u][n][2 * j], s[u][n][2 * j + 1]);
            pf[u][n][0][j] = tc::movmatrix_trans(hi);
            if constexpr (TERMS == 2) {
              const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              pf[u][n][1][j] = tc::movmatrix_trans(tc::pack_f16(
                  (s[u][n][2 * j] - b.x) * kSecond, (s[u][n][2 * j + 1] - b.y) * kSecond));
            }
          }
        }
      int next = stage + 1;
      uint32_t next_parity = parity;
      if (next == STAGES) {
        next = 0;
        next_parity ^= 1;
      }
      const bool more = i + 1 < count;
      const bool ends_unit = cp.tile + 1 == cp.tiles;
      if (more && !ends_unit) {
        // values of tile i and scores of tile i + 1, two independent streams side by side
        fed = wait(next, next_parity);
        Keys k;
        load_keys(sm.ring[warp][next], k, 0);
#pragma unroll
        for (int u = 0; u < kTileGroups; ++u) {
          if (u > 0 && KLOADS == 2) load_keys(sm.ring[warp][next], k, u);
          Values v;
          load_values(base, u, v, left[u]);
#pragma unroll
          for (int wd = 0; wd < VW; ++wd) {
            score_word(k, u * VW + wd);
            value_word(v, vs[u], u, wd);
          }
        }
        ++cp.tile;
      } else {
#pragma unroll
        for (int u = 0; u < kTileGroups; ++u) {
          Values v;
          load_values(base, u, v, left[u]);
#pragma unroll
          for (int wd = 0; wd < VW; ++wd) value_word(v, vs[u], u, wd);
        }
        end_part(ends_unit);
        if (!ends_unit && seg_tile == 0)
          open_job(1 + warp, x1 + (cp.tiles - cp.tile - 1));
        if (more) {
          cp.next(c, a, seq0, nseq, range, ROWS);
          fetch_queries();
          start_unit();
          fed = wait(next, next_parity);
          tile_scores(sm.ring[warp][next]);
        }
      }
      __syncwarp();  // every lane has read the stage
      if (issued < count) issue(stage);
      stage = next;
      parity = next_parity;
    }
    if (!fed) {  // the copies under way, of tiles i on, land before the shared memory goes away
      if (lane < a.withheld) tc::mbar_arrive(&sm.full[warp][0]);
      for (; i < issued; ++i)
        wait_phase(&sm.full[warp][i % STAGES], i / STAGES & 1, a.wait_cycles, nullptr);
    }
  }

  // ---- join the parts of units that several warps of this CTA had ----
  __syncthreads();
  const int w0 = blockIdx.x * WARPS;
  if (tid == 0) parts.open[blockIdx.x].last = -1;
  int dealt = 0;  // rows dealt out to the warps in turn, over all jobs
  for (int j = 0; j <= WARPS; ++j) {
    const auto job = sm.job[j];
    if (job.rows == 0) continue;
    const bool starts = j > 0, ends = job.last < w0 + WARPS;
    const int first = w0 + (starts ? j - 1 : 0);
    const int last = (int)min(job.last, (unsigned long long)(w0 + WARPS - 1));
    if (starts && !ends && tid == 0)
      parts.open[blockIdx.x] = {job.bos, job.row0, job.rows, job.head, (int)(job.last / WARPS)};
    const int row_first = (warp - dealt % WARPS + WARPS) % WARPS;
    dealt += job.rows;
    for (int row = row_first; row < job.rows; row += WARPS) {
      RowSum<D> sum;
      sum.add(parts.o, parts.ml, first, last, [&](int w) {
        return (int64_t)(2 * w + (starts && w == first ? 1 : 0)) * ROWS + row;
      });
      if (starts && ends) {
        const int rr = job.row0 + row;
        const int64_t at = (int64_t)(job.bos + rr / group) * a.num_heads + job.head * group +
                           rr % group;
        sum.store(static_cast<T*>(a.out), a.lse, at, exponent_scale(c.v_exp, job.head, 1));
      } else {
        sum.store_part(parts.o, parts.ml,
                       (int64_t)(shape.warp_slots() + 2 * blockIdx.x + (starts ? 1 : 0)) * ROWS +
                           row);
      }
    }
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// One CTA of `WARPS` warps with `STAGES` tiles in flight each, `CTAS` per SM.
template <int BITS, typename T, int D, int NT, int WARPS, int STAGES, int CTAS>
struct Split {
  static constexpr int ROWS = 8 * NT;
  static Shape shape() { return Shape{sm_count() * CTAS, WARPS}; }
  static size_t workspace() {
    const size_t slots = shape().slots();
    return up256(shape().ctas * sizeof(OpenUnit)) + slots * ROWS * (D * 4 + 8);
  }
  static cudaError_t launch(const View& c, const AttentionArgs& a, const RowRange& range,
                            cudaStream_t st) {
    static PerDeviceInit init;
    using S = Smem<BITS, T, D, NT, WARPS, STAGES>;
    static_assert(CTAS * (sizeof(S) + 1024) <= 228 * 1024, "more shared memory than an SM has");
    auto* kernel = split_kernel<BITS, T, D, NT, WARPS, STAGES, CTAS>;
    cudaError_t e = init.run([&] {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)sizeof(S));
    });
    if (e != cudaSuccess) return e;
    const Shape sh = shape();
    Parts parts;
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    parts.open = reinterpret_cast<OpenUnit*>(ws);
    parts.o = reinterpret_cast<float*>(ws + up256(sh.ctas * sizeof(OpenUnit)));
    parts.ml = reinterpret_cast<float2*>(parts.o + (size_t)sh.slots() * ROWS * D);
    const int64_t es = sizeof(T);
    const int q_vec = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 &&
                      a.q_token_stride * es % 16 == 0 && a.q_head_stride * es % 16 == 0;
    for (int64_t seq0 = 0; seq0 < a.num_seqs; seq0 += kMaxSeqs) {
      const int nseq = (int)std::min<int64_t>(kMaxSeqs, a.num_seqs - seq0);
      if constexpr (BITS == 8) {
        e = launch_after(kernel, dim3(sh.ctas), WARPS * 32, sizeof(S), st, c, a, (int)seq0, nseq,
                         range, parts, q_vec);
      } else {
        kernel<<<sh.ctas, WARPS * 32, sizeof(S), st>>>(c, a, (int)seq0, nseq, range, parts, q_vec);
        e = cudaGetLastError();
      }
      if (e != cudaSuccess) return e;
      e = launch_join<T, D, 1, 4>(c, a, parts.open, parts.o, parts.ml, sh.warp_slots(), ROWS, sh.ctas,
                               st);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
};

}  // namespace
}  // namespace kda
