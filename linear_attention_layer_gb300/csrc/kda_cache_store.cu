// kda_cache_store.cu -- kda_cache_append and kda_cache_read: keys and values
// between their own type and the cache's 4-bit blocks.
//
// One thread takes one block of 16 channels: its scale is a maximum over the
// thread's own registers, its codes are one 8-byte store, and nothing is shared
// between threads.  Both calls read and write each value once and are bound by
// HBM as long as a value costs few enough instructions (about six; HBM's rate
// leaves 11), which decides how the rounding below is done.
//
// Threads of K go blocks first: the 8 (4) blocks of a token's head are one run of
// code bytes.  Threads of V go 8 neighbouring tokens first: the layout keeps the
// blocks of 8 tokens together, so tokens of one prompt fill whole sectors.
#include <algorithm>

#include "kda_cache.cuh"
#include "kda_launch.h"
#include "tc_ptx.cuh"

namespace kda {
namespace {

using namespace cache;

constexpr int kThreads = 256;

// n / d for n < 2^31 by a product (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994): m = floor(2^(31 + s) / d) + 1, 2^s >= d.
struct FastDiv {
  uint32_t d, m, s;
  explicit FastDiv(uint32_t x) : d(x), s(0) {
    while ((1ull << s) < d) ++s;
    m = (uint32_t)((1ull << (31 + s)) / d + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (uint32_t)(((uint64_t)n * m) >> (31 + s));
  }
};

// Where the threads' blocks lie: kv heads of a token, tokens of a page.
struct Grid {
  FastDiv heads, page;
  int tokens;
  int64_t limit;
  Grid(const View& c, int n)
      : heads(c.kv_heads), page(c.page_size), tokens(n),
        limit((int64_t)c.num_pages * c.page_size) {}
};

// One thread's block: a CTA takes 8 tokens, K in the first half of the grid's y.
template <int D>
struct Item {
  int token, head, block;
  __device__ __forceinline__ bool set(const Grid& gr, bool is_v, int i) {
    constexpr int kBlocks = D / kGroup;
    int t;
    if (is_v) {  // tokens, blocks, heads
      t = i & 7;
      block = (i >> 3) & (kBlocks - 1);
      head = i / (8 * kBlocks);
    } else {  // blocks, heads, tokens
      block = i & (kBlocks - 1);
      const uint32_t r = (uint32_t)i / kBlocks;
      t = gr.heads.div(r);
      head = r - t * gr.heads.d;
    }
    token = blockIdx.x * 8 + t;
    return token < gr.tokens;
  }
};

// Which bytes of the cache a slot's block has.
struct Place {
  uint8_t* codes;
  uint8_t* scale;
};
template <int D>
__device__ __forceinline__ Place place_of(const View& c, const Grid& gr, bool is_v, int64_t slot,
                                          int head, int b) {
  const int page = gr.page.div((uint32_t)slot);
  const int tok = (int)slot - page * c.page_size;
  uint8_t* g = group_of<D>(c, page, tok, head);
  const int i = tok % kGroup;
  return {g + (is_v ? Layout<D>::v_codes(i, b) : Layout<D>::k_codes(i, b)),
          g + (is_v ? Layout<D>::v_scale(i, b) : Layout<D>::k_scale(i, b))};
}

struct Source {
  const void* p;
  int64_t token_stride;
  int64_t head_stride;
};

// Scale byte and codes of 16 fp32 values; `pre` is the head's power of two.
__device__ __forceinline__ uint32_t quantise(float (&x)[16], float pre, uint2& codes,
                                             bool& not_finite) {
  float top = 0.f, probe = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    probe = fmaf(x[i], 0.f, probe);  // NaN as soon as one value is not finite
    x[i] *= pre;
    top = fmaxf(top, fabsf(x[i]));
  }
  if (probe != 0.f) {
    not_finite = true;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (isnan(x[i])) x[i] = 0.f;
  }
  const uint32_t sb = isinf(top) ? 0x7eu : f32_to_e4m3(div_to_odd(top, 6.f));
  const float s = e4m3_to_f32(sb);
  uint32_t w[2] = {0u, 0u};
  if (sb != 0u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = isinf(x[2 * i]) ? x[2 * i] : div_to_odd(x[2 * i], s);
      const float b = isinf(x[2 * i + 1]) ? x[2 * i + 1] : div_to_odd(x[2 * i + 1], s);
      w[i >> 2] |= f32x2_to_e2m1(a, b) << (8 * (i & 3));
    }
  }
  codes = make_uint2(w[0], w[1]);
  return sb;
}

// The same of 16 bf16 values, two in a word.  x has 8 significant bits and s 4, a
// border between two codes times s at most 7, so x / s either is a border or lies
// 2^-9 of it away at least: the product with the rounded 1 / s, 2^-23 off at most,
// is brought back onto the borders by rounding it to 16 fraction bits.  That costs
// two integer instructions a value where the exact division above costs twenty.
__device__ __forceinline__ uint32_t quantise(uint32_t (&x)[8], float pre, uint2& codes,
                                             bool& not_finite) {
  uint32_t top2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top2 = __vmaxu2(top2, x[i] & 0x7fff7fffu);
  const uint32_t top_bits = max(top2 & 0xffffu, top2 >> 16);
  if (top_bits >= 0x7f80u) {
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = tc::bf16_lo(x[i]);
      y[2 * i + 1] = tc::bf16_hi(x[i]);
    }
    return quantise(y, pre, codes, not_finite);
  }
  const float top = fminf(__uint_as_float(top_bits << 16) * pre, 3.e38f);
  const uint32_t sb = f32_to_e4m3(div_to_odd(top, 6.f));
  const float r = sb ? pre / e4m3_to_f32(sb) : 0.f;  // a power of two times 8 / 8 .. 8 / 15
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = tc::bf16_lo(x[i]) * r, b = tc::bf16_hi(x[i]) * r;
    w[i >> 2] |= f32x2_to_e2m1(__uint_as_float((__float_as_uint(a) + 0x40u) & ~0x7fu),
                               __uint_as_float((__float_as_uint(b) + 0x40u) & ~0x7fu))
                 << (8 * (i & 3));
  }
  codes = make_uint2(w[0], w[1]);
  return sb;
}

template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kThreads)
    append_kernel(View c, Grid gr, Source k, Source v, const int64_t* __restrict__ slots,
                  int* err) {
  const bool is_v = blockIdx.y;
  const Source src = is_v ? v : k;
  const int items = 8 * c.kv_heads * (D / kGroup);
  for (int j = threadIdx.x; j < items; j += kThreads) {
    Item<D> it;
    if (!it.set(gr, is_v, j)) continue;
    const int64_t slot = __ldg(slots + it.token);
    const T* p = static_cast<const T*>(src.p) + it.token * src.token_stride +
                 it.head * src.head_stride + it.block * kGroup;
    uint2 codes;
    uint32_t sb;
    bool not_finite = false;
    const float pre = exponent_scale(is_v ? c.v_exp : c.k_exp, it.head, -1);
    if (slot < 0 || slot >= gr.limit) {
      if (slot != -1) report_error(err, kErrDeviceCheck);
      continue;
    }
    if constexpr (sizeof(T) == 2 && VEC) {
      const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
      const uint4 b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
      uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      sb = quantise(x, pre, codes, not_finite);
    } else if constexpr (sizeof(T) == 2) {
      uint32_t x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = __float_as_uint(IO<T>::ld(p + 2 * i)) >> 16 |
               __float_as_uint(IO<T>::ld(p + 2 * i + 1));
      sb = quantise(x, pre, codes, not_finite);
    } else {
      float x[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (VEC) {
          const float4 f = __ldcs(reinterpret_cast<const float4*>(p) + i);
          x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
        } else {
#pragma unroll
          for (int l = 0; l < 4; ++l) x[4 * i + l] = IO<T>::ld(p + 4 * i + l);
        }
      }
      sb = quantise(x, pre, codes, not_finite);
    }
    if (not_finite) report_error(err, kErrDeviceCheck);
    const Place pl = place_of<D>(c, gr, is_v, slot, it.head, it.block);
    *reinterpret_cast<uint2*>(pl.codes) = codes;
    *pl.scale = (uint8_t)sb;
  }
}

template <typename T>
__device__ __forceinline__ void store_block(T* p, const float (&x)[16]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __stcs(reinterpret_cast<float4*>(p) + i,
             make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
  } else {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(reinterpret_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    read_kernel(View c, Grid gr, const int64_t* __restrict__ slots, T* __restrict__ k,
                T* __restrict__ v, int* err) {
  const bool is_v = blockIdx.y;
  const int items = 8 * c.kv_heads * (D / kGroup);
  for (int j = threadIdx.x; j < items; j += kThreads) {
    Item<D> it;
    if (!it.set(gr, false, j)) continue;  // blocks first for both: whole rows are written
    const int64_t slot = __ldg(slots + it.token);
    float x[16];
    if (slot < 0 || slot >= gr.limit) {
      if (slot != -1) report_error(err, kErrDeviceCheck);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.f;
    } else {
      const Place pl = place_of<D>(c, gr, is_v, slot, it.head, it.block);
      const uint2 codes = *reinterpret_cast<const uint2*>(pl.codes);
      const float s =
          e4m3_to_f32(*pl.scale) * exponent_scale(is_v ? c.v_exp : c.k_exp, it.head, 1);
      const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
      for (int l = 0; l < 2; ++l) {
        uint32_t r4[4];
        e2m1x8_to_f16(w[l], r4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r4[i]));
          x[8 * l + 2 * i] = f.x * s;
          x[8 * l + 2 * i + 1] = f.y * s;
        }
      }
    }
    store_block((is_v ? v : k) + ((int64_t)it.token * c.kv_heads + it.head) * D + it.block * kGroup,
                x);
  }
}

template <typename T, int D>
cudaError_t append(const CacheArgs& a, cudaStream_t st) {
  const Source k{a.k, a.strides[0], a.strides[1]}, v{a.v, a.strides[2], a.strides[3]};
  const int el = 16 / sizeof(T);
  bool vec = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15) == 0;
  for (int64_t s : a.strides) vec = vec && s % el == 0;
  const Grid gr(a.view, a.tokens);
  const dim3 grid((unsigned)((a.tokens + 7ll) / 8), 2);
  auto* kernel = vec ? append_kernel<T, D, true> : append_kernel<T, D, false>;
  kernel<<<grid, kThreads, 0, st>>>(a.view, gr, k, v, a.slots, a.err);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t read(const CacheArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.tokens + 7ll) / 8), 2);
  read_kernel<T, D><<<grid, kThreads, 0, st>>>(a.view, Grid(a.view, a.tokens), a.slots,
                                               static_cast<T*>(a.k_out), static_cast<T*>(a.v_out),
                                               a.err);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheArgs& a, cudaStream_t st) {
  if (a.bf16)
    return a.head_dim == 128 ? append<__nv_bfloat16, 128>(a, st) : append<__nv_bfloat16, 64>(a, st);
  return a.head_dim == 128 ? append<float, 128>(a, st) : append<float, 64>(a, st);
}

cudaError_t launch_cache_read(const CacheArgs& a, cudaStream_t st) {
  if (a.bf16)
    return a.head_dim == 128 ? read<__nv_bfloat16, 128>(a, st) : read<__nv_bfloat16, 64>(a, st);
  return a.head_dim == 128 ? read<float, 128>(a, st) : read<float, 64>(a, st);
}

}  // namespace kda
