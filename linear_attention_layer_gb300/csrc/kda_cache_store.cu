// kda_cache_store.cu -- kda_cache_append and kda_cache_read: keys and values
// between their own type and the cache's 4-bit blocks.
//
// One thread takes one block of 16 channels: its scale is a maximum over the
// thread's own registers, its codes are one 8-byte store, and nothing is shared
// between threads.  Both calls read and write each value once and are bound by
// HBM as long as a value costs few enough instructions (about six; HBM's rate
// leaves 11), which decides how the rounding below is done.  Measured for 270336 tokens x 8
// heads x 128 channels of bf16, 1.42 GB each way: append 283 us (0.75 of the measured HBM
// rate; 175 warp instructions a block, most of the wait for the loads of CTAs that live
// for one of them), read 240 us (0.88).
//
// A CTA takes 8 tokens of K or of V, a thread one token and block and every so many
// heads: where the token's slot lies is worked out once, the heads are strides.  Lanes
// of K go blocks first, then tokens (a token's codes are one run, the next token's follow);
// lanes of V tokens first, the layout keeping the blocks of 8 tokens together.  Either way
// neighbouring tokens of a prompt fill whole sectors.
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

// One thread's token, block and first head of a CTA's 8 tokens.
template <int D, bool TOKENS_FIRST>
struct Item {
  static constexpr int kBlocks = D / kGroup;
  int token, block, head;
  __device__ __forceinline__ Item() {
    const int i = threadIdx.x & (8 * kBlocks - 1);
    head = threadIdx.x / (8 * kBlocks);
    token = blockIdx.x * 8 + (TOKENS_FIRST ? i & 7 : i / kBlocks);
    block = TOKENS_FIRST ? i >> 3 : i & (kBlocks - 1);
  }
  __device__ __forceinline__ static int head_step() { return blockDim.x / (8 * kBlocks); }
};

// Threads that give every head of a few its own, up to 256.
template <int D>
int threads_for(int heads) {
  const int per_head = 8 * (D / kGroup);
  return per_head * std::min(heads, kThreads / per_head);
}

// Offset of head 0's group in the cache and of the block's bytes in it.
template <int D, bool V>
__device__ __forceinline__ int64_t place_of(const View& c, FastDiv page_div, int slot, int b,
                                            int& codes, int& scale) {
  const int page = page_div.div(slot);
  const int tok = slot - page * c.page_size, i = tok % kGroup;
  codes = V ? Layout<D>::v_codes(i, b) : Layout<D>::k_codes(i, b);
  scale = V ? Layout<D>::v_scale(i, b) : Layout<D>::k_scale(i, b);
  // groups of a cache are fewer than 2^31: each has 1152 bytes at least
  const int group = page * c.kv_heads * (c.page_size / kGroup) + tok / kGroup;
  return (int64_t)group * Layout<D>::kGroupBytes;
}

struct Source {
  const void* p;
  int token_stride, head_stride;  // elements
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
    for (int h = 0; h < 2; ++h) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        y[i] = isinf(x[8 * h + i]) ? x[8 * h + i] : div_to_odd(x[8 * h + i], s);
      w[h] = f32x8_to_e2m1(y);
    }
  }
  codes = make_uint2(w[0], w[1]);
  return sb;
}

// The same of 16 bf16 values, two in a word.  x has 8 significant bits and s 4, a
// border between two codes times s at most 7: x / s either is a border, a multiple of
// 1/4, or lies 2^-9 of it away, 2^-11 at least.  So the product with an approximate 1 / s
// (2^-21 off at most) is brought back onto the borders by rounding it to a multiple of
// 2^-12: adding a number between 2^11 and 2^12 and taking it away again, the first in
// one operation with the product.  The exact division above costs twenty instructions a
// value.  The same holds of max |x| / 6 and the borders of E4M3: times 6 they have 8 bits
// too, and rounding to 16 fraction bits brings the product with 1 / 6 back onto them.
__device__ __forceinline__ uint32_t quantise(uint32_t (&x)[8], float pre, uint2& codes,
                                             bool& not_finite) {
  constexpr float kOnto = 2560.f;
  uint32_t top2 = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t m;
    asm("abs.bf16x2 %0, %1;" : "=r"(m) : "r"(x[i]));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top2) : "r"(m));
  }
  const uint32_t top_bits = max(top2 & 0x7fffu, top2 >> 16 & 0x7fffu);
  if (top_bits >= 0x7f80u) {
    float y[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = tc::bf16_lo(x[i]);
      y[2 * i + 1] = tc::bf16_hi(x[i]);
    }
    return quantise(y, pre, codes, not_finite);
  }
  const float top = fminf(__uint_as_float(top_bits << 16) * pre, 3.e38f) * (1.f / 6.f);
  const uint32_t sb =
      f32_to_e4m3(__uint_as_float((__float_as_uint(top) + 0x40u) & ~0x7fu));
  const float r = sb ? __fdividef(pre, e4m3_to_f32(sb)) : 0.f;
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = fmaf(tc::bf16_lo(x[4 * h + i]), r, kOnto) - kOnto;
      y[2 * i + 1] = fmaf(tc::bf16_hi(x[4 * h + i]), r, kOnto) - kOnto;
    }
    w[h] = f32x8_to_e2m1(y);
  }
  codes = make_uint2(w[0], w[1]);
  return sb;
}

// 16 values at p as 32-bit words.  VEC: p is 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void fetch(const T* p, uint32_t (&w)[4 * sizeof(T)]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = __float_as_uint(IO<T>::ld(p + 2 * i)) >> 16 |
             __float_as_uint(IO<T>::ld(p + 2 * i + 1));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(IO<T>::ld(p + i));
  }
}

template <typename T, int D, bool VEC, bool V>
__device__ __forceinline__ void append_blocks(const View& c, FastDiv page_div, int tokens,
                                              const Source& src,
                                              const int64_t* __restrict__ slots, int* err) {
  const Item<D, V> it;
  if (it.token >= tokens || it.head >= c.kv_heads) return;
  const int step = it.head_step(), head_bytes = c.page_size / kGroup * Layout<D>::kGroupBytes;
  const T* p = static_cast<const T*>(src.p) + (int64_t)it.token * src.token_stride +
               (int64_t)it.head * src.head_stride + it.block * kGroup;
  const int64_t next = (int64_t)step * src.head_stride;
  // The values of two heads are under way before the slot is looked at: a CTA lives for one
  // latency of memory, not two (append of 270336 tokens x 8 heads: 355 us -> 283).
  uint32_t w[2][4 * sizeof(T)];
  auto fetch2 = [&](int h) {
    fetch<T, VEC>(p, w[0]);
    if (h + step < c.kv_heads) fetch<T, VEC>(p + next, w[1]);
    p += 2 * next;
  };
  fetch2(it.head);
  const int64_t slot = __ldg(slots + it.token);
  if (slot < 0 || slot >= (int64_t)c.num_pages * c.page_size) {
    if (slot != -1) report_error(err, kErrDeviceCheck);
    return;
  }
  int codes_at, scale_at;
  uint8_t* g = c.pages + place_of<D, V>(c, page_div, (int)slot, it.block, codes_at, scale_at);
  g += (int64_t)it.head * head_bytes;
  bool not_finite = false;
  for (int h = it.head; h < c.kv_heads; h += 2 * step) {
    if (h != it.head) fetch2(h);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (h + e * step < c.kv_heads) {
        uint2 codes;
        uint32_t sb;
        const float pre = exponent_scale(V ? c.v_exp : c.k_exp, h + e * step, -1);
        if constexpr (sizeof(T) == 2) {
          sb = quantise(w[e], pre, codes, not_finite);
        } else {
          float x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(w[e][i]);
          sb = quantise(x, pre, codes, not_finite);
        }
        *reinterpret_cast<uint2*>(g + codes_at) = codes;
        g[scale_at] = (uint8_t)sb;
      }
      g += (int64_t)step * head_bytes;
    }
  }
  if (not_finite) report_error(err, kErrDeviceCheck);
}

template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kThreads)
    append_kernel(View c, FastDiv page_div, int tokens, Source k, Source v,
                  const int64_t* __restrict__ slots, int* err) {
  if (blockIdx.y)
    append_blocks<T, D, VEC, true>(c, page_div, tokens, v, slots, err);
  else
    append_blocks<T, D, VEC, false>(c, page_div, tokens, k, slots, err);
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

template <typename T, int D, bool V>
__device__ __forceinline__ void read_blocks(const View& c, FastDiv page_div, int tokens,
                                            const int64_t* __restrict__ slots,
                                            T* __restrict__ out, int* err) {
  const Item<D, false> it;  // blocks first for both: whole rows are written
  if (it.token >= tokens) return;
  const int64_t slot = __ldg(slots + it.token);
  const bool there = slot >= 0 && slot < (int64_t)c.num_pages * c.page_size;
  if (!there && slot != -1) report_error(err, kErrDeviceCheck);
  int codes_at = 0, scale_at = 0;
  const uint8_t* g = c.pages;
  if (there) g += place_of<D, V>(c, page_div, (int)slot, it.block, codes_at, scale_at);
  const int step = it.head_step(), head_bytes = c.page_size / kGroup * Layout<D>::kGroupBytes;
  g += (int64_t)it.head * head_bytes;
  T* p = out + ((int64_t)it.token * c.kv_heads + it.head) * D + it.block * kGroup;
#pragma unroll 2
  for (int h = it.head; h < c.kv_heads; h += step) {
    float x[16] = {};
    if (there) {
      const uint2 codes = *reinterpret_cast<const uint2*>(g + codes_at);
      const float s = e4m3_to_f32(g[scale_at]) * exponent_scale(V ? c.v_exp : c.k_exp, h, 1);
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
    store_block(p, x);
    p += step * D;
    g += (int64_t)step * head_bytes;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    read_kernel(View c, FastDiv page_div, int tokens, const int64_t* __restrict__ slots,
                T* __restrict__ k, T* __restrict__ v, int* err) {
  if (blockIdx.y)
    read_blocks<T, D, true>(c, page_div, tokens, slots, v, err);
  else
    read_blocks<T, D, false>(c, page_div, tokens, slots, k, err);
}

template <typename T, int D>
cudaError_t append(const CacheArgs& a, cudaStream_t st) {
  const Source k{a.k, (int)a.strides[0], (int)a.strides[1]},
      v{a.v, (int)a.strides[2], (int)a.strides[3]};
  const int el = 16 / sizeof(T);
  bool vec = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15) == 0;
  for (int64_t s : a.strides) vec = vec && s % el == 0;
  const dim3 grid((unsigned)((a.tokens + 7ll) / 8), 2);
  auto* kernel = vec ? append_kernel<T, D, true> : append_kernel<T, D, false>;
  kernel<<<grid, threads_for<D>(a.view.kv_heads), 0, st>>>(a.view, FastDiv(a.view.page_size),
                                                           a.tokens, k, v, a.slots, a.err);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t read(const CacheArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.tokens + 7ll) / 8), 2);
  read_kernel<T, D><<<grid, threads_for<D>(a.view.kv_heads), 0, st>>>(
      a.view, FastDiv(a.view.page_size), a.tokens, a.slots, static_cast<T*>(a.k_out),
      static_cast<T*>(a.v_out), a.err);
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
