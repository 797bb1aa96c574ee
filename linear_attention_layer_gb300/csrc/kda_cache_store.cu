// kda_cache_store.cu -- kda_cache_append and kda_cache_read: keys and values
// between their own type and the cache's 4-bit blocks.
//
// One thread takes one block of 16 channels: its scale is a maximum over the
// thread's own registers, its codes are one 8-byte store, and nothing is shared
// between threads.  Both calls are bound by HBM: they read and write each value
// once.
#include <algorithm>

#include "kda_cache.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

using namespace cache;

constexpr int kThreads = 256;

// 16 channels at p, as fp32.  VEC: p is 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void load_block(const T* p, float (&x)[16]) {
  if constexpr (!VEC) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = IO<T>::ld(p + i);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldcs(reinterpret_cast<const float4*>(p) + i);
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
}

struct Source {
  const void* p;
  int64_t token_stride;
  int64_t head_stride;
};

// The block's scale byte and its 16 codes.
__device__ __forceinline__ uint32_t quantise(float (&x)[16], float pre, uint2& codes,
                                             bool& odd_values) {
  float top = 0.f, probe = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    probe = fmaf(x[i], 0.f, probe);  // NaN as soon as one value is not finite
    x[i] *= pre;
    top = fmaxf(top, fabsf(x[i]));
  }
  if (probe != 0.f) {
    odd_values = true;
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

template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kThreads)
    append_kernel(View c, Source k, Source v, const int64_t* __restrict__ slots, int tokens,
                  int* err) {
  constexpr int kBlocks = D / kGroup;
  const int per_token = c.kv_heads * kBlocks;
  const int64_t n = 2ll * tokens * per_token;
  const int64_t limit = (int64_t)c.num_pages * c.page_size;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < n;
       e += (int64_t)gridDim.x * kThreads) {
    // neighbouring threads: blocks, heads, k then v, tokens
    const int b = (int)(e % kBlocks);
    const int64_t r = e / kBlocks;
    const int h = (int)(r % c.kv_heads);
    const int64_t r2 = r / c.kv_heads;
    const bool is_v = r2 & 1;
    const int64_t t = r2 >> 1;
    const int64_t slot = __ldg(slots + t);
    if (slot < 0 || slot >= limit) {
      if (slot != -1) report_error(err, kErrDeviceCheck);
      continue;
    }
    const Source& src = is_v ? v : k;
    float x[16];
    load_block<T, VEC>(static_cast<const T*>(src.p) + t * src.token_stride + h * src.head_stride +
                           b * kGroup,
                       x);
    uint2 codes;
    bool odd_values = false;
    const uint32_t sb =
        quantise(x, exponent_scale(is_v ? c.v_exp : c.k_exp, h, -1), codes, odd_values);
    if (odd_values) report_error(err, kErrDeviceCheck);
    const int64_t page = slot / c.page_size;
    const int tok = (int)(slot - page * c.page_size);
    uint8_t* g = group_of<D>(c, page, tok, h);
    const int i = tok % kGroup;
    *reinterpret_cast<uint2*>(
        g + (is_v ? Layout<D>::v_codes(i, b) : Layout<D>::k_codes(i, b))) = codes;
    g[is_v ? Layout<D>::v_scale(i, b) : Layout<D>::k_scale(i, b)] = (uint8_t)sb;
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
    read_kernel(View c, const int64_t* __restrict__ slots, int tokens, T* __restrict__ k,
                T* __restrict__ v, int* err) {
  constexpr int kBlocks = D / kGroup;
  const int64_t n = 2ll * tokens * c.kv_heads * kBlocks;
  const int64_t limit = (int64_t)c.num_pages * c.page_size;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < n;
       e += (int64_t)gridDim.x * kThreads) {
    const int b = (int)(e % kBlocks);
    const int64_t r = e / kBlocks;
    const int h = (int)(r % c.kv_heads);
    const int64_t r2 = r / c.kv_heads;
    const bool is_v = r2 & 1;
    const int64_t t = r2 >> 1;
    const int64_t slot = __ldg(slots + t);
    float x[16];
    if (slot < 0 || slot >= limit) {
      if (slot != -1) report_error(err, kErrDeviceCheck);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.f;
    } else {
      const int64_t page = slot / c.page_size;
      const int tok = (int)(slot - page * c.page_size);
      const uint8_t* g = group_of<D>(c, page, tok, h);
      const int i = tok % kGroup;
      const uint2 codes = *reinterpret_cast<const uint2*>(
          g + (is_v ? Layout<D>::v_codes(i, b) : Layout<D>::k_codes(i, b)));
      const float s = e4m3_to_f32(
                          g[is_v ? Layout<D>::v_scale(i, b) : Layout<D>::k_scale(i, b)]) *
                      exponent_scale(is_v ? c.v_exp : c.k_exp, h, 1);
      const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t r4[4];
        e2m1x8_to_f16(w[j], r4);
#pragma unroll
        for (int l = 0; l < 4; ++l) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r4[l]));
          x[8 * j + 2 * l] = f.x * s;
          x[8 * j + 2 * l + 1] = f.y * s;
        }
      }
    }
    store_block((is_v ? v : k) + (t * c.kv_heads + h) * D + b * kGroup, x);
  }
}

// Enough CTAs for every block once, at most 16 per SM (a grid stride takes the rest).
int grid_for(int64_t n) {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return (int)std::min<int64_t>((n + kThreads - 1) / kThreads, 16ll * sms);
}

template <typename T, int D>
cudaError_t append(const CacheArgs& a, cudaStream_t st) {
  const int64_t n = 2ll * a.tokens * a.view.kv_heads * (D / kGroup);
  const Source k{a.k, a.strides[0], a.strides[1]}, v{a.v, a.strides[2], a.strides[3]};
  const int el = 16 / sizeof(T);
  bool vec = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15) == 0;
  for (int64_t s : a.strides) vec = vec && s % el == 0;
  if (vec)
    append_kernel<T, D, true><<<grid_for(n), kThreads, 0, st>>>(a.view, k, v, a.slots, a.tokens,
                                                                a.err);
  else
    append_kernel<T, D, false><<<grid_for(n), kThreads, 0, st>>>(a.view, k, v, a.slots, a.tokens,
                                                                 a.err);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t read(const CacheArgs& a, cudaStream_t st) {
  const int64_t n = 2ll * a.tokens * a.view.kv_heads * (D / kGroup);
  read_kernel<T, D><<<grid_for(n), kThreads, 0, st>>>(a.view, a.slots, a.tokens,
                                                      static_cast<T*>(a.k_out),
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
