// kda_byte_cache.cuh -- the 8-bit paged cache: byte layout and number format shared by
// the kernels that write and read it (contract in include/kda.h).
#pragma once

#include "kda_cache.cuh"

namespace kda {
namespace cache {

// Byte offsets inside a group of 16 tokens (32 D + 16 bytes) of token i's code of channel c.
// The orders are those in which the attention kernel's lanes take the bytes for its matrix
// products (kda_cache_split.cuh): 16 neighbouring channels of a token's K stay together, D / 8
// of its V, so that one token is written without touching another's bytes.
template <int D>
struct Layout8 {
  static constexpr int kGroupBytes = 32 * D + 16;
  static constexpr int kVCodes = 16 * D;
  static constexpr int kScales = 32 * D;  // exponents of K and of V plus 127, a byte each
  static __host__ __device__ constexpr int k_code(int i, int c) {
    return c % (D / 4) / 16 * 1024 + i * 64 + c / (D / 4) * 16 + c % 16;
  }
  static __host__ __device__ constexpr int v_code(int i, int c) {
    return kVCodes + ((i >> 3) * 2 + (i & 1)) * 4 * D + c / (D / 8) * (D / 2) +
           ((i & 7) >> 1) * (D / 8) + c % (D / 8);
  }
};

// Exponents of a block: 448 2^e is the largest magnitude it holds.  With 120 a value next to
// fp32's largest would round up to 2^128.
constexpr int kLeastExponent = -100, kMostExponent = 119, kExponentBias = 127;

// 2^(b - 127) for the exponent byte b of a block that append wrote.
__device__ __forceinline__ float exponent_factor(int b) { return __int_as_float(b << 23); }

// 2^-d as two equal halves, 0 <= d; from 2^-25 on zero.
__device__ __forceinline__ uint32_t half_power(int d) {
  const uint32_t h = d <= 14 ? (uint32_t)(15 - d) << 10 : d <= 24 ? 1u << (24 - d) : 0u;
  return h * 0x10001u;
}

// Two halves as two E4M3 bytes, nearest with ties to even, saturating.
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
// The same of two fp32 values, x in the low byte.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}

// The four codes of a word as two pairs of halves; exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

}  // namespace cache
}  // namespace kda
