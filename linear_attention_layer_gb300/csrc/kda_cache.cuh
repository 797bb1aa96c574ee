// kda_cache.cuh -- the 4-bit paged cache: byte layout and number formats
// shared by the kernels that write and read it (contract in include/kda.h).
#pragma once

#include <cuda_fp16.h>

#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {
namespace cache {

constexpr int kGroup = 16;  // tokens of one layout group, channels of one scale

// Programmatic dependent launch: a kernel lets the next one's CTAs start, which wait here
// until the memory of the one before is complete.
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launches a kernel that waits so: its CTAs may start as soon as the kernel ahead of it in the
// stream has none left to start or run, or has let it (append + read of 256 tokens 12.3 -> 8.8 us,
// attention of 1 x 2048 tokens 13.1 -> 11.4).  The short kernels of these calls do not let the next
// one start earlier: its CTAs then wait in their way (append + read of 256 tokens 11 to 14 us).
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                         A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Byte offsets inside a group of 16 tokens (18 D bytes), for token i and the
// block b of 16 channels.  The orders are those in which the attention
// kernel's lanes take the bytes for its matrix products (kda_cache_attention.cu);
// a block's 8 code bytes stay together, so that one token is written without
// touching another's bytes.
template <int D>
struct Layout {
  static constexpr int kGroupBytes = 18 * D;
  static constexpr int kVCodes = 8 * D;
  static constexpr int kKScales = 16 * D;
  static constexpr int kVScales = 17 * D;
  static constexpr int kPer = D / 64;
  static __host__ __device__ constexpr int k_codes(int i, int b) { return i * (D / 2) + b * 8; }
  static __host__ __device__ constexpr int v_codes(int i, int b) {
    return kVCodes + (i >> 3) * 4 * D + b * 64 + (i & 7) * 8;
  }
  static __host__ __device__ constexpr int k_scale(int i, int b) {
    return kKScales + (i & 7) * (D / 8) + (b / kPer) * (2 * kPer) + (i >> 3) * kPer + b % kPer;
  }
  static __host__ __device__ constexpr int v_scale(int i, int b) {
    return kVScales + b * 16 + ((i & 7) >> 1) * 4 + (i >> 3) * 2 + (i & 1);
  }
};

// 2^e for a head's exponent, held to the documented range.
__device__ __forceinline__ float exponent_scale(const int32_t* e, int head, int sign) {
  if (!e) return 1.f;
  const int x = max(-64, min(64, __ldg(e + head))) * sign;
  return __int_as_float((127 + x) << 23);
}

// ---- formats (conversion instructions of sm_100a and later) ----

// Two E4M3 bytes (low, high) as two halves; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)b));
  return r;
}

// Nearest E4M3 (ties to even, saturating) of a value that is already rounded to odd.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  const uint32_t h = e4m3x2_to_f16x2(b & 0xffu);
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

// The four bytes of a word, each two E2M1 codes, as four pairs of halves; exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Product of two pairs of halves.
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// E2M1 codes of eight values, nearest with ties to even, saturating: one word.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// x / y rounded to odd: truncated, the last bit set when something was cut off.
// Rounding that to fewer bits gives what rounding the exact quotient gives
// (Boldo and Melquiond, "When double rounding is odd", 2005).
__device__ __forceinline__ float div_to_odd(float x, float y) {
  const float q = __fdiv_rz(x, y);
  const bool cut = __fmaf_rn(-q, y, x) != 0.f;
  return __int_as_float(__float_as_int(q) | (cut ? 1 : 0));
}

}  // namespace cache
}  // namespace kda
