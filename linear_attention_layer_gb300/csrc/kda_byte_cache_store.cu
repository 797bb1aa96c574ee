// kda_byte_cache_store.cu -- kda_byte_cache_append and kda_byte_cache_read: keys and values between
// their own type and the cache's 8-bit blocks.
//
// A block is 16 tokens of one head, K or V.  Its exponent e is the least with max |x| <=
// 448 2^e over the tokens appended to it, its codes are e4m3(x 2^-e): the product with a power
// of two is exact, so a value is rounded once.  New tokens that raise the exponent of a block
// begun earlier take its codes along, e4m3(c 2^(e - e')), which is exact but for codes that run
// into E4M3's smallest numbers.
//
// One warp takes the new tokens of one block, a run of neighbours in the batch, and keeps
// them in registers: 16 bytes of bf16 a lane and token, the largest magnitude by one redux.
// Nothing is shared between warps.  What bounds it is HBM as long as enough warps have their
// loads under way: with bf16 28 a SM of 72 registers (with 128 channels 12 to 36 bytes of them
// spilled; CTAs of 256 threads of 140 registers left 8 warps, 672 us for the prompts below), with
// fp32 16 of up to 127.
//
// Measured (GB300; bf16, 8 heads of 128; rates are the call's bytes over its time, of the measured HBM
// rate): prompts of 270336 tokens, 1.66 GB, appended in 293 us (0.84), read back in 254 us (0.96; the
// kernel keeps DRAM 82% busy); 8000 tokens 9.2 us; a decode step of 256 tokens 6.3 us into a cache that
// it meets for the first time, 4.1 when the same tokens are appended again (no exponent rises, its
// lines are in L2), of 4096 58 and 26.  fp32: 100000 tokens 163 us (0.93), with heads of 64 103 (0.73),
// read back in 199 (0.76) and 101 (0.75); 4096 tokens 81 and 35.
#include <algorithm>

#include "kda_byte_cache.cuh"
#include "kda_launch.h"
#include "tc_ptx.cuh"

namespace kda {
namespace {

using namespace cache;

constexpr int kThreads = 128;
// Of a CTA that reads back (270336 tokens x 8 x 128 of bf16: 256 us, with 256 threads 280; 100000 of
// fp32 210 and 202).
template <typename T>
constexpr int kReadThreads = sizeof(T) == 2 ? 128 : 256;

struct Source {
  const void* p;
  int token_stride, head_stride;  // elements
};

// 8 neighbouring values of a row as they lie in memory.  VEC: 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ void fetch8(const T* p, uint32_t (&w)[2 * sizeof(T)]) {
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
  } else if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = reinterpret_cast<const uint16_t*>(p)[2 * i] |
             (uint32_t)reinterpret_cast<const uint16_t*>(p)[2 * i + 1] << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}

// Value i of them.
template <typename T>
__device__ __forceinline__ float value8(const uint32_t (&w)[2 * sizeof(T)], int i) {
  if constexpr (sizeof(T) == 4)
    return __uint_as_float(w[i]);
  else
    return i & 1 ? tc::bf16_hi(w[i / 2]) : tc::bf16_lo(w[i / 2]);
}

// Bits of the largest magnitude as fp32 (magnitudes order like their bits).
template <typename T>
__device__ __forceinline__ uint32_t top8(const uint32_t (&w)[2 * sizeof(T)]) {
  uint32_t top = 0;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, w[i] & 0x7fffffffu);
    return top;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
    return max(top << 16, top & 0xffff0000u);
  }
}

// The least e with x <= 448 2^e, in the range of exponents; x given by its bits and finite:
// 448 = 1.75 * 2^8.
__device__ __forceinline__ int exponent_of(uint32_t bits) {
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(kLeastExponent, min(e, kMostExponent));
}

// First byte of a token's 8 channels from c on, which are one run.
template <int D, bool V>
__device__ __forceinline__ int place8(int i, int c) {
  return V ? Layout8<D>::v_code(i, c) : Layout8<D>::k_code(i, c);
}

// Magnitude bits of value i, 0 where it is not finite.
template <typename T>
__device__ __forceinline__ uint32_t finite8(const uint32_t (&w)[2 * sizeof(T)], int i) {
  const uint32_t m = __float_as_uint(value8<T>(w, i)) & 0x7fffffffu;
  return m < 0x7f800000u ? m : 0u;
}

// Zero in place of the bytes of a word that are codes of NaN (0x7f and 0xff).
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
  return w & ~__vcmpeq4(w | 0x80808080u, 0xffffffffu);
}

// How a warp's lanes share the tokens of a run: 8 channels each, AT_ONCE tokens a step.
template <int D>
struct Lanes {
  static constexpr int PER_TOKEN = D / 8, AT_ONCE = 32 / PER_TOKEN, STEPS = kGroup / AT_ONCE;
  int c, t;
  __device__ __forceinline__ Lanes() {
    const int lane = threadIdx.x & 31;
    c = lane % PER_TOKEN * 8;
    t = lane / PER_TOKEN;
  }
};

// A run of n tokens of the batch, which fill places of one block; lane k < n has the place of
// the k-th of them.  p: the lane's channels of its first token, whose values (those of the next as
// well, where a step takes two or four) are in `first` if `have`.  leave_out: nothing is written.
// SHORT: runs of one step go a way of their own, which saves decode steps of thousands a quarter and
// costs prompts 2% -- but for fp32 with 128 channels, where the compiler then finds room for what it
// spills otherwise (100000 tokens 163 us for 183).  All lanes of the warp.
template <typename T, int D, bool VEC, bool V, bool SHORT>
__device__ __forceinline__ void append_run(uint8_t* group, const T* p, int token_stride, int n,
                                           int place, const uint32_t (&first)[2 * sizeof(T)],
                                           bool have, bool leave_out, bool& not_finite) {
  using W = Lanes<D>;
  const W at;
  const int lane = threadIdx.x & 31;
  uint32_t w[W::STEPS][2 * sizeof(T)];
#pragma unroll
  for (int s = 0; s < W::STEPS; ++s) {
#pragma unroll
    for (int i = 0; i < 2 * (int)sizeof(T); ++i) w[s][i] = 0;
    if (s * W::AT_ONCE + at.t < n) {
      if (s == 0 && have) {
#pragma unroll
        for (int i = 0; i < 2 * (int)sizeof(T); ++i) w[0][i] = first[i];
      } else {
        fetch8<T, VEC>(p, w[s]);
      }
    }
    p += (int64_t)W::AT_ONCE * token_stride;
  }
  uint8_t* const exp_at = group + Layout8<D>::kScales + (V ? 1 : 0);
  // places that the run fills, and whether it begins the block anew
  const uint32_t filled = __reduce_or_sync(0xffffffffu, lane < n ? 1u << place : 0u);
  const bool fresh = filled & 1;
  // (a byte that append did not write is held to the range of those it does)
  const int before = fresh ? kLeastExponent
                           : max(kLeastExponent, min((int)*exp_at - kExponentBias, kMostExponent));
  const bool one_step = SHORT && n <= W::AT_ONCE;  // all lanes
  uint32_t top = top8<T>(w[0]);
  if (!one_step) {
#pragma unroll
    for (int s = 1; s < W::STEPS; ++s) top = max(top, top8<T>(w[s]));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const bool odd = top >= 0x7f800000u;  // infinities do not count, NaN becomes zero
  if (odd) {
    not_finite = true;
    top = 0;
#pragma unroll
    for (int s = 0; s < W::STEPS; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, finite8<T>(w[s], i));
    top = __reduce_max_sync(0xffffffffu, top);
  }
  const int e = max(exponent_of(top), before);
  if (leave_out) return;  // asked only here, behind the loads
  if (!fresh && e > before) {
    // pieces of 8 codes, each of one token: 2 D of them, four of a lane asked for at once
    const uint32_t f = half_power(e - before);
#pragma unroll 1
    for (int q0 = 0; q0 < D / 16; q0 += 4) {
      uint2 old[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        old[q] = *reinterpret_cast<const uint2*>(
            group + place8<D, V>((q0 + q) * W::AT_ONCE + at.t, at.c));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = (q0 + q) * W::AT_ONCE + at.t;
        if (filled >> i & 1) continue;
        uint32_t h[4];
        e4m3x4_to_f16(old[q].x, h[0], h[1]);
        e4m3x4_to_f16(old[q].y, h[2], h[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = f16x2_to_e4m3x2(mul_f16x2(h[j], f));
        *reinterpret_cast<uint2*>(group + place8<D, V>(i, at.c)) =
            make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
      }
    }
  }
  const float down = __int_as_float((127 - e) << 23);
  auto put = [&](int s) {
    const int i = __shfl_sync(0xffffffffu, place, (s * W::AT_ONCE + at.t) & 31);
    if (s * W::AT_ONCE + at.t < n) {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[j] = f32x2_to_e4m3x2(value8<T>(w[s], 2 * j) * down, value8<T>(w[s], 2 * j + 1) * down);
      uint2 codes = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
      if (odd) codes = make_uint2(without_nan(codes.x), without_nan(codes.y));
      *reinterpret_cast<uint2*>(group + place8<D, V>(i, at.c)) = codes;
    }
  };
  put(0);
  if (!one_step) {
#pragma unroll
    for (int s = 1; s < W::STEPS; ++s) put(s);
  }
  if (lane == 0) *exp_at = (uint8_t)(e + kExponentBias);
}

// A run of a block that one of the 16 tokens before the run is of already is left out: two warps
// would read and write that block's exponent and codes.  (A block that the batch comes back to
// further on is not found out.)  `back`: lane l has the block of the window's token l - 16.
//
// Whether that is so of the run of block b that starts at the window's token i: a vote for each run.
__device__ __forceinline__ bool second_run(int back, int b, int i) {
  return (__ballot_sync(0xffffffffu, back == b) & 0xffffu << i) != 0;
}
// Bit i for each such token i: 16 shuffles a window (a match over the warp instead: a decode step of
// 256 tokens 4.7 us for 4.4).  Where a warp has several short runs one after the other, the votes
// cost more (4096 fp32 tokens 44 us for 34), elsewhere less (256 tokens 4.1 us).
__device__ __forceinline__ uint32_t second_runs(int back) {
  bool met = false;
#pragma unroll
  for (int d = 2; d <= kGroup; ++d) met |= __shfl_up_sync(0xffffffffu, back, d) == back;
  const bool starts = __shfl_up_sync(0xffffffffu, back, 1) != back;
  return __ballot_sync(0xffffffffu, met && starts && back >= 0) >> kGroup;
}

// How the runs that start among 16 tokens of the batch, a window, are dealt out with the heads to
// `share` warps: a warp a head, what a prompt's one or two runs want; more warps; or one for each
// head and token, what a small decode step wants.
enum Deal { kByHead, kMore, kByToken };

template <typename T, int D, bool VEC, bool V, Deal DEAL>
__device__ __forceinline__ void append_window(const View& c, int tokens, int share,
                                              const Source& src, const int64_t* slots, int* err) {
  const int lane = threadIdx.x & 31;
  constexpr bool ALONE = DEAL != kByHead;
  const uint32_t unit = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);  // (host: 32 bits)
  const uint32_t window = unit / (uint32_t)share;
  const int mine = (int)(unit - window * (uint32_t)share);
  const int64_t start = (int64_t)window * kGroup;
  if (start >= tokens) return;
  const Lanes<D> at;
  const T* base = static_cast<const T*>(src.p);
  // lane l: the slot of token start - 1 + l, as far as a run of the window may reach
  const int64_t token = start - 1 + lane;
  const int64_t token_back = token - (kGroup - 1);
  int64_t slot = -1, slot_back = -1;
  if (token >= 0 && token < tokens) slot = slots[token];
  if (token_back >= 0 && token_back < tokens) slot_back = slots[token_back];
  // Values are asked for before the slots say which they are.  Many warps to a window: the token
  // that is this warp's if each is a run of its own; else all of the window's, into L2.
  uint32_t first[2 * sizeof(T)] = {};
  const int guess = (uint32_t)mine / (uint32_t)c.kv_heads;
  if constexpr (ALONE) {
    if (start + guess + at.t < tokens)
      fetch8<T, VEC>(base + (start + guess + at.t) * src.token_stride +
                         (int64_t)(mine - guess * c.kv_heads) * src.head_stride + at.c,
                     first);
  } else {
    constexpr int kLines = D * (int)sizeof(T) / 128;
#pragma unroll
    for (int i = lane; i < kGroup * kLines; i += 32)
      if (start + i / kLines < tokens)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            base + (start + i / kLines) * src.token_stride + (int64_t)mine * src.head_stride +
            i % kLines * (128 / (int)sizeof(T))));
  }
  const bool there = slot >= 0 && slot < (int64_t)c.num_pages * c.page_size;
  const bool counts = lane >= 1 && lane <= kGroup;
  if (!there && slot != -1 && counts && mine == 0 && !V) report_error(err, kErrDeviceCheck);
  const int block = there ? (int)(slot / kGroup) : -1;  // fewer than 2^27
  const int prev = __shfl_up_sync(0xffffffffu, block, 1);
  const bool goes_on = there && lane > 0 && prev == block;
  const uint32_t on = __ballot_sync(0xffffffffu, goes_on);
  const bool there_back = slot_back >= 0 && slot_back < (int64_t)c.num_pages * c.page_size;
  const int back = there_back ? (int)(slot_back / kGroup) : -1;
  uint32_t second = 0;
  if constexpr (DEAL == kMore) second = second_runs(back);
  const bool starts_here = counts && there && !goes_on && !(second << 1 >> lane & 1);
  const uint32_t starts = __ballot_sync(0xffffffffu, starts_here);
  const int rank = __popc(starts & ((1u << lane) - 1));  // runs before the lane's
  const int tasks = __popc(starts) * c.kv_heads;
  bool not_finite = false, met_again = second != 0;
  const int groups = c.page_size / kGroup;
  for (int task = mine; task < tasks; task += share) {
    const int run = task / c.kv_heads, head = task - run * c.kv_heads;
    const int l = __ffs(__ballot_sync(0xffffffffu, starts_here && rank == run)) - 1;
    // tokens l, l + 1, ... as long as they go on
    const uint32_t after = ~(on >> (l + 1));
    const int n = min(after ? __ffs(after) : 32, kGroup);
    const int place = __shfl_sync(0xffffffffu, (int)(slot & (kGroup - 1)), (l + lane) & 31);
    const int b = __shfl_sync(0xffffffffu, block, l);
    const bool again = DEAL != kMore && second_run(back, b, l - 1);
    met_again |= again;
    const int page = b / groups;
    uint8_t* group =
        c.pages + (((int64_t)page * c.kv_heads + head) * groups + (b - page * groups)) *
                      Layout8<D>::kGroupBytes;
    const T* from = base + (start + l - 1 + at.t) * src.token_stride +
                    (int64_t)head * src.head_stride + at.c;
    append_run<T, D, VEC, V, ALONE || (sizeof(T) == 4 && D == 128)>(
        group, from, src.token_stride, n, place, first, ALONE && task == mine && l - 1 == guess,
        again, not_finite);
  }
  if ((not_finite || met_again) && lane == 0) report_error(err, kErrDeviceCheck);
}

template <typename T, int D, bool VEC, Deal DEAL>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 7 : 4)
    append_kernel(View c, int tokens, int share, Source k, Source v,
                  const int64_t* slots, int* err) {
  wait_for_previous();
  if (blockIdx.y)
    append_window<T, D, VEC, true, DEAL>(c, tokens, share, v, slots, err);
  else
    append_window<T, D, VEC, false, DEAL>(c, tokens, share, k, slots, err);
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&x)[16]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __stcs(reinterpret_cast<float4*>(p) + i,
             make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __stcs(reinterpret_cast<uint4*>(p) + i,
             make_uint4(tc::pack_bf16(x[8 * i], x[8 * i + 1]),
                        tc::pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                        tc::pack_bf16(x[8 * i + 4], x[8 * i + 5]),
                        tc::pack_bf16(x[8 * i + 6], x[8 * i + 7])));
  }
}

// A thread takes 16 channels of a token and every so many heads, of K or V.
template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads<T>)
    read_kernel(View c, int tokens, const int64_t* slots, T* k, T* v, int* err) {
  wait_for_previous();
  constexpr int PIECES = D / 16;
  const int piece = threadIdx.x % PIECES;
  const int first = threadIdx.x / (8 * PIECES), step = blockDim.x / (8 * PIECES);
  const int64_t token = (int64_t)blockIdx.x * 8 + threadIdx.x / PIECES % 8;
  if (token >= tokens) return;
  const int64_t slot = slots[token];
  const bool there = slot >= 0 && slot < (int64_t)c.num_pages * c.page_size;
  if (!there && slot != -1) report_error(err, kErrDeviceCheck);
  const bool is_v = blockIdx.y;
  const int groups = c.page_size / kGroup;
  const int64_t head_bytes = (int64_t)groups * Layout8<D>::kGroupBytes;
  const uint8_t* g = c.pages;
  int at = 0;
  if (there) {
    const int page = (int)(slot / c.page_size), tok = (int)(slot % c.page_size), i = tok % kGroup;
    g += (int64_t)page * c.kv_heads * head_bytes + tok / kGroup * Layout8<D>::kGroupBytes;
    at = is_v ? Layout8<D>::v_code(i, piece * 16) : Layout8<D>::k_code(i, piece * 16);
  }
  T* out = (is_v ? v : k) + token * c.kv_heads * D + piece * 16;
#pragma unroll 2
  for (int h = first; h < c.kv_heads; h += step) {
    float x[16] = {};
    if (there) {
      const uint8_t* p = g + h * head_bytes;
      uint4 w;
      if (D == 128 || !is_v) {
        w = *reinterpret_cast<const uint4*>(p + at);
      } else {  // V of 64 channels: 8 to a run
        const uint2 a = *reinterpret_cast<const uint2*>(p + at);
        const uint2 b = *reinterpret_cast<const uint2*>(p + at + D / 2);
        w = make_uint4(a.x, a.y, b.x, b.y);
      }
      const float f = exponent_factor(p[Layout8<D>::kScales + (is_v ? 1 : 0)]);
      const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t lo, hi;
        e4m3x4_to_f16(words[j], lo, hi);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        x[4 * j] = a.x * f, x[4 * j + 1] = a.y * f;
        x[4 * j + 2] = b.x * f, x[4 * j + 3] = b.y * f;
      }
    }
    store16(out + (int64_t)h * D, x);
  }
}

// Warps of a window: one a head, what a prompt has work for, or more while that leaves the GPU
// short of kWarps -- up to one a head and token, what a decode step has work for.
constexpr int64_t kWarps = 8192;

template <typename T, int D>
cudaError_t append(const CacheArgs& a, cudaStream_t st) {
  const Source k{a.k, (int)a.strides[0], (int)a.strides[1]},
      v{a.v, (int)a.strides[2], (int)a.strides[3]};
  const int el = 16 / sizeof(T);
  bool vec = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15) == 0;
  for (int64_t s : a.strides) vec = vec && s % el == 0;
  const int64_t windows = ((int64_t)a.tokens + kGroup - 1) / kGroup, heads = a.view.kv_heads;
  const int64_t share = std::max(heads, std::min(kGroup * heads, kWarps / 2 / windows));
  const int64_t ctas = (windows * share * 32 + kThreads - 1) / kThreads;
  if (ctas > INT32_MAX / (kThreads / 32)) return cudaErrorInvalidConfiguration;
  auto pick = [&](auto* by_head, auto* more, auto* by_token) {
    return share == heads ? by_head : share < kGroup * heads ? more : by_token;
  };
  auto* kernel =
      vec ? pick(append_kernel<T, D, true, kByHead>, append_kernel<T, D, true, kMore>,
                 append_kernel<T, D, true, kByToken>)
          : pick(append_kernel<T, D, false, kByHead>, append_kernel<T, D, false, kMore>,
                 append_kernel<T, D, false, kByToken>);
  return launch_after(kernel, dim3((unsigned)ctas, 2), kThreads, 0, st, a.view, a.tokens, (int)share,
                      k, v, a.slots, a.err);
}

template <typename T, int D>
cudaError_t read(const CacheArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.tokens + 7ll) / 8), 2);
  const int per_head = 8 * (D / 16);
  const int threads = per_head * std::min(a.view.kv_heads, kReadThreads<T> / per_head);
  return launch_after(read_kernel<T, D>, grid, threads, 0, st, a.view, a.tokens, a.slots,
                      static_cast<T*>(a.k_out), static_cast<T*>(a.v_out), a.err);
}

}  // namespace

cudaError_t launch_byte_cache_append(const CacheArgs& a, cudaStream_t st) {
  if (a.bf16)
    return a.head_dim == 128 ? append<__nv_bfloat16, 128>(a, st) : append<__nv_bfloat16, 64>(a, st);
  return a.head_dim == 128 ? append<float, 128>(a, st) : append<float, 64>(a, st);
}

cudaError_t launch_byte_cache_read(const CacheArgs& a, cudaStream_t st) {
  if (a.bf16)
    return a.head_dim == 128 ? read<__nv_bfloat16, 128>(a, st) : read<__nv_bfloat16, 64>(a, st);
  return a.head_dim == 128 ? read<float, 128>(a, st) : read<float, 64>(a, st);
}

}  // namespace kda
