// kda_cache_attention.cu -- kda_cache_attention: causal attention of new tokens
// over the 4-bit paged cache.
//
// One warp per (new token, query head): the lanes share the channels, the keys
// are walked one after another with a running maximum and sum.
#include <math.h>

#include "kda_cache.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

using namespace cache;

constexpr int kWarps = 4;

// Channels per lane of one token: a lane's D/32 channels are D/64 code bytes.
template <int D>
__device__ __forceinline__ void load_row(const uint8_t* codes, uint32_t scale, int lane,
                                         float (&x)[D / 32]) {
  uint32_t bits = codes[0];
  if constexpr (D == 128) bits |= (uint32_t)codes[1] << 8;
  uint32_t r[4];
  e2m1x8_to_f16(bits, r);
  const float s = e4m3_to_f32(scale);
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
    x[2 * i] = f.x * s;
    x[2 * i + 1] = f.y * s;
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) rows_kernel(View c, AttentionArgs a) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int h = (int)(w % a.num_heads);
  const int64_t t = w / a.num_heads;
  int lo_b, hi_b;
  for (int64_t b = w; b < a.num_seqs; b += (int64_t)gridDim.x * kWarps)  // every range is checked
    seq_range(a.cu_new, (int)b, a.total_tokens, a.err, lo_b, hi_b);
  if (t >= a.total_tokens || t >= a.cu_new[a.num_seqs]) return;
  int lo = 0, hi = a.num_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_new[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  int bos, eos;
  if (!seq_range(a.cu_new, lo, a.total_tokens, a.err, bos, eos) || t < bos || t >= eos) return;
  const int kv = a.kv_lens[lo];
  if (kv < 0 || kv > (int64_t)a.max_blocks * c.page_size) {
    report_error(a.err, kErrDeviceCheck);
    return;
  }
  const int n = eos - bos;
  const int see = kv - n + (int)(t - bos) + 1;  // keys 0 .. see - 1
  const int kh = h / (a.num_heads / c.kv_heads);
  const T* q = static_cast<const T*>(a.q) + t * a.q_token_stride + h * a.q_head_stride + lane * C;
  const float sc = a.scale * exponent_scale(c.k_exp, kh, 1);
  float qv[C], o[C] = {};
#pragma unroll
  for (int i = 0; i < C; ++i) qv[i] = IO<T>::ld(q + i);
  float top = -INFINITY, sum = 0.f;
  const int32_t* row = a.block_table + (int64_t)lo * a.max_blocks;
  const int ch = lane * C, b = ch / kGroup, in_block = (ch % kGroup) / 2;
  for (int j = 0; j < see; ++j) {
    const int page = row[j / c.page_size];
    if (page < 0 || page >= c.num_pages) {
      report_error(a.err, kErrDeviceCheck);
      continue;
    }
    const int tok = j % c.page_size, i = tok % kGroup;
    const uint8_t* g = group_of<D>(c, page, tok, kh);
    float k[C], v[C];
    load_row<D>(g + Layout<D>::k_codes(i, b) + in_block, g[Layout<D>::k_scale(i, b)], lane, k);
    load_row<D>(g + Layout<D>::v_codes(i, b) + in_block, g[Layout<D>::v_scale(i, b)], lane, v);
    float s = 0.f;
#pragma unroll
    for (int x = 0; x < C; ++x) s = fmaf(qv[x], k[x], s);
    s = warp_sum(s) * sc;
    const float next = fmaxf(top, s);
    const float keep = next == -INFINITY ? 1.f : expf(top - next);
    const float p = next == -INFINITY && !isnan(s) ? 0.f : expf(s - next);  // NaN stays NaN
    sum = fmaf(sum, keep, p);
#pragma unroll
    for (int x = 0; x < C; ++x) o[x] = fmaf(o[x], keep, p * v[x]);
    top = next;
  }
  const float inv = sum == 0.f ? 0.f : exponent_scale(c.v_exp, kh, 1) / sum;
  T* out = static_cast<T*>(a.out) + (t * a.num_heads + h) * D + ch;
#pragma unroll
  for (int x = 0; x < C; ++x) IO<T>::st(out + x, o[x] * inv);
  if (a.lse && lane == 0)
    a.lse[t * a.num_heads + h] = sum == 0.f ? -INFINITY : top + logf(sum);
}

template <typename T, int D>
cudaError_t rows(const View& c, const AttentionArgs& a, cudaStream_t st) {
  const int64_t warps = (int64_t)a.total_tokens * a.num_heads;
  rows_kernel<T, D><<<(unsigned)((warps + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(c, a);
  return cudaGetLastError();
}

}  // namespace

size_t cache_attention_workspace_bytes(const View& c, const AttentionArgs& a) { return 0; }

cudaError_t launch_cache_attention(const View& c, const AttentionArgs& a, cudaStream_t st) {
  if (a.bf16)
    return a.head_dim == 128 ? rows<__nv_bfloat16, 128>(c, a, st)
                             : rows<__nv_bfloat16, 64>(c, a, st);
  return a.head_dim == 128 ? rows<float, 128>(c, a, st) : rows<float, 64>(c, a, st);
}

}  // namespace kda
