// kda_byte_cache_attention.cu -- kda_byte_cache_attention: causal attention over the 8-bit paged cache.
//
// The kernel is that of the 4-bit cache (kda_cache_attention.cu), with 8-bit codes and scales
// that are powers of two of a whole block:
//   - a code becomes a half by one conversion, without a product;
//   - K's power of two 2^e goes into the factor of a group's 16 raw scores;
//   - V's goes into the weights: p 2^(e - E), E the largest exponent that the unit's part has
//     met (o is rescaled when it rises, in the branch that moves the softmax's reference), so
//     that a half holds it and the sums o stay in units of 2^E.  The sum l of weights does not
//     take part in it.
#include "kda_cache_split.cuh"

namespace kda {
namespace {

// Calls f with the variant for the call's types and expected rows per kv head (kda_cache_attention.cu
// has what tiles of 8 and 16 rows are for).  Warps, stages, CTAs a SM by measurement; us of 100
// requests of 256 to 8192 tokens, 8 kv heads, 4 query heads each, one or four new tokens:
//     bf16 128   8 rows   4 x 2 x 3  154   8 x 3 x 1  157   12 x 2 x 1  151
//               16 rows   8 x 3 x 1  171   4 x 2 x 3  256   12 x 2 x 1  254 (these spill)
//     bf16  64   8 rows   8 x 3 x 2   87   4 x 4 x 3   90    4 x 2 x 5  123
//               16 rows   8 x 4 x 1  113   4 x 4 x 3  112    8 x 3 x 2  171
//     fp32 128   8 rows   8 x 3 x 1  153   4 x 2 x 3  184
//               16 rows   8 x 2 x 1  268   4 x 2 x 2  266    4 x 3 x 1  332
//     fp32  64   8 rows   8 x 3 x 2  119   4 x 4 x 3  105    4 x 2 x 4  113
//               16 rows   8 x 4 x 1  158   4 x 3 x 3  172    8 x 2 x 2  214
// Few units, fewer than half the SMs, are each cut over many CTAs, whose parts a second kernel joins:
// one CTA of 8 warps leaves it a third of the parts that three of 4 do (one request
// of 2048 tokens 11.5 us for 12.1, of 131072 on one kv head 20 for 31; 256 requests 349 for 335).
template <typename F>
auto dispatch(const View& c, const AttentionArgs& a, F&& f) {
  const bool few = (int64_t)a.max_new * (a.num_heads / c.kv_heads) <= 8;
  const bool few_units = (int64_t)a.num_seqs * c.kv_heads <= 64;
  if (a.bf16) {
    using T = __nv_bfloat16;
    if (a.head_dim == 128) {
      if (few && few_units) return f(Split<8, T, 128, 1, 8, 3, 1>{});
      return few ? f(Split<8, T, 128, 1, 4, 2, 3>{}) : f(Split<8, T, 128, 2, 8, 3, 1>{});
    }
    return few ? f(Split<8, T, 64, 1, 8, 3, 2>{}) : f(Split<8, T, 64, 2, 8, 4, 1>{});
  }
  if (a.head_dim == 128)
    return few ? f(Split<8, float, 128, 1, 8, 3, 1>{}) : f(Split<8, float, 128, 2, 8, 2, 1>{});
  return few ? f(Split<8, float, 64, 1, 4, 4, 3>{}) : f(Split<8, float, 64, 2, 8, 4, 1>{});
}

}  // namespace

size_t byte_cache_attention_workspace_bytes(const View& c, const AttentionArgs& a) {
  const size_t split = dispatch(c, a, [&](auto v) { return decltype(v)::workspace(); });
  return std::max(split, cache_chunk_wanted(c, a) ? cache_chunk_workspace_bytes(c, a) : 0);
}

cudaError_t launch_byte_cache_attention(const View& c, const AttentionArgs& args, cudaStream_t st) {
  AttentionArgs a = args;
  if (take_injected_timeout()) {
    a.wait_cycles = kInjectedWaitCycles;
    a.withheld = 1;
  }
  const bool chunk = cache_chunk_wanted(c, a);
  // without the second kernel the first takes every request, whatever max_new said
  const RowRange few{0, chunk ? kSplitRows : INT64_MAX}, many{kSplitRows, INT64_MAX};
  const cudaError_t e =
      dispatch(c, a, [&](auto v) { return decltype(v)::launch(c, a, few, st); });
  if (e != cudaSuccess || !chunk) return e;
  return launch_cache_chunk(8, c, a, many, st);
}

}  // namespace kda
