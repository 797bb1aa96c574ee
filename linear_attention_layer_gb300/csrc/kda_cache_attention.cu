// kda_cache_attention.cu -- kda_cache_attention for few rows per kv head (decode
// steps, drafted windows): causal attention over the 4-bit paged cache.
//
// Mathematics.  A unit is a request, a kv head and up to 8 NT of the rows (new
// token x query head) that share it.  Its keys are walked in tiles of 32 with the
// usual running maximum m and sum l of a softmax,
//     p_j = 2^(s_j - m),  l = sum p_j,  o = sum p_j v_j,   s = scale log2(e) q . k,
// partial (m, l, o) of parts of a unit's keys being joined by rescaling to the
// common maximum.  m is set 7 below the largest score and moved (and o, l rescaled)
// only when some score passes it by more than 15, so p <= 2^15: any reference gives
// the same quotient o / l.
//
// Products.  mma.sync m16n8k16 on halves with the cache as the 16-row operand:
// scores^T = K q^T (16 keys x 8 rows), o^T += V^T p^T (16 channels x 8 rows).
// The call is bound by HBM -- 9/8 byte a key channel pair for 4 G flops of a group
// of G query heads -- so what counts is the issue slots it takes to turn the codes
// into operands.  A lane's A fragment of K^T or V takes its codes straight from
// the bytes of a group (the layout in include/kda.h is the fragments' order), a
// conversion instruction makes two halves of each byte, and one half2 product
// applies the E4M3 scale: code x scale has 6 significant bits, exact in a half.
// q is scaled by a power of two per row (row_scale) and rounded to halves: bf16
// fits exactly, fp32 goes in as two halves.  p is rounded to a half (2^-11, below
// the output's own 2^-8), for fp32 outputs to two, the second held 2^11 times
// larger.  All sums are fp32.
//
// Work split.  The tiles of all units in one sequence are cut evenly over the
// warps of the whole GPU, wherever that falls in a unit: lengths of any mix fill
// the machine, one long request included.  A warp streams its tiles through its
// own ring of bulk copies (no CTA-wide synchronisation while it runs).  Parts of a
// unit are joined inside their CTA through the workspace, and across CTAs by a
// second kernel.
//
// Measured (GB300; 32 query heads on 8 kv heads of 128, bf16).  256 requests of 256 to
// 8192 tokens: 257 to 260 us for 1.27 GB, 0.73 of the measured HBM rate; 1 x 262144 tokens 68 us
// (0.66), 1 x 2048 tokens 12.5 us.  What bounds it: the copies alone took 217 us, the
// arithmetic alone 267 (the whole 262 then).  A tile is 560 warp instructions and about
// 1000 cycles of a quadrant: 128 conversions and 100 other integer instructions of 2 cycles,
// 128 half2 products of 2 beside them, and 32 products of 8 that do not run beside either.
#include "kda_cache_split.cuh"

namespace kda {
namespace {

using namespace cache;

// 12 warps of 160 registers a SM (three CTAs of four): the decode step above takes 257 us; 16
// warps of 128 registers 278 to 281 (they spill), 8 warps 375.  Values of one tile and scores
// of the next are interleaved in the source; without that 16 warps were as fast, not faster.
//
// Calls f with the variant for the call's types and expected rows per kv head: tiles of 8
// rows where those are enough, else of 16, more rows taking several passes over the keys
// (the second finds them in L2).  67 windows of 1 to 5 tokens, 8 query heads on a kv head,
// 128 channels: 8 rows 191 us, 16 rows 172, 24 rows 186, 32 rows 240 -- the larger tiles'
// sums leave registers for too few warps.
template <typename F>
auto dispatch(const View& c, const AttentionArgs& a, F&& f) {
  const bool few = (int64_t)a.max_new * (a.num_heads / c.kv_heads) <= 8;
  if (a.bf16) {
    using T = __nv_bfloat16;
    if (a.head_dim == 128)
      return few ? f(Split<4, T, 128, 1, 4, 3, 3>{}) : f(Split<4, T, 128, 2, 8, 4, 1>{});
    return few ? f(Split<4, T, 64, 1, 8, 4, 2>{}) : f(Split<4, T, 64, 2, 8, 4, 1>{});
  }
  if (a.head_dim == 128)
    return few ? f(Split<4, float, 128, 1, 8, 4, 1>{}) : f(Split<4, float, 128, 2, 8, 4, 1>{});
  return few ? f(Split<4, float, 64, 1, 8, 4, 2>{}) : f(Split<4, float, 64, 2, 8, 4, 1>{});
}

}  // namespace

size_t cache_attention_workspace_bytes(const View& c, const AttentionArgs& a) {
  const size_t split = dispatch(c, a, [&](auto v) { return decltype(v)::workspace(); });
  return std::max(split, cache_chunk_wanted(c, a) ? cache_chunk_workspace_bytes(c, a) : 0);
}

bool cache_chunk_wanted(const View& c, const AttentionArgs& a) {
  return a.bf16 && (int64_t)a.max_new * (a.num_heads / c.kv_heads) > kSplitRows;
}

cudaError_t launch_cache_attention(const View& c, const AttentionArgs& args, cudaStream_t st) {
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
  return launch_cache_chunk(4, c, a, many, st);
}

}  // namespace kda
