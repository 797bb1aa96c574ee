// kda_cache_api.cu -- the C ABI of the 4-bit paged cache: argument validation
// and dispatch (contract in include/kda.h).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kda_cache.cuh"
#include "kda_launch.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

kda_status_t check_cache(const kda_cache_t* c) {
  if (!c || c->num_pages < 0 || c->page_size <= 0 || c->num_kv_heads <= 0)
    return KDA_ERR_INVALID_ARGUMENT;
  if (c->page_size % 16 != 0 || c->page_size > 4096) return KDA_ERR_INVALID_ARGUMENT;
  if (c->head_dim != 64 && c->head_dim != 128) return KDA_ERR_UNSUPPORTED;
  if (c->num_kv_heads > 4096) return KDA_ERR_UNSUPPORTED;
  if ((int64_t)c->num_pages * c->page_size > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if ((c->num_pages > 0 && !c->pages) || !aligned(c->pages, 16)) return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned(c->k_exponent, 4) || !aligned(c->v_exponent, 4)) return KDA_ERR_INVALID_ARGUMENT;
  return KDA_OK;
}

kda::cache::View view_of(const kda_cache_t* c) {
  kda::cache::View v;
  v.pages = static_cast<uint8_t*>(c->pages);
  v.num_pages = c->num_pages;
  v.page_size = c->page_size;
  v.kv_heads = c->num_kv_heads;
  v.k_exp = c->k_exponent;
  v.v_exp = c->v_exponent;
  return v;
}

bool known_dtype(int32_t t) { return t == KDA_F32 || t == KDA_BF16; }

kda_status_t check_attention(const kda_cache_t* cache, const kda_attention_t* d) {
  const kda_status_t s = check_cache(cache);
  if (s != KDA_OK) return s;
  if (!d || d->num_seqs < 0 || d->total_tokens < 0 || d->num_heads <= 0 || d->max_new < 1 ||
      d->max_blocks < 0 || !known_dtype(d->io_dtype) || !isfinite(d->scale))
    return KDA_ERR_INVALID_ARGUMENT;
  if (d->num_heads % cache->num_kv_heads != 0) return KDA_ERR_INVALID_ARGUMENT;
  if ((int64_t)d->total_tokens * (d->num_heads / cache->num_kv_heads) > INT32_MAX)
    return KDA_ERR_UNSUPPORTED;  // rows of one kv head
  if ((d->q_strides[0] == 0) != (d->q_strides[1] == 0)) return KDA_ERR_INVALID_ARGUMENT;
  return KDA_OK;
}

void fill_attention(const kda_cache_t* cache, const kda_attention_t* d, kda::AttentionArgs& a) {
  a.num_seqs = d->num_seqs;
  a.total_tokens = d->total_tokens;
  a.num_heads = d->num_heads;
  a.head_dim = cache->head_dim;
  a.max_new = d->max_new;
  a.max_blocks = d->max_blocks;
  a.bf16 = d->io_dtype == KDA_BF16;
  a.scale = d->scale;
  const bool packed = d->q_strides[0] == 0;
  a.q_token_stride = packed ? (int64_t)d->num_heads * cache->head_dim : d->q_strides[0];
  a.q_head_stride = packed ? cache->head_dim : d->q_strides[1];
}

kda_status_t status_of(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

extern "C" {

kda_status_t kda_cache_tables(int32_t page_size, int32_t num_seqs, int32_t max_blocks,
                              int32_t max_tokens, int32_t ring_size, const int32_t* held_lens,
                              const int32_t* seq_lens, const int32_t* new_lens,
                              int32_t* block_table, int32_t* free_pages,
                              const int64_t* free_range, int64_t* free_range_out,
                              int32_t* kv_lens, int32_t* cu_new, int64_t* slots,
                              kda_stream_t stream) {
  if (page_size <= 0 || page_size % 16 != 0 || page_size > 4096) return KDA_ERR_INVALID_ARGUMENT;
  if (num_seqs < 0 || max_blocks < 0 || max_tokens < 0 || ring_size < 1)
    return KDA_ERR_INVALID_ARGUMENT;
  if ((int64_t)num_seqs * max_blocks > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if (!cu_new || !free_range || !free_range_out || !free_pages) return KDA_ERR_INVALID_ARGUMENT;
  if (num_seqs > 0 && (!held_lens || !seq_lens || !new_lens || !kv_lens))
    return KDA_ERR_INVALID_ARGUMENT;
  if (num_seqs > 0 && max_blocks > 0 && !block_table) return KDA_ERR_INVALID_ARGUMENT;
  if (max_tokens > 0 && !slots) return KDA_ERR_INVALID_ARGUMENT;
  const void* words[] = {held_lens, seq_lens, new_lens, block_table, free_pages, kv_lens, cu_new};
  const void* longs[] = {free_range, free_range_out, slots};
  for (const void* p : words)
    if (!aligned(p, 4)) return KDA_ERR_INVALID_ARGUMENT;
  for (const void* p : longs)
    if (!aligned(p, 8)) return KDA_ERR_INVALID_ARGUMENT;
  const void* in[] = {held_lens, seq_lens, new_lens};
  const void* out[] = {cu_new, slots, block_table, free_pages, free_range_out};
  for (const void* o : out)
    for (const void* i : in)
      if (o && o == i) return KDA_ERR_INVALID_ARGUMENT;
  if (kv_lens && (kv_lens == new_lens || kv_lens == cu_new || kv_lens == block_table ||
                  kv_lens == free_pages))
    return KDA_ERR_INVALID_ARGUMENT;
  kda::TableArgs a;
  a.page_size = page_size;
  a.num_seqs = num_seqs;
  a.max_blocks = max_blocks;
  a.max_tokens = max_tokens;
  a.ring_size = ring_size;
  a.held_lens = held_lens;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.free_range = free_range;
  a.free_range_out = free_range_out;
  a.kv_lens = kv_lens;
  a.cu_new = cu_new;
  a.slots = slots;
  a.err = kda::device_error();
  if (!a.err) return KDA_ERR_CUDA;
  return status_of(kda::launch_cache_tables(a, (cudaStream_t)stream));
}

kda_status_t kda_cache_append(const kda_cache_t* cache, int32_t io_dtype, int32_t num_tokens,
                              const void* k, const void* v, const int64_t* strides,
                              const int64_t* slots, kda_stream_t stream) {
  const kda_status_t s = check_cache(cache);
  if (s != KDA_OK) return s;
  if (!known_dtype(io_dtype) || num_tokens < 0) return KDA_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return KDA_OK;
  const uintptr_t size = io_dtype == KDA_BF16 ? 2 : 4;
  if (!k || !v || !slots || !aligned(k, size) || !aligned(v, size) || !aligned(slots, 8))
    return KDA_ERR_INVALID_ARGUMENT;
  kda::CacheArgs a;
  a.view = view_of(cache);
  a.head_dim = cache->head_dim;
  a.bf16 = io_dtype == KDA_BF16;
  a.tokens = num_tokens;
  a.k = k;
  a.v = v;
  a.slots = slots;
  for (int i = 0; i < 4; ++i)
    a.strides[i] = strides ? strides[i]
                   : i % 2 ? (int64_t)cache->head_dim
                           : (int64_t)cache->head_dim * cache->num_kv_heads;
  for (int64_t x : a.strides)
    if (x > INT32_MAX || x < INT32_MIN) return KDA_ERR_UNSUPPORTED;
  a.err = kda::device_error();
  if (!a.err) return KDA_ERR_CUDA;
  return status_of(kda::launch_cache_append(a, (cudaStream_t)stream));
}

kda_status_t kda_cache_read(const kda_cache_t* cache, int32_t io_dtype, int32_t num_tokens,
                            const int64_t* slots, void* k, void* v, kda_stream_t stream) {
  const kda_status_t s = check_cache(cache);
  if (s != KDA_OK) return s;
  if (!known_dtype(io_dtype) || num_tokens < 0) return KDA_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return KDA_OK;
  if (!k || !v || !slots || k == v || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
    return KDA_ERR_INVALID_ARGUMENT;
  kda::CacheArgs a;
  a.view = view_of(cache);
  a.head_dim = cache->head_dim;
  a.bf16 = io_dtype == KDA_BF16;
  a.tokens = num_tokens;
  a.k_out = k;
  a.v_out = v;
  a.slots = slots;
  a.err = kda::device_error();
  if (!a.err) return KDA_ERR_CUDA;
  return status_of(kda::launch_cache_read(a, (cudaStream_t)stream));
}

kda_status_t kda_cache_attention_workspace_size(const kda_cache_t* cache,
                                                const kda_attention_t* desc, size_t* bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARGUMENT;
  const kda_status_t s = check_attention(cache, desc);
  if (s != KDA_OK) return s;
  kda::AttentionArgs a;
  fill_attention(cache, desc, a);
  *bytes = kda::cache_attention_workspace_bytes(view_of(cache), a);
  return KDA_OK;
}

kda_status_t kda_cache_attention(const kda_cache_t* cache, const kda_attention_t* desc,
                                 const void* q, const int32_t* block_table,
                                 const int32_t* kv_lens, const int32_t* cu_new, void* out,
                                 float* lse, kda_stream_t stream) {
  const kda_status_t s = check_attention(cache, desc);
  if (s != KDA_OK) return s;
  if (desc->num_seqs == 0 || desc->total_tokens == 0) return KDA_OK;
  if (!q || !kv_lens || !cu_new || !out || q == out) return KDA_ERR_INVALID_ARGUMENT;
  if (desc->max_blocks > 0 && !block_table) return KDA_ERR_INVALID_ARGUMENT;
  const uintptr_t size = desc->io_dtype == KDA_BF16 ? 2 : 4;
  if (!aligned(q, size) || !aligned(out, 16)) return KDA_ERR_INVALID_ARGUMENT;
  if (!aligned(block_table, 4) || !aligned(kv_lens, 4) || !aligned(cu_new, 4) || !aligned(lse, 4))
    return KDA_ERR_INVALID_ARGUMENT;
  kda::AttentionArgs a;
  fill_attention(cache, desc, a);
  a.q = q;
  a.block_table = block_table;
  a.kv_lens = kv_lens;
  a.cu_new = cu_new;
  a.out = out;
  a.lse = lse;
  const size_t need = kda::cache_attention_workspace_bytes(view_of(cache), a);
  if (need > 0 && (!desc->workspace || desc->workspace_bytes < need ||
                   !aligned(desc->workspace, 256)))
    return KDA_ERR_INVALID_ARGUMENT;
  a.workspace = desc->workspace;
  a.err = kda::device_error();
  if (!a.err) return KDA_ERR_CUDA;
  return status_of(kda::launch_cache_attention(view_of(cache), a, (cudaStream_t)stream));
}

}  // extern "C"
