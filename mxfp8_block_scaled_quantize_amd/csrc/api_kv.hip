// C ABI of the paged MXFP4 key-value cache and of the rotary positions: host-side
// validation, then one launch sequence on the caller's stream.  See
// include/kvcache.h and include/rotary.h for the contracts.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "../../include/kvcache.h"
#include "../../include/rotary.h"
#include "kv.h"
#include "launch.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 40;
constexpr int64_t kMaxIndex = 0x7FFFFFFF;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mxfp8_status hip_status(hipError_t e) {
  if (e == hipSuccess) return MXFP8_OK;
  mx::note_hip_error(e);
  return MXFP8_ERR_HIP;
}

// a * b below 2^40, both not negative
bool product_ok(int64_t a, int64_t b) { return a <= kMaxDim && b <= kMaxDim && (a == 0 || b <= kMaxDim / a); }

int page_shift(int32_t page_size) {
  for (int s = 4; s <= 8; s++)
    if (page_size == 1 << s) return s;
  return -1;
}

mxfp8_status check_pages(int64_t pages, int32_t page_size) {
  if (pages < 1 || page_shift(page_size) < 0) return MXFP8_ERR_SHAPE;
  return pages > kMaxIndex / page_size ? MXFP8_ERR_LIMIT : MXFP8_OK;
}

mxfp8_status check_table(const void* table, int64_t ld_table, int64_t table_width, int64_t rows, int32_t page_size) {
  if (table_width < 0 || ld_table < table_width || rows < 0) return MXFP8_ERR_SHAPE;
  if (!product_ok(rows, ld_table) || table_width > (kMaxIndex - 4096) / page_size) return MXFP8_ERR_LIMIT;
  if (rows > 0 && table_width > 0 && !table) return MXFP8_ERR_NULL;
  return aligned(table, 4) ? MXFP8_OK : MXFP8_ERR_MISALIGNED;
}

mxfp8_status check_cache(const void* cache, int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim) {
  const mxfp8_status st = check_pages(pages, page_size);
  if (st != MXFP8_OK) return st;
  if (kv_heads < 1 || (head_dim != 64 && head_dim != 128 && head_dim != 256)) return MXFP8_ERR_SHAPE;
  const int64_t record = (int64_t)page_size * (head_dim + head_dim / 16);
  if (kv_heads > kMaxIndex / record || !product_ok(pages, kv_heads * record)) return MXFP8_ERR_LIMIT;
  if (!cache) return MXFP8_ERR_NULL;
  return aligned(cache, 16) ? MXFP8_OK : MXFP8_ERR_MISALIGNED;
}

mx::KvCache cache_of(const uint8_t* data, int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim) {
  return mx::KvCache{data, pages, page_size, page_shift(page_size), kv_heads, head_dim};
}

mx::KvAttention attention_of(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t sequences,
                             int64_t table_width, int32_t page_size, const int32_t* offsets, int64_t max_queries,
                             int64_t window) {
  mx::KvAttention a{};
  a.tokens = tokens;
  a.heads = heads;
  a.cache = cache_of(nullptr, 1, page_size, kv_heads, head_dim);
  a.table_width = table_width;
  a.offsets = offsets;
  a.sequences = sequences;
  a.max_queries = !offsets ? 1 : max_queries < tokens ? max_queries : tokens > 1 ? tokens : 1;
  a.window = window > kMaxIndex ? 0 : window;   // no sequence is longer
  return a;
}

// Sizes that the workspace depends on.
mxfp8_status check_attention(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t sequences,
                             int64_t table_width, int32_t page_size, int64_t max_queries, int64_t window, bool ragged) {
  if (page_shift(page_size) < 0 || kv_heads < 1 || heads < 1 || heads % kv_heads) return MXFP8_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return MXFP8_ERR_SHAPE;
  if (tokens < 0 || sequences < 0 || table_width < 0 || max_queries < 1 || window < 0) return MXFP8_ERR_SHAPE;
  if (!ragged && tokens != sequences) return MXFP8_ERR_SHAPE;
  if (heads / kv_heads > 65536 || sequences > kMaxIndex || tokens > kMaxIndex / heads) return MXFP8_ERR_LIMIT;
  if (table_width > (kMaxIndex - 4096) / page_size) return MXFP8_ERR_LIMIT;
  return MXFP8_OK;
}

}  // namespace

extern "C" {

mxfp8_status kv_extend(int32_t* table, int64_t ld_table, int64_t table_width, const int32_t* lengths, const int32_t* counts,
                       int64_t requests, const int32_t* free, const int32_t* free_count, int64_t pages, int32_t page_size,
                       int64_t tokens, int32_t* offsets, int32_t* lengths_out, int32_t* slots, int32_t* positions,
                       int32_t* free_count_out, void* stream) {
  mxfp8_status st = check_pages(pages, page_size);
  if (st == MXFP8_OK && tokens < 0) st = MXFP8_ERR_SHAPE;
  if (st == MXFP8_OK) st = check_table(table, ld_table, table_width, requests, page_size);
  if (st != MXFP8_OK) return st;
  if (requests >= (1 << 24) || tokens >= kMaxIndex) return MXFP8_ERR_LIMIT;
  if (!offsets || !free || !free_count || !free_count_out || (requests > 0 && (!lengths || !counts || !lengths_out)) ||
      (tokens > 0 && (!slots || !positions)))
    return MXFP8_ERR_NULL;
  for (const void* p : {(const void*)lengths, (const void*)counts, (const void*)free, (const void*)free_count,
                        (const void*)offsets, (const void*)lengths_out, (const void*)slots, (const void*)positions,
                        (const void*)free_count_out})
    if (!aligned(p, 4)) return MXFP8_ERR_MISALIGNED;
  return hip_status(mx::launch_kv_extend(table, ld_table, table_width, lengths, counts, requests, free, free_count, pages,
                                         page_shift(page_size), tokens, offsets, lengths_out, slots, positions, free_count_out,
                                         static_cast<hipStream_t>(stream)));
}

mxfp8_status kv_release(int32_t* table, int64_t ld_table, int64_t table_width, const int32_t* lengths, const uint8_t* finished,
                        int64_t requests, int32_t* free, const int32_t* free_count, int64_t pages, int32_t page_size,
                        int32_t* lengths_out, int32_t* free_count_out, void* stream) {
  mxfp8_status st = check_pages(pages, page_size);
  if (st == MXFP8_OK) st = check_table(table, ld_table, table_width, requests, page_size);
  if (st != MXFP8_OK) return st;
  if (requests >= (1 << 24)) return MXFP8_ERR_LIMIT;
  if (!free || !free_count || !free_count_out || (requests > 0 && (!lengths || !finished || !lengths_out))) return MXFP8_ERR_NULL;
  for (const void* p : {(const void*)lengths, (const void*)free, (const void*)free_count, (const void*)lengths_out,
                        (const void*)free_count_out})
    if (!aligned(p, 4)) return MXFP8_ERR_MISALIGNED;
  return hip_status(mx::launch_kv_release(table, ld_table, table_width, lengths, finished, requests, free, free_count, pages,
                                          page_shift(page_size), lengths_out, free_count_out,
                                          static_cast<hipStream_t>(stream)));
}

mxfp8_status kv_append(uint8_t* cache, int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim, const void* k,
                       int64_t k_token, int64_t k_head, const void* v, int64_t v_token, int64_t v_head, const int32_t* slots,
                       int64_t tokens, void* stream) {
  const mxfp8_status st = check_cache(cache, pages, page_size, kv_heads, head_dim);
  if (st != MXFP8_OK) return st;
  if (tokens < 0 || k_token < 0 || k_head < 0 || v_token < 0 || v_head < 0) return MXFP8_ERR_SHAPE;
  if (!product_ok(tokens, k_token) || !product_ok(tokens, v_token) || !product_ok(kv_heads, k_head) ||
      !product_ok(kv_heads, v_head) || !mx::kv_copy_grid_fits(tokens, kv_heads, head_dim))
    return MXFP8_ERR_LIMIT;
  if (tokens == 0) return MXFP8_OK;
  if (!k || !v || !slots) return MXFP8_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || k_token % 8 || k_head % 8 || v_token % 8 || v_head % 8)
    return MXFP8_ERR_MISALIGNED;
  return hip_status(mx::launch_kv_append(cache_of(cache, pages, page_size, kv_heads, head_dim),
                                         {static_cast<const uint16_t*>(k), k_token, k_head},
                                         {static_cast<const uint16_t*>(v), v_token, v_head}, slots, tokens,
                                         static_cast<hipStream_t>(stream)));
}

mxfp8_status kv_read(const uint8_t* cache, int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim,
                     const int32_t* slots, int64_t tokens, void* k, void* v, void* stream) {
  const mxfp8_status st = check_cache(cache, pages, page_size, kv_heads, head_dim);
  if (st != MXFP8_OK) return st;
  if (tokens < 0) return MXFP8_ERR_SHAPE;
  if (!mx::kv_copy_grid_fits(tokens, kv_heads, head_dim)) return MXFP8_ERR_LIMIT;
  if (tokens == 0) return MXFP8_OK;
  if (!k || !v || !slots) return MXFP8_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return MXFP8_ERR_MISALIGNED;
  return hip_status(mx::launch_kv_read(cache_of(cache, pages, page_size, kv_heads, head_dim), slots, tokens,
                                       static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), static_cast<hipStream_t>(stream)));
}

size_t kv_attention_workspace_bytes(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t sequences,
                                    int64_t table_width, int32_t page_size, int32_t ragged, int64_t max_queries,
                                    int64_t window) {
  static const int32_t some = 0;
  if (check_attention(tokens, heads, kv_heads, head_dim, sequences, table_width, page_size, max_queries, window, ragged != 0) !=
          MXFP8_OK ||
      tokens == 0 || sequences == 0)
    return 0;
  return mx::kv_attention_workspace(attention_of(tokens, heads, kv_heads, head_dim, sequences, table_width, page_size,
                                                 ragged ? &some : nullptr, max_queries, window));
}

mxfp8_status kv_attention(const void* q, int64_t q_token, int64_t q_head, int64_t tokens, int32_t heads, const uint8_t* cache,
                          int64_t pages, int32_t page_size, int32_t kv_heads, int32_t head_dim, const int32_t* table,
                          int64_t ld_table, int64_t table_width, const int32_t* lengths, const int32_t* offsets,
                          int64_t sequences, int64_t max_queries, float scale, int64_t window, void* out, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream) {
  mxfp8_status st = check_attention(tokens, heads, kv_heads, head_dim, sequences, table_width, page_size, max_queries, window,
                                    offsets != nullptr);
  if (st == MXFP8_OK) st = check_cache(cache, pages, page_size, kv_heads, head_dim);
  if (st == MXFP8_OK) st = check_table(table, ld_table, table_width, sequences, page_size);
  if (st != MXFP8_OK) return st;
  if (q_token < 0 || q_head < 0 || !(scale > 0.0f) || !std::isfinite(scale)) return MXFP8_ERR_SHAPE;
  if (!product_ok(tokens, q_token) || !product_ok(heads, q_head)) return MXFP8_ERR_LIMIT;
  if (tokens == 0 || sequences == 0) return MXFP8_OK;
  if (!q || !out || !lengths) return MXFP8_ERR_NULL;
  if (!aligned(q, 16) || q_token % 8 || q_head % 8 || !aligned(out, 16) || !aligned(lengths, 4) || !aligned(offsets, 4) ||
      !aligned(lse, 4))
    return MXFP8_ERR_MISALIGNED;
  mx::KvAttention a = attention_of(tokens, heads, kv_heads, head_dim, sequences, table_width, page_size, offsets, max_queries, window);
  if (!mx::kv_attention_grid_fits(a)) return MXFP8_ERR_LIMIT;
  const size_t need = mx::kv_attention_workspace(a);
  if (need && (!workspace || workspace_bytes < need)) return MXFP8_ERR_WORKSPACE;
  if (need && !aligned(workspace, 16)) return MXFP8_ERR_MISALIGNED;
  a.q = static_cast<const uint16_t*>(q);
  a.q_token = q_token;
  a.q_head = q_head;
  a.cache = cache_of(cache, pages, page_size, kv_heads, head_dim);
  a.table = table;
  a.ld_table = ld_table;
  a.lengths = lengths;
  a.scale = scale;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.workspace = static_cast<float*>(workspace);
  return hip_status(mx::launch_kv_attention(a, static_cast<hipStream_t>(stream)));
}

mxfp8_status rotary_rotate(const void* q, int64_t q_token, int64_t q_head, int64_t q_heads, const void* k, int64_t k_token,
                           int64_t k_head, int64_t k_heads, int32_t dtype, int64_t tokens, int64_t head_dim, int64_t pairs,
                           const int32_t* positions, const double* turns, float magnitude, uint32_t flags, void* q_out,
                           void* k_out, void* stream) {
  if (dtype < ROTARY_FP32 || dtype > ROTARY_FP16 || (flags & ~(ROTARY_INTERLEAVED | ROTARY_INVERSE))) return MXFP8_ERR_FLAGS;
  if (tokens < 0 || q_heads < 0 || k_heads < 0 || head_dim < 1 || pairs < 0 || pairs > head_dim / 2 || q_token < 0 ||
      q_head < 0 || k_token < 0 || k_head < 0)
    return MXFP8_ERR_SHAPE;
  if (head_dim > 65536 || q_heads > (1 << 20) || k_heads > (1 << 20) || !product_ok(tokens, q_token) ||
      !product_ok(tokens, k_token) || !product_ok(q_heads, q_head) || !product_ok(k_heads, k_head) ||
      !product_ok(tokens, (q_heads + k_heads) * head_dim))
    return MXFP8_ERR_LIMIT;
  const mx::RotaryCall call{{q, q_out, q_token, q_head, q_heads}, {k, k_out, k_token, k_head, k_heads}, dtype, tokens, head_dim, pairs,
                            positions, turns, magnitude, (flags & ROTARY_INTERLEAVED) != 0, (flags & ROTARY_INVERSE) != 0};
  if (tokens > 0 && q_heads + k_heads > 0 && !mx::rotary_grid_fits(call)) return MXFP8_ERR_LIMIT;
  if (tokens == 0 || q_heads + k_heads == 0) return MXFP8_OK;
  if ((q_heads > 0 && (!q || !q_out)) || (k_heads > 0 && (!k || !k_out)) || (pairs > 0 && (!positions || !turns)))
    return MXFP8_ERR_NULL;
  const uintptr_t size = dtype == ROTARY_FP32 ? 4 : 2;
  if (!aligned(q, size) || !aligned(k, size) || !aligned(q_out, size) || !aligned(k_out, size) || !aligned(positions, 4) ||
      !aligned(turns, 8))
    return MXFP8_ERR_MISALIGNED;
  return hip_status(mx::launch_rotary(call, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
