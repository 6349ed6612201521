// The paged MXFP4 key-value cache: its layout on the device, and the launchers
// behind include/kvcache.h and include/rotary.h (sizes as checked there).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mx {

// One cache: records [pages][heads] of a page's tokens (see include/kvcache.h).
struct KvCache {
  const uint8_t* data;
  int64_t pages;
  int32_t page_size, page_shift, heads, head_dim;
  __host__ __device__ int64_t record() const { return (int64_t)page_size * (head_dim + head_dim / 16); }
  __host__ __device__ int32_t v_codes() const { return page_size * (head_dim / 2); }
  __host__ __device__ int32_t k_scales() const { return page_size * head_dim; }
  __host__ __device__ int32_t v_scales() const { return page_size * head_dim + page_size * (head_dim / 32); }
};

hipError_t launch_kv_extend(int32_t* table, int64_t ld, int64_t width, const int32_t* lengths, const int32_t* counts,
                            int64_t requests, const int32_t* free, const int32_t* free_count, int64_t pages, int page_shift,
                            int64_t tokens, int32_t* offsets, int32_t* lengths_out, int32_t* slots, int32_t* positions,
                            int32_t* free_count_out, hipStream_t stream);
hipError_t launch_kv_release(int32_t* table, int64_t ld, int64_t width, const int32_t* lengths, const uint8_t* finished,
                             int64_t requests, int32_t* free, const int32_t* free_count, int64_t pages, int page_shift,
                             int32_t* lengths_out, int32_t* free_count_out, hipStream_t stream);

struct KvRows {   // keys or values of tokens, BF16, strides in elements
  const uint16_t* data;
  int64_t token, head;
};
bool kv_copy_grid_fits(int64_t tokens, int32_t heads, int32_t head_dim);
hipError_t launch_kv_append(const KvCache& c, KvRows k, KvRows v, const int32_t* slots, int64_t tokens, hipStream_t stream);
hipError_t launch_kv_read(const KvCache& c, const int32_t* slots, int64_t tokens, uint16_t* k, uint16_t* v, hipStream_t stream);

struct KvAttention {
  const uint16_t* q;
  int64_t q_token, q_head, tokens;
  int32_t heads;
  KvCache cache;
  const int32_t* table;
  int64_t ld_table, table_width;
  const int32_t* lengths;
  const int32_t* offsets;   // null: one query a sequence
  int64_t sequences, max_queries;
  float scale;
  int64_t window;
  uint16_t* out;
  float* lse;
  float* workspace;
};
size_t kv_attention_workspace(const KvAttention& a);
bool kv_attention_grid_fits(const KvAttention& a);
hipError_t launch_kv_attention(const KvAttention& a, hipStream_t stream);

struct RotaryRows {   // strides in elements
  const void* in;
  void* out;
  int64_t token, head, heads;
};
struct RotaryCall {
  RotaryRows q, k;
  int dtype;
  int64_t tokens, head_dim, pairs;
  const int32_t* positions;
  const double* turns;
  float magnitude;
  bool interleaved, inverse;
};
bool rotary_grid_fits(const RotaryCall& c);
hipError_t launch_rotary(const RotaryCall& c, hipStream_t stream);

}  // namespace mx
