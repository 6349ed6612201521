// Writing keys and values into the paged MXFP4 cache, and reading them back.
//
// A lane takes 8 values of a token's key and the same 8 of its value; a block of 32
// is a DPP quad, as in the MXFP4 quantizer, whose rule for scales and codes this
// is.  Four tokens of a head stand next to each other in a wave, so that their
// values' codes, which the cache keeps by groups of four tokens, leave as whole
// runs.  Bound by HBM for many tokens (16381 tokens of 8 heads of 128: written in 16.5 us,
// 83 MB at 5.0 TB/s, read back in 14.3, 89 MB at 6.2), by one load's latency for few (2.5 us
// each).
#include "kv.h"
#include "launch.h"
#include "mx_device.h"

namespace mx {

namespace {

// E8M0 byte of a block from the 15-bit pattern of its amax, as the quantizer's,
// but at most 252: 6 * 2^125 is the largest finite value of a code in BF16, and a
// token with an infinity or NaN must not reach the queries that do not see it.
__device__ __forceinline__ uint32_t cache_scale(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 7);
  return (uint32_t)(e > 2 ? (e < 255 ? e - 2 : 252) : 0);
}
#define MX4_CVT(word, pair, scale, i) \
  (uint32_t) __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16((word), __builtin_bit_cast(bf16x2, (uint32_t)(pair)), (scale), (i))
__device__ __forceinline__ uint32_t codes_of(uint4 v, uint32_t* byte) {
  uint32_t m = pk_max_u16(pk_max_u16(abs_bits2(v.x), abs_bits2(v.y)), pk_max_u16(abs_bits2(v.z), abs_bits2(v.w)));
  m = quad_max(max(m & 0xFFFFu, m >> 16));
  *byte = cache_scale(m);
  const float f = __uint_as_float(*byte << 23);
  uint32_t w = 0;
  w = MX4_CVT(w, v.x, f, 0);
  w = MX4_CVT(w, v.y, f, 1);
  w = MX4_CVT(w, v.z, f, 2);
  w = MX4_CVT(w, v.w, f, 3);
  return w;
}
__device__ __forceinline__ uint4 values_of(uint32_t codes, uint32_t byte) {
  const float f = __uint_as_float(byte << 23);
  uint4 o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, f, 0));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, f, 1));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, f, 2));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, f, 3));
  return o;
}

// Lane -> (four tokens, head, token of the four, 8 values): the token and head
// count of a call are those of its grid.
template <int D>
struct Place {
  int64_t token;
  int head, c;
  bool valid;
  __device__ __forceinline__ Place(int64_t tokens, int heads) {
    const uint32_t x = blockIdx.x * 256 + threadIdx.x;   // below 2^32, as the grid
    const uint32_t row = x / (D / 8), group = row / 4;
    c = (int)(x % (D / 8));
    head = (int)(group % (uint32_t)heads);
    token = (int64_t)(group / (uint32_t)heads) * 4 + row % 4;
    valid = token < tokens;
  }
};

// Where the 8 values c of a slot are.
template <int D>
struct Entry {
  uint32_t k, v, ks, vs;
  __device__ __forceinline__ Entry(const KvCache& g, int o, int c) {
    k = (uint32_t)o * (D / 2) + 4 * c;
    v = g.v_codes() + ((uint32_t)(o >> 2) * (D / 8) + c) * 16 + (o & 3) * 4;
    ks = g.k_scales() + (uint32_t)o * (D / 32) + c / 4;
    vs = g.v_scales() + (uint32_t)(c / 4) * g.page_size + o;
  }
};

template <int D>
__global__ __launch_bounds__(256) void kv_append_kernel(KvCache g, uint8_t* __restrict__ cache, KvRows k, KvRows v,
                                                        const int32_t* __restrict__ slots, int64_t tokens) {
  const Place<D> at(tokens, g.heads);
  if (!at.valid) return;   // whole quads
  const int64_t slot = slots[at.token];
  if (slot < 0 || (slot >> g.page_shift) >= g.pages) return;
  const uint4 kv = load_nt16(k.data + at.token * k.token + at.head * k.head + 8 * at.c);
  const uint4 vv = load_nt16(v.data + at.token * v.token + at.head * v.head + 8 * at.c);
  uint8_t* record = cache + ((slot >> g.page_shift) * g.heads + at.head) * g.record();
  const Entry<D> e(g, (int)(slot & (g.page_size - 1)), at.c);
  uint32_t ks, vs;
  const uint32_t kc = codes_of(kv, &ks), vc = codes_of(vv, &vs);
  *reinterpret_cast<uint32_t*>(record + e.k) = kc;
  *reinterpret_cast<uint32_t*>(record + e.v) = vc;
  if ((at.c & 3) == 0) {
    record[e.ks] = (uint8_t)ks;
    record[e.vs] = (uint8_t)vs;
  }
}

template <int D>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache g, const int32_t* __restrict__ slots, int64_t tokens,
                                                      uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  const Place<D> at(tokens, g.heads);
  if (!at.valid) return;
  const int64_t slot = slots[at.token];
  uint4 kv = make_uint4(0u, 0u, 0u, 0u), vv = kv;
  if (slot >= 0 && (slot >> g.page_shift) < g.pages) {
    const uint8_t* record = g.data + ((slot >> g.page_shift) * g.heads + at.head) * g.record();
    const Entry<D> e(g, (int)(slot & (g.page_size - 1)), at.c);
    kv = values_of(*reinterpret_cast<const uint32_t*>(record + e.k), record[e.ks]);
    vv = values_of(*reinterpret_cast<const uint32_t*>(record + e.v), record[e.vs]);
  }
  const int64_t to = (at.token * g.heads + at.head) * D + 8 * at.c;
  *reinterpret_cast<uint4*>(k + to) = kv;
  *reinterpret_cast<uint4*>(v + to) = vv;
}

unsigned blocks_of(int64_t tokens, int32_t heads, int32_t head_dim) {
  return (unsigned)(((tokens + 3) / 4 * 4 * heads * (head_dim / 8) + 255) / 256);
}

}  // namespace

bool kv_copy_grid_fits(int64_t tokens, int32_t heads, int32_t head_dim) {
  return tokens <= kMaxWorkItems && grid_fits((tokens + 3) / 4 * 4, (int64_t)heads * (head_dim / 8), 1) &&
         (tokens + 3) / 4 * 4 * heads * (head_dim / 8) <= kMaxWorkItems - 255;
}

hipError_t launch_kv_append(const KvCache& c, KvRows k, KvRows v, const int32_t* slots, int64_t tokens, hipStream_t stream) {
  const dim3 grid(blocks_of(tokens, c.heads, c.head_dim));
  uint8_t* cache = const_cast<uint8_t*>(c.data);
  if (c.head_dim == 64) hipLaunchKernelGGL(kv_append_kernel<64>, grid, dim3(256), 0, stream, c, cache, k, v, slots, tokens);
  else if (c.head_dim == 128) hipLaunchKernelGGL(kv_append_kernel<128>, grid, dim3(256), 0, stream, c, cache, k, v, slots, tokens);
  else hipLaunchKernelGGL(kv_append_kernel<256>, grid, dim3(256), 0, stream, c, cache, k, v, slots, tokens);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache& c, const int32_t* slots, int64_t tokens, uint16_t* k, uint16_t* v, hipStream_t stream) {
  const dim3 grid(blocks_of(tokens, c.heads, c.head_dim));
  if (c.head_dim == 64) hipLaunchKernelGGL(kv_read_kernel<64>, grid, dim3(256), 0, stream, c, slots, tokens, k, v);
  else if (c.head_dim == 128) hipLaunchKernelGGL(kv_read_kernel<128>, grid, dim3(256), 0, stream, c, slots, tokens, k, v);
  else hipLaunchKernelGGL(kv_read_kernel<256>, grid, dim3(256), 0, stream, c, slots, tokens, k, v);
  return hipGetLastError();
}

}  // namespace mx
