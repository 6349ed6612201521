// Attention of many queries (prompts, pieces of prompts) over the paged MXFP4 cache:
// bound by the matrix cores and, beside them, by the softmax's exponentials.
//
// A workgroup of W = 4 (or 2) waves has 32 W rows of one sequence and key-value head,
// and goes through its keys 64 at a time.  S^T = K Q^T by 32x32x64 scaled MFMAs whose
// FP4 operand is 16 bytes of a key's codes a lane, loaded straight from the cache a
// step ahead.  Lane (c, h) = (l % 32, l / 32) gets the scores of row c and keys 8 (i /
// 4) + 4 h + i % 4 of each 32: its eight registers of every 16 keys are the second
// product's operand as they are, with that product's keys in the order (4 h + 0..3, 8 +
// 4 h + 0..3) for lane half h.  The values are turned to BF16 once for the workgroup,
// a step ahead: a lane takes 4 keys x 8 values, swaps them pairwise and writes, for each
// value, the 4 keys to an LDS row of 64 keys in that order (two buffers).  O^T = V^T P^T
// by 32x32x16 MFMAs.  One barrier a step.
//
// LDS: a row is 8 chunks of 8 keys (16 bytes), chunk k of value 8 e + i in place k ^ (i /
// 2) ^ (e with its bits 1 and 2 swapped).  Reads take 16 bytes of 32 neighbouring rows,
// which the hardware serves 16 lanes at a time (lanes 0-3, 12-15, 20-23, 24-27, then the
// others): these meet all 16 chunks of 64 banks.  Writes of 8 bytes go 16 neighbouring
// lanes at a time to 32 banks: 8 neighbouring e times the two halves of a chunk, which is
// why lane bit 3 is the half.  No conflicts are counted (with the chunks placed by k ^ e
// in padded rows 161 cycles a wave and step, and 3 % of the time).
//
// What bounds it: of the 2160 cycles that a SIMD takes for a wave's step (500 queries over
// 49152 keys, 32 heads of 128, 2 waves a SIMD at 2.0 GHz) the matrix cores work 1025 and the
// vector unit 1050, of which the exponentials are a quarter, and the two overlap little.  With
// 64 values the vector unit works 70 % of the time and the matrix cores 31; with 256, one wave
// a SIMD, 35 and 27, as nothing stands beside a wave's waiting (prompts of up to 4096
// queries).  Tried and slower: 3 waves a SIMD with 32 keys a softmax (470 us against 432),
// 8 waves that share the values (511), 64 rows a wave (600), wave priorities (442),
// fragments read a product ahead (400 against 395).
#include "kv_attention.h"

namespace mx {

using namespace kv;

namespace {

constexpr int KEYS = 64;
constexpr int ROW = 2 * KEYS;   // bytes of a value's LDS row: 8 chunks of 8 keys
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;

// Place of chunk k (bytes from its row's start) in the row of value 8 e + i: see the head.
__device__ __forceinline__ uint32_t place_of(uint32_t k, uint32_t e, uint32_t i) {
  return ((k ^ (i >> 1) ^ ((e & 1) | (e & 2) << 1 | (e & 4) >> 1)) & 7) * 16;
}

// WHOLE: 32 keys lie in one page (pages of 32 tokens or more), so that a step's keys have
// scalar bases and their loads no address arithmetic (500 queries over 49152 keys, pages of
// 64: 400 us, with an address for every lane 430).  Else pages are 16 tokens, a run each.
//
// The page numbers of a step's four runs of 16 keys, and of the wave's R.  No branch
// here and in the loads (a number that is no page, a key behind the end are read as ones
// that are there, and masked): the compiler can then wait for one step's loads among the
// next one's.
template <bool WHOLE, int R>
struct Runs {
  uint32_t p[4], own[R];
  __device__ __forceinline__ void find(const Args& a, const Tile& t, int key, int end, int w) {
    const int32_t* row = a.table + t.sequence * a.ld_table;
    const int shift = WHOLE ? a.page_shift : 4;
#pragma unroll
    for (int i = 0; i < 4; i++) p[i] = WHOLE && (i & 1) ? p[i - 1] : (uint32_t)row[min(key + 16 * i, end - 1) >> shift];
#pragma unroll
    for (int j = 0; j < R; j++) own[j] = (uint32_t)row[min(key + 16 * (R * w + j), end - 1) >> shift];
  }
  __device__ __forceinline__ bool there(const Args& a, int i) const { return p[i] < (uint32_t)a.pages; }
  __device__ __forceinline__ bool all(const Args& a) const { return max(max(p[0], p[1]), max(p[2], p[3])) < (uint32_t)a.pages; }
};
__device__ __forceinline__ const uint8_t* safe_record(const Args& a, int head, uint32_t page) {
  return record_of(a, head, (int)min(page, (uint32_t)a.pages - 1));
}

// What a lane loads of a step's keys: 32 codes (16 bytes) and a scale for every MFMA.
template <int D>
struct KeyPart {
  static constexpr int KS = D / 64;   // MFMA steps along a key
  u32x4 k[2][KS];
  uint32_t s[2][(KS + 1) / 2];
  template <bool WHOLE, int R>
  __device__ __forceinline__ void load(const Args& a, const Runs<WHOLE, R>& runs, int head, int key) {
    const uint32_t lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      if (WHOLE) {
        const int page_size = 1 << a.page_shift;
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(safe_record(a, head, runs.p[2 * i])), 0, (int)a.record, 0x00020000);
        const int at = (key + 32 * i) & (page_size - 1);
#pragma unroll
        for (int f = 0; f < KS; f++) k[i][f] = __builtin_amdgcn_raw_buffer_load_b128(r, c * (D / 2) + 16 * h + 32 * f, at * (D / 2), 0);
        if (D == 64) s[i][0] = __builtin_amdgcn_raw_buffer_load_b16(r, c * (D / 32), page_size * D + at * (D / 32), 0);
        else {
#pragma unroll
          for (int f = 0; f < KS / 2; f++) s[i][f] = __builtin_amdgcn_raw_buffer_load_b32(r, c * (D / 32) + 4 * f, page_size * D + at * (D / 32), 0);
        }
        continue;
      }
      // a page for every 16 lanes
      const uint8_t *r0 = safe_record(a, head, runs.p[2 * i]), *r1 = safe_record(a, head, runs.p[2 * i + 1]);
      const uint8_t* const r = c & 16 ? r1 : r0;
      const uint8_t *k0 = r + ((c & 15) * (D / 2) + 16 * h), *s0 = r + (16 * D + (c & 15) * (D / 32));
#pragma unroll
      for (int f = 0; f < KS; f++) k[i][f] = *reinterpret_cast<const u32x4*>(k0 + 32 * f);
      if (D == 64) s[i][0] = *reinterpret_cast<const uint16_t*>(s0);
      else {
#pragma unroll
        for (int f = 0; f < KS / 2; f++) s[i][f] = reinterpret_cast<const uint32_t*>(s0)[f];
      }
    }
  }
};

// What a lane loads of a run's values: units of 4 keys x 8 values of 16 keys, run w of the
// step (with 64 values both halves of the wave the same ones).
template <int D>
struct ValuePart {
  static constexpr int UNITS = D == 256 ? 2 : 1;
  u32x4 v[UNITS];
  uint32_t s[UNITS];
  // quad 2 * half + odd of the run's four
  static __device__ __forceinline__ uint32_t half() { return (threadIdx.x >> 3) & 1; }
  static __device__ __forceinline__ uint32_t odd(int u) { return D == 256 ? u : (threadIdx.x >> (D == 64 ? 4 : 5)) & 1; }
  static __device__ __forceinline__ uint32_t quad(int u) { return 2 * half() + odd(u); }
  static __device__ __forceinline__ uint32_t eight() { return ((threadIdx.x & 7) | ((threadIdx.x & 63) >> 4) << 3) & (D / 8 - 1); }
  template <bool WHOLE>
  __device__ __forceinline__ void load(const Args& a, uint32_t page, int head, int key, int w) {
    const uint32_t page_size = WHOLE ? 1u << a.page_shift : 16;
    const uint32_t at = WHOLE ? (uint32_t)(key + 16 * w) & (page_size - 1) : 0;
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(safe_record(a, head, page)), 0, (int)a.record, 0x00020000);
#pragma unroll
    for (int u = 0; u < UNITS; u++) {
      v[u] = __builtin_amdgcn_raw_buffer_load_b128(r, quad(u) * (2 * D) + 16 * eight(), page_size * (D / 2) + (at >> 2) * (2 * D), 0);
      s[u] = __builtin_amdgcn_raw_buffer_load_b32(r, (eight() >> 2) * page_size + 4 * quad(u), page_size * (D + D / 32) + at, 0);
    }
  }
  // Of places that no query of the tile sees, zeros: [lo, end) are the keys of some.
  __device__ __forceinline__ void mask(const Args& a, uint32_t page, int key, int lo, int end, int w) {
    const bool there = page < (uint32_t)a.pages;
    const int at = key + 16 * w;
    if ((uint32_t)(at - lo) < (uint32_t)max(end - lo - 15, 0) && there) return;
#pragma unroll
    for (int u = 0; u < UNITS; u++)
#pragma unroll
      for (int j = 0; j < 4; j++)
        if (!there || (uint32_t)(at + 4 * (int)quad(u) + j - lo) >= (uint32_t)(end - lo)) {
          v[u][j] = 0;
          s[u] &= ~(0xFFu << (8 * j));
        }
  }
  // As BF16 to the LDS rows.
  __device__ __forceinline__ void store(lds_u8* to, int w) const {
#pragma unroll
    for (int u = 0; u < UNITS; u++) {
      uint32_t x[4][4];
#pragma unroll
      for (int j = 0; j < 4; j++) bf16_of(v[u][j], scale_of(s[u], j), x[j]);
      lds_u8* const row = to + eight() * (8 * ROW) + 8 * half();
      const uint32_t first = place_of(2 * w + odd(u), eight(), 0);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        u32x2 word;
        word.x = (i & 1) ? highs(x[0][i >> 1], x[1][i >> 1]) : lows(x[0][i >> 1], x[1][i >> 1]);
        word.y = (i & 1) ? highs(x[2][i >> 1], x[3][i >> 1]) : lows(x[2][i >> 1], x[3][i >> 1]);
        *reinterpret_cast<lds_u32x2*>(row + (first ^ (16 * (i >> 1))) + i * ROW) = word;
      }
    }
  }
};

template <int D, bool WHOLE, int W>
__global__ __launch_bounds__(64 * W, D == 256 ? 1 : 2) void kv_attention_tile_kernel(Args a) {
  constexpr int KS = KeyPart<D>::KS;
  __shared__ __attribute__((aligned(16))) uint8_t values[2][D * ROW];
  lds_u8* const lds = (lds_u8*)&values[0][0];
  const int lane = threadIdx.x & 63, c = lane & 31, h = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const Place place(a);
  const int head = place.head, part = place.part;
  Tile t;
  // the last tiles of a sequence, which see the most keys, first
  if (!find_tile<32 * W>(a, place.tile < a.likely ? a.likely - 1 - place.tile : place.tile, &t)) return;   // the whole workgroup
  const int rows = t.rows < 32 * W ? t.rows : 32 * W;
  const int64_t all_rows = (int64_t)a.tokens * a.heads;

  int first_lo, first_hi, last_lo, last_hi;
  seen(a, t, t.row0 / a.group, &first_lo, &first_hi);
  seen(a, t, (t.row0 + rows - 1) / a.group, &last_lo, &last_hi);
  const int end = last_hi, begin = first_lo < end ? first_lo & ~(KEYS - 1) : 0;
  const int steps = first_lo < end ? (end - begin + KEYS - 1) / KEYS : 0;
  const int each = steps ? __builtin_amdgcn_readfirstlane(part_steps<KEYS>(a, steps)) : 1;
  const int used = __builtin_amdgcn_readfirstlane((steps + each - 1) / each);
  const bool whole = used <= 1;   // the outputs are written here
  const int s0 = part * each, s1 = s0 + each < steps ? s0 + each : steps;

  // this lane's row, and the keys of the wave's rows
  // (a workgroup without a part has none: a return here would cost the kernel 7 to 14 registers)
  const int row = 32 * w + c;
  const bool valid = row < rows && (part == 0 || part < used);
  const int x = (t.row0 + (valid ? row : 0)) / a.group;
  const int64_t token = t.first_token + x;
  const int q_head = head * a.group + (t.row0 + (valid ? row : 0)) - x * a.group;
  int lo, hi;
  seen(a, t, x, &lo, &hi);
  if (!valid) lo = hi = 0;
  const bool has_rows = 32 * w < rows;   // wave-uniform
  int wave_lo = 0, wave_hi = 0, all_lo = 0, all_hi = 0;   // keys that some row of the wave, that all of them see
  if (has_rows) {
    const int last = 32 * w + 31 < rows ? 32 * w + 31 : rows - 1;
    seen(a, t, (t.row0 + 32 * w) / a.group, &wave_lo, &all_hi);
    seen(a, t, (t.row0 + last) / a.group, &all_lo, &wave_hi);
  }
  v8i qh[KS], ql[KS];
  int scale;
  {
    const uint16_t* q = a.q + token * a.q_token + q_head * a.q_head;
    uint4 v[KS][4];
    uint32_t m = 0;
#pragma unroll
    for (int s = 0; s < KS; s++)
#pragma unroll
      for (int i = 0; i < 4; i++) {   // bytes 0 .. 15: dimensions 16 h + .., 16 .. 31: 32 + 16 h + ..
        v[s][i] = valid ? *reinterpret_cast<const uint4*>(q + 64 * s + 32 * (i >> 1) + 16 * h + 8 * (i & 1)) : make_uint4(0u, 0u, 0u, 0u);
        m = max(m, amax8(v[s][i]));
      }
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    scale = query_scale(m);
#pragma unroll
    for (int s = 0; s < KS; s++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        uint32_t x2[2], y2[2];
        split8(v[s][i], scale, x2, y2);
#pragma unroll
        for (int j = 0; j < 2; j++) {
          qh[s][2 * i + j] = (int)x2[j];
          ql[s][2 * i + j] = (int)y2[j];
        }
      }
  }

  v16f o[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; d++)
#pragma unroll
    for (int i = 0; i < 16; i++) o[d][i] = 0.0f;
  float top = -INFINITY, sum = 0.0f;

  constexpr int R = 4 / W;   // runs of 16 keys whose values a wave turns to BF16
  Runs<WHOLE, R> runs, ahead;   // of this step and the next
  KeyPart<D> keys;
  ValuePart<D> vals[R];
  auto load_values = [&](const Runs<WHOLE, R>& of, int key) {
#pragma unroll
    for (int j = 0; j < R; j++) vals[j].template load<WHOLE>(a, of.own[j], head, key, R * w + j);
  };
  auto mask_values = [&](const Runs<WHOLE, R>& of, int key) {
#pragma unroll
    for (int j = 0; j < R; j++) vals[j].mask(a, of.own[j], key, first_lo, end, R * w + j);
  };
  auto store_values = [&](lds_u8* to) {
#pragma unroll
    for (int j = 0; j < R; j++) vals[j].store(to, R * w + j);
  };
  if (s0 < s1) {
    runs.find(a, t, begin + KEYS * s0, end, w);
    ahead.find(a, t, begin + KEYS * (s0 + 1), end, w);
    load_values(runs, begin + KEYS * s0);
    keys.load(a, runs, head, begin + KEYS * s0);
    mask_values(runs, begin + KEYS * s0);
    store_values(lds + (s0 & 1) * D * ROW);
  }
  __syncthreads();
  for (int s = s0; s < s1; s++) {
    const int key = begin + KEYS * s;
    Runs<WHOLE, R> later;
    later.find(a, t, key + 2 * KEYS, end, w);
    load_values(ahead, key + KEYS);
    lds_u8* const to = lds + ((s + 1) & 1) * D * ROW;
    const bool work = key < wave_hi && key + KEYS > wave_lo;   // wave-uniform
    v16f y[2];
    if (work) {
#pragma unroll
      for (int i = 0; i < 2; i++) {
#pragma unroll
        for (int j = 0; j < 16; j++) y[i][j] = 0.0f;
#pragma unroll
        for (int f = 0; f < KS; f++) {
          v8i k{};
          k.lo = __builtin_bit_cast(v4i, keys.k[i][f]);
          const int ks = (int)(keys.s[i][f >> 1] >> (8 * h));   // byte 0, or 2 for an odd f
          if (f & 1) {
            y[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k, ql[f], y[i], 4, 0, 2, ks, 0, scale - 4);
            y[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k, qh[f], y[i], 4, 0, 2, ks, 0, scale);
          } else {
            y[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k, ql[f], y[i], 4, 0, 0, ks, 0, scale - 4);
            y[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k, qh[f], y[i], 4, 0, 0, ks, 0, scale);
          }
        }
      }
    }
    keys.load(a, ahead, head, key + KEYS);   // in the registers that the products are done with
    mask_values(ahead, key + KEYS);
    if (!work) {
      store_values(to);
    } else {
      const bool all = runs.all(a);
      if (!(key >= all_lo && key + KEYS <= all_hi && all)) {
        if (!all) {
#pragma unroll
          for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < 16; j++)
              if (!runs.there(a, 2 * i + (j >> 3))) y[i][j] = -INFINITY;
        }
        const uint32_t from = (uint32_t)(key + 4 * h - lo), span = (uint32_t)max(hi - lo, 0);
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
          for (int j = 0; j < 16; j++)
            if (from + (32 * i + 8 * (j >> 2) + (j & 3)) >= span) y[i][j] = -INFINITY;
      }
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 16; j++) mx = fmaxf(mx, y[i][j]);
      const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
      mx = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])) * a.scale2;
      if (__any(mx > top + 8.0f)) {   // the maximum may be 8 too low: see kv_attention.h
        const float higher = fmaxf(mx, top);
        const float shrink = higher > -INFINITY ? __builtin_amdgcn_exp2f(top - higher) : 1.0f;
        top = higher;
        sum *= shrink;
#pragma unroll
        for (int d = 0; d < D / 32; d++) o[d] *= shrink;
      }
      const float base = top > -INFINITY ? top : 0.0f;
      const lds_u8* v = lds + (s & 1) * D * ROW + c * ROW;
      const uint32_t first = place_of(h, c >> 3, c & 7);
      u32x4 p[4];   // weights of 16 keys each
      auto weights = [&](int i) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float e0 = __builtin_amdgcn_exp2f(fmaf(y[i][2 * j], a.scale2, -base));
          const float e1 = __builtin_amdgcn_exp2f(fmaf(y[i][2 * j + 1], a.scale2, -base));
          sum += e0 + e1;
          p[2 * i + (j >> 2)][j & 3] = bf16_pair(e0, e1);
        }
      };
      auto product = [&](int f) {
#pragma unroll
        for (int d = 0; d < D / 32; d++) {
          const u32x4 vw = *reinterpret_cast<const lds_u32x4*>(v + (first ^ (32 * (f ^ (d & 1)))) + d * (32 * ROW));
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vw), __builtin_bit_cast(bf16x8, p[f]), o[d], 0, 0, 0);
        }
      };
      weights(0);
      product(0);
      product(1);
      weights(1);
      store_values(to);
      product(2);
      product(3);
    }
    runs = ahead;
    ahead = later;
    __syncthreads();
  }

  sum += __shfl_xor(sum, 32, 64);
  if (!valid) return;
  const int64_t at = token * a.heads + q_head;
  const bool some = sum > 0.0f || sum != sum;
  if (a.sums && part == 0 && h == 0) a.used[at] = used;
  if (!whole) {
    if (h == 0) {
      float* ml = a.sums + a.parts * all_rows * D + (part * all_rows + at) * 2;
      ml[0] = top;
      ml[1] = sum;
    }
    float* to = a.sums + (part * all_rows + at) * D;
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        *reinterpret_cast<v4f*>(to + 32 * d + 8 * i + 4 * h) = v4f{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
  } else {
    const float factor = some ? 1.0f / sum : 0.0f;
    if (a.lse && h == 0) a.lse[at] = some ? (top + __builtin_amdgcn_logf(sum)) * kLn2 : -INFINITY;
    uint16_t* to = a.out + at * D;
#pragma unroll
    for (int d = 0; d < D / 32; d++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        *reinterpret_cast<u32x2*>(to + 32 * d + 8 * i + 4 * h) =
            u32x2{bf16_pair(o[d][4 * i] * factor, o[d][4 * i + 1] * factor), bf16_pair(o[d][4 * i + 2] * factor, o[d][4 * i + 3] * factor)};
  }
}

template <int D, int W>
void launch(const KvCache& c, const Args& g, dim3 grid, hipStream_t stream) {
  if (c.page_size >= 32) hipLaunchKernelGGL((kv_attention_tile_kernel<D, true, W>), grid, dim3(64 * W), 0, stream, g);
  else hipLaunchKernelGGL((kv_attention_tile_kernel<D, false, W>), grid, dim3(64 * W), 0, stream, g);
}
template <int D>
void launch(const KvCache& c, const Args& g, int64_t rows, dim3 grid, hipStream_t stream) {
  if (rows == 64) launch<D, 2>(c, g, grid, stream);
  else launch<D, 4>(c, g, grid, stream);
}

}  // namespace

hipError_t launch_kv_attention_tile(const KvCache& c, const kv::Args& g, int64_t rows, dim3 grid, hipStream_t stream) {
  if (c.head_dim == 64) launch<64>(c, g, rows, grid, stream);
  else if (c.head_dim == 128) launch<128>(c, g, rows, grid, stream);
  else launch<256>(c, g, rows, grid, stream);
  return hipGetLastError();
}

}  // namespace mx
