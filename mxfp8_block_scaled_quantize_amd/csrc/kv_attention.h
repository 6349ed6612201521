// Device code shared by the two attention kernels over the paged MXFP4 cache.
//
// Rows.  The queries of a sequence and the heads that share a key-value head are
// rows of one product: row = query * group + head of the group.  A tile is some
// rows of one sequence and key-value head; its keys may be cut into parts, each for a
// workgroup, whose sums meet in the workspace (`sums`) and are joined by
// kv_join_kernel.  A launch has as many places for parts as the table's width may
// want; how many a tile really has is settled on the device, by its keys: a tile of one
// writes its outputs at once, and a workgroup without a part does nothing.
//
// Scores.  S^T = K Q^T on the scaled matrix instructions: the keys' codes go from
// the cache into the FP4 operand as they are, 32 codes and a scale byte a lane.  The
// other operand takes FP8, so a query is split: its row is divided by 2^(E - 7)
// (E: the exponent of its largest value, which lands in [128, 256)), `hi` is the
// E4M3 rounding (4 of the 8 significant bits) and `lo` that of 16 times the rest,
// which has 4 bits too: together they are the query's bits down to half of E4M3's
// smallest step of lo, 2^-14, i.e. 2^-21 of the row's largest value.  Two products
// of half the cost of a BF16 one, and no conversion of the keys.
//
// Values.  O^T = V^T P^T on the BF16 matrix instructions, as a token's values have
// scales of their own: codes and scale become BF16 (exactly).  The weights are rounded to
// BF16 for it, by 2^-8 of themselves at most; their sums are not.  The outputs are then
// 0.0023 of their norm off, of which their own rounding is 0.0017.  A second product, with
// what the rounding left of the weights, would bring 0.0017 and cost 6 % of the time with few
// rows (64 sequences of up to 8192 tokens: 71 us, not 66.5), 17 to 39 % with many (500
// queries over 49152 keys: 524 us, not 380).
//
// Maximum.  The running maximum follows the scores only when one passes it by more than 8
// (in log2), so that most steps rescale nothing.  Weights are then up to 2^8 and rounded in
// the same relation, but the weight of a row's largest score need not be 1, which BF16 holds
// exactly: an output that one key dominates carries that rounding too.  Sums overflow 2^8
// earlier; those of 2^31 keys hold values up to 2^88.
#pragma once

#include "kv.h"
#include "launch.h"
#include "mx_device.h"
#include "wave_scan.h"

namespace mx {
namespace kv {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;

// What the kernels take, of KvAttention.
struct Args {
  const uint16_t* __restrict__ q;
  int64_t q_token, q_head;
  const uint8_t* __restrict__ cache;
  int64_t record;
  uint32_t page_stride;        // bytes of a page's records, below 2^31
  const int32_t* __restrict__ table;
  int64_t ld_table;
  const int32_t* __restrict__ lengths;
  const int32_t* __restrict__ offsets;
  uint16_t* __restrict__ out;
  float* __restrict__ lse;
  float* __restrict__ sums;   // O [parts][rows][D], then (m, l) [parts][rows][2]; null: one part
  int32_t* __restrict__ used; // [rows], behind them: the parts that a row has (one: its outputs are written)
  int32_t tokens, heads, kv_heads, group, sequences, pages, page_shift, keys_most, window;
  int32_t tiles, likely;      // of the launch: as any offsets may need, as runs of max_queries have
  int32_t parts, fill;        // places for parts; parts that give the chip enough workgroups
  float scale2;               // scale * log2(e)
};

// Keys of a part: at least (a second launch joins the parts, about 3 us, in which a
// workgroup goes through 1000 keys), and at most where there are tiles enough (parts then
// bound what one very long sequence among them takes: 16384 keys are 70 us).
constexpr int LEAST_KEYS = 512, MOST_KEYS = 16384;

// Steps (of STEP keys) of a part of a tile that has `steps` > 0: as many as make `fill`
// parts, between the two bounds, or as `parts` places need.
template <int STEP>
__device__ __forceinline__ int part_steps(const Args& a, int steps) {
  if (!a.sums) return steps;
  const int even = (steps + a.fill - 1) / a.fill, room = (steps + a.parts - 1) / a.parts;
  return max(min(max(even, LEAST_KEYS / STEP), MOST_KEYS / STEP), room);
}

// The workgroup's head, tile and part.  The hardware deals workgroups out in turn, those that
// have nothing to do like the others, so that they must not stand between those with work: parts
// are the slowest (the places behind a tile's last part come at the end), and tiles past the
// likely number come behind all parts of the likely ones.
struct Place {
  int head, tile, part;
  __device__ __forceinline__ explicit Place(const Args& a) {
    unsigned rest = blockIdx.x / (unsigned)a.kv_heads;
    head = (int)(blockIdx.x % (unsigned)a.kv_heads);
    const unsigned inside = (unsigned)a.likely * (unsigned)a.parts;
    const bool first = rest < inside;
    rest = first ? rest : rest - inside;
    const unsigned run = first ? (unsigned)a.likely : (unsigned)(a.tiles - a.likely);   // not 0: the grid has it
    part = (int)(rest / run);
    tile = (int)(rest % run) + (first ? 0 : a.likely);
  }
};

struct Tile {
  int sequence, first_token, row0, rows;   // rows: of the sequence behind row0
  int queries, length;
};

// Tile `t` among the sequences' tiles of TM rows.  False: past the last one.
template <int TM>
__device__ __forceinline__ bool find_tile(const Args& a, int t, Tile* tile) {
  if (!a.offsets) {
    const int per = (a.group + TM - 1) / TM;
    const int b = t / per;
    if (b >= a.sequences) return false;
    tile->sequence = b;
    tile->first_token = b;
    tile->row0 = (t - b * per) * TM;
    tile->queries = 1;
  } else {
    const int lane = threadIdx.x & 63;
    int carry = 0;
    for (int g0 = 0;; g0 += 64) {
      if (g0 >= a.sequences) return false;
      const int g = g0 + lane;
      int lo = 0, hi = 0;
      if (g < a.sequences) {
        const int l = a.offsets[g], h = a.offsets[g + 1];
        lo = l < 0 ? 0 : (l > a.tokens ? a.tokens : l);
        hi = h < 0 ? 0 : (h > a.tokens ? a.tokens : h);
      }
      lo = lo > carry ? lo : carry;
      lo = scan64(lo, [](int x, int y) { return x > y ? x : y; });
      hi = hi > lo ? hi : lo;
      carry = __builtin_amdgcn_readlane(hi, 63);
      const int nt = (int)(((unsigned)(hi - lo) * (unsigned)a.group + TM - 1) / TM);
      const int incl = scan64(nt, [](int x, int y) { return x + y; });
      const int total = __builtin_amdgcn_readlane(incl, 63);
      if (t < total) {
        const int fl = __builtin_ctzll(__ballot(incl > t));
        tile->sequence = g0 + fl;
        tile->row0 = (t - __builtin_amdgcn_readlane(incl - nt, fl)) * TM;
        tile->first_token = __builtin_amdgcn_readlane(lo, fl);
        tile->queries = __builtin_amdgcn_readlane(hi, fl) - tile->first_token;
        break;
      }
      t -= total;
    }
  }
  tile->rows = tile->queries * a.group - tile->row0;
  const int length = __builtin_amdgcn_readfirstlane(a.lengths[tile->sequence]);
  tile->length = length < 0 ? 0 : length;
  return true;
}

// Keys [lo, hi) that query x of a tile's sequence sees, none where lo >= hi: those up to its
// place, which the sequence's length alone gives, as far as the table has them.  Both rise
// with x (hi may be negative, lo is not).
__device__ __forceinline__ void seen(const Args& a, const Tile& t, int x, int* lo, int* hi) {
  const int behind = t.length - t.queries + x + 1;
  *hi = behind < a.keys_most ? behind : a.keys_most;
  *lo = a.window > 0 && behind > a.window ? behind - a.window : 0;
}

// A page's record of a head.
__device__ __forceinline__ const uint8_t* record_of(const Args& a, int head, int page) {
  return a.cache + head * a.record + (uint64_t)(uint32_t)page * a.page_stride;
}

// Eight BF16 query values as E4M3 parts (two words each) on the scale 2^(e - 127).
// `lo` is 16 times what `hi` leaves.
__device__ __forceinline__ void split8(uint4 v, int e, uint32_t* hi, uint32_t* lo) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 2; i++) {
    int h = 0, l = 0;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const uint32_t d = w[2 * i + j];
      const float x = ldexpf(bf_lo(d), 127 - e), y = ldexpf(bf_hi(d), 127 - e);
      h = j ? __builtin_amdgcn_cvt_pk_fp8_f32(x, y, h, true) : __builtin_amdgcn_cvt_pk_fp8_f32(x, y, h, false);
      const f32x2 r = j ? __builtin_amdgcn_cvt_pk_f32_fp8(h, true) : __builtin_amdgcn_cvt_pk_f32_fp8(h, false);
      const float rx = (x - r.x) * 16.0f, ry = (y - r.y) * 16.0f;
      l = j ? __builtin_amdgcn_cvt_pk_fp8_f32(rx, ry, l, true) : __builtin_amdgcn_cvt_pk_fp8_f32(rx, ry, l, false);
    }
    hi[i] = (uint32_t)h;
    lo[i] = (uint32_t)l;
  }
}
__device__ __forceinline__ uint32_t amax8(uint4 v) {
  const uint32_t m = pk_max_u16(pk_max_u16(abs_bits2(v.x), abs_bits2(v.y)), pk_max_u16(abs_bits2(v.z), abs_bits2(v.w)));
  return max(m & 0xFFFFu, m >> 16);
}
// Scale byte of `hi` (that of `lo` is 4 less, and not below 0) for a row's amax pattern.  On the
// least, 2^-123, half of lo's smallest step is 2^-137, and BF16's smallest number 2^-133.
__device__ __forceinline__ int query_scale(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 7);
  return (e < 11 ? 11 : e > 254 ? 254 : e) - 7;
}

// Codes 2 x and 2 x + 1 of a word as a BF16 pair.
__device__ __forceinline__ uint32_t bf16_pair_of(uint32_t codes, float scale, int x) {
  const bf16x2 v = x == 0   ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0)
                   : x == 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1)
                   : x == 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2)
                            : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return __builtin_bit_cast(uint32_t, v);
}
// A token's eight codes as four words of BF16 pairs.
__device__ __forceinline__ void bf16_of(uint32_t codes, float scale, uint32_t* w) {
#pragma unroll
  for (int x = 0; x < 4; x++) w[x] = bf16_pair_of(codes, scale, x);
}
__device__ __forceinline__ float scale_of(uint32_t word, int byte) { return __uint_as_float(((word >> (8 * byte)) & 0xFFu) << 23); }

// BF16 pair (t0, t1) of the low or high halves of two words.
__device__ __forceinline__ uint32_t lows(uint32_t t0, uint32_t t1) { return __builtin_amdgcn_perm(t1, t0, 0x05040100u); }
__device__ __forceinline__ uint32_t highs(uint32_t t0, uint32_t t1) { return __builtin_amdgcn_perm(t1, t0, 0x07060302u); }

__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
  const bf16x2 h = {(__bf16)x, (__bf16)y};
  return __builtin_bit_cast(uint32_t, h);
}

}  // namespace kv

// Tiles of TM rows that any offsets can give.
inline int64_t kv_tiles(const KvAttention& a, int64_t tm) {
  const int64_t group = a.heads / a.cache.heads;
  if (!a.offsets) return a.sequences * ((group + tm - 1) / tm);
  const int64_t with = a.sequences < a.tokens ? a.sequences : a.tokens;
  return (a.tokens * group + with * (tm - 1)) / tm;
}
// rows: 64 or 128 a workgroup.
hipError_t launch_kv_attention_tile(const KvCache& c, const kv::Args& g, int64_t rows, dim3 grid, hipStream_t stream);

}  // namespace mx
