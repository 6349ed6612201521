// Mixture-of-experts kernels for gfx950: routing and its gradient, the stable
// counting sort of the (token, slot) pairs, the weighted combination of the
// experts' outputs and its gradients.
#include <type_traits>

#include "mx_device.h"
#include "launch.h"
#include "wave_scan.h"

namespace mx {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------ element types
struct Fp32 {
  typedef float T;
  static constexpr int V = 4;   // elements in 16 bytes
};
struct Bf16 {
  typedef uint16_t T;
  static constexpr int V = 8;
};
struct Fp16 {
  typedef uint16_t T;
  static constexpr int V = 8;
};

template <typename D>
__device__ __forceinline__ float to_f32(typename D::T v) {
  if constexpr (__is_same(D, Fp32)) return v;
  else if constexpr (__is_same(D, Bf16)) return __uint_as_float((uint32_t)v << 16);
  else return (float)__builtin_bit_cast(_Float16, v);
}
template <typename D>
__device__ __forceinline__ typename D::T from_f32(float v) {
  if constexpr (__is_same(D, Fp32)) return v;
  else if constexpr (__is_same(D, Bf16)) return __builtin_bit_cast(uint16_t, (__bf16)v);
  else return __builtin_bit_cast(uint16_t, (_Float16)v);
}
// 16 bytes <-> V floats
template <typename D>
__device__ __forceinline__ void unpack(u32x4 d, float* f) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (__is_same(D, Fp32)) f[i] = __uint_as_float(d[i]);
    else if constexpr (__is_same(D, Bf16)) { f[2 * i] = bf_lo(d[i]); f[2 * i + 1] = bf_hi(d[i]); }
    else {
      const f16x2 h = __builtin_bit_cast(f16x2, (uint32_t)d[i]);
      f[2 * i] = (float)h.x;
      f[2 * i + 1] = (float)h.y;
    }
  }
}
template <typename D>
__device__ __forceinline__ u32x4 pack(const float* f) {
  u32x4 d;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (__is_same(D, Fp32)) d[i] = __float_as_uint(f[i]);
    else if constexpr (__is_same(D, Bf16)) {
      const bf16x2 h = {(__bf16)f[2 * i], (__bf16)f[2 * i + 1]};
      d[i] = __builtin_bit_cast(uint32_t, h);
    } else {
      const f16x2 h = {(_Float16)f[2 * i], (_Float16)f[2 * i + 1]};
      d[i] = __builtin_bit_cast(uint32_t, h);
    }
  }
  return d;
}

// ------------------------------------------------- reductions over lane rows
// Over the aligned runs of L lanes (16, 32 or 64); every lane gets the result.
// Inside 16 lanes by DPP (lane ^ 1, lane ^ 2, mirrored halves, mirrored row),
// then by the row swaps v_permlane16_swap / v_permlane32_swap.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
template <typename X, int CTRL>
__device__ __forceinline__ X dppx(X v) {
  if constexpr (sizeof(X) == 4) return __builtin_bit_cast(X, dpp32<CTRL>(__builtin_bit_cast(uint32_t, v)));
  else {
    const u32x2 d = __builtin_bit_cast(u32x2, v);
    const u32x2 r = {dpp32<CTRL>(d.x), dpp32<CTRL>(d.y)};
    return __builtin_bit_cast(X, r);
  }
}
template <int L, typename X, typename Op>
__device__ __forceinline__ X lanes_reduce(X v, Op op) {
  v = op(v, dppx<X, 0xB1>(v));
  v = op(v, dppx<X, 0x4E>(v));
  v = op(v, dppx<X, 0x141>(v));
  v = op(v, dppx<X, 0x140>(v));
  if constexpr (L >= 32) {
    X a, b;
    if constexpr (sizeof(X) == 4) {
      const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                      false, false);
      a = __builtin_bit_cast(X, (uint32_t)r[0]);
      b = __builtin_bit_cast(X, (uint32_t)r[1]);
    } else {
      const u32x2 d = __builtin_bit_cast(u32x2, v);
      const auto r = __builtin_amdgcn_permlane16_swap(d.x, d.x, false, false);
      const auto s = __builtin_amdgcn_permlane16_swap(d.y, d.y, false, false);
      const u32x2 p = {r[0], s[0]}, q = {r[1], s[1]};
      a = __builtin_bit_cast(X, p);
      b = __builtin_bit_cast(X, q);
    }
    v = op(a, b);
  }
  if constexpr (L >= 64) {
    X a, b;
    if constexpr (sizeof(X) == 4) {
      const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v),
                                                      false, false);
      a = __builtin_bit_cast(X, (uint32_t)r[0]);
      b = __builtin_bit_cast(X, (uint32_t)r[1]);
    } else {
      const u32x2 d = __builtin_bit_cast(u32x2, v);
      const auto r = __builtin_amdgcn_permlane32_swap(d.x, d.x, false, false);
      const auto s = __builtin_amdgcn_permlane32_swap(d.y, d.y, false, false);
      const u32x2 p = {r[0], s[0]}, q = {r[1], s[1]};
      a = __builtin_bit_cast(X, p);
      b = __builtin_bit_cast(X, q);
    }
    v = op(a, b);
  }
  return v;
}
struct OpMax {
  template <typename X>
  __device__ __forceinline__ X operator()(X a, X b) const { return a > b ? a : b; }
};
struct OpMin {
  template <typename X>
  __device__ __forceinline__ X operator()(X a, X b) const { return a < b ? a : b; }
};
struct OpAdd {
  template <typename X>
  __device__ __forceinline__ X operator()(X a, X b) const { return a + b; }
};

// LDS written by some lanes of a wave and read by others of the same wave.
__device__ __forceinline__ void wave_lds_fence() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// -------------------------------------------------------------------- scores
// exp in 32 bits with the product x log2(e) kept in two parts, so that a result
// in fp32's normal range is within about 2 ulp (the plain exp2(x log2 e) loses
// |x| / 2 ulp).  Past the range it is +inf or 0, for NaN it is NaN.
__device__ __forceinline__ float exp_of(float x) {
  const float h = x * 1.44269504088896341f;
  const float l = fmaf(x, 1.92596299e-08f, fmaf(x, 1.44269504088896341f, -h));
  const float e = __builtin_amdgcn_exp2f(h);
  // from h = 128 on e is +inf, which no correction may touch (inf - inf); below
  // -128 there is nothing left to correct, and of +-inf and NaN l is undefined
  return fabsf(h) < 128.0f ? fmaf(e * l, 0.69314718055994531f, e) : e;
}
__device__ __forceinline__ float rcp_of(float x) { return __builtin_amdgcn_rcpf(x); }

// Order-preserving integers: NaN 2, -inf and up above it, +-0 the same; 1 is
// left for experts of closed groups and 0 for those that are out.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t k = b ^ (((int32_t)b >> 31) | 0x80000000u);
  return x != x ? 2u : k;
}
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x + 0.0);
  const uint64_t k = b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
  return x != x ? 2ull : k;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

template <int VPL, typename D>
__device__ __forceinline__ void load_logits(const typename D::T* __restrict__ row, int e0, int E, bool wide, float* x) {
  constexpr int V = D::V;
  if (wide && e0 + VPL <= E) {   // rows and lanes start at whole vectors of min(VPL, V) elements
    if constexpr (VPL % V == 0) {
#pragma unroll
      for (int j = 0; j < VPL / V; j++) unpack<D>(*reinterpret_cast<const u32x4*>(row + e0 + V * j), x + V * j);
    } else {   // VPL = 4 or 12 two-byte elements
#pragma unroll
      for (int j = 0; j < VPL / 4; j++) {
        const u32x2 d = *reinterpret_cast<const u32x2*>(row + e0 + 4 * j);
        const u32x4 p = {d.x, d.y, 0u, 0u};
        float f[8];
        unpack<D>(p, f);
#pragma unroll
        for (int i = 0; i < 4; i++) x[4 * j + i] = f[i];
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; j++) x[j] = e0 + j < E ? to_f32<D>(row[e0 + j]) : -INFINITY;
  }
}

// Scores of the lane's experts (those past E: 0).
template <int LPR, int VPL>
__device__ __forceinline__ void scores_of(const float* x, bool sigmoid, float* s) {
  if (sigmoid) {
#pragma unroll
    for (int j = 0; j < VPL; j++) s[j] = rcp_of(1.0f + exp_of(-x[j]));
    return;
  }
  float m = x[0];
#pragma unroll
  for (int j = 1; j < VPL; j++) m = fmaxf(m, x[j]);
  m = lanes_reduce<LPR>(m, OpMax{});
  if (m == -INFINITY) m = 0.0f;   // a row of -inf alone: every exp is 0
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; j++) {
    s[j] = exp_of(x[j] - m);
    sum += s[j];
  }
  sum = lanes_reduce<LPR>(sum, OpAdd{});
  const float r = sum == 0.0f ? 0.0f : rcp_of(sum);
#pragma unroll
  for (int j = 0; j < VPL; j++) s[j] *= r;
}

constexpr int kMaxGroups = 64, kMaxTopK = 64;

struct RouteArgs {
  int E, K, groups, top_groups, group_top, per;
  int group_lanes;   // lanes that hold a group and nothing else (1, 2, 4, 8, 16); 0: groups do not end with lanes
  bool sigmoid, renorm, wide, wide_bias;
  const float* bias;
};

// The two largest of a lane's values and of another lane's.
struct Top2 {
  float m1, m2;
  __device__ __forceinline__ void add(float v) {
    v = v == v ? v : -INFINITY;   // NaN is last
    m2 = __builtin_amdgcn_fmed3f(m1, m2, v);
    m1 = fmaxf(m1, v);
  }
  __device__ __forceinline__ void merge(float o1, float o2) {
    m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
    m1 = fmaxf(m1, o1);
  }
  template <int CTRL>
  __device__ __forceinline__ void merge_dpp() {
    merge(dppx<float, CTRL>(m1), dppx<float, CTRL>(m2));
  }
};

// How many of `n` group values (padded with -inf to a multiple of four) come
// before group g with value v: the larger ones, and equal ones of lower index.
__device__ __forceinline__ int rank_of(const float* gval, int n, int g, float v) {
  int rank = 0;
  for (int h0 = 0; h0 < n; h0 += 4) {
    const float4 o = *reinterpret_cast<const float4*>(gval + h0);
    rank += (o.x > v || (o.x == v && h0 < g)) + (o.y > v || (o.y == v && h0 + 1 < g)) +
            (o.z > v || (o.z == v && h0 + 2 < g)) + (o.w > v || (o.w == v && h0 + 3 < g));
  }
  return rank;
}

// LDS of a row: a score (before that: choice) per expert, then the groups'
// values and who is open, and in their place the picks.
template <int LPR, int VPL>
struct RouteLds {
  static constexpr int NV = LPR * VPL;
  static constexpr int PICKS = (kMaxTopK + 2) * 8;
  static constexpr int ROW = NV * 4 + (PICKS > kMaxGroups * 8 ? PICKS : kMaxGroups * 8);
  static constexpr int EXACT = NV * 8 + kMaxGroups * 12 + kMaxTopK * 4;   // of a wave that chooses again
  static constexpr int ROWS = 64 / LPR * ROW;
  static constexpr int WAVE = ((ROWS > EXACT ? ROWS : EXACT) + 15) / 16 * 16;
};

// One row on LPR lanes, lane l holding experts l VPL .. + VPL - 1.  SURE: the
// order is the logits' own.  Else the choice is made in 32 bits, and nothing is
// written for a row in which two values that matter are closer than what they
// can be off by (returned for all its lanes):
//   u = 2^-24.  exp_of is within 4 u of its value, rcp_of within 2 u (or both
//   are 0 or +inf for a score below 2^-126, far less than any of these bounds).
//   softmax  a score s is within (18 + VPL) u s: 4 u of its own exp, 4 u of the
//            sum's terms, (VPL + 6) u of adding them up, 3 u of 1 / sum and the
//            product, and the rounding of x - max, |d| e^-|d| u <= 0.4 u.  The
//            scores of two experts add up to 1 at most, and to twice the
//            largest (of two pairs: four times).
//   sigmoid  e / (1 + e)^2 4 u + 3 u s <= 4 u, two of them 8 u, two pairs 16 u.
//   each sum with the bias, and of two choices, rounds by u of its value more.
template <int LPR, int VPL, bool SURE>
__device__ __forceinline__ bool route_row(const RouteArgs& a, const float* x, const float* bias, int l, char* lds, float* __restrict__ w_out,
                                          int32_t* __restrict__ id_out, bool live) {
  constexpr float U = 5.9604645e-8f;
  float* const vals = reinterpret_cast<float*>(lds);                  // [LPR * VPL]
  float* const gval = vals + LPR * VPL;                               // [64]
  uint32_t* const keep = reinterpret_cast<uint32_t*>(gval + kMaxGroups);
  u32x2* const pick = reinterpret_cast<u32x2*>(gval);                 // [66] (expert, key), after the groups are done
  const int e0 = l * VPL;
  const int seg = (threadIdx.x & 63) & ~(LPR - 1);
  bool doubt = false;
  float s[VPL], v[VPL];
  scores_of<LPR, VPL>(x, a.sigmoid, s);
  uint32_t key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; j++) {
    v[j] = SURE ? x[j] : s[j] + bias[j];
    key[j] = e0 + j >= a.E ? 0 : key_of(SURE || !a.bias ? x[j] : v[j]);
  }
  float largest = 1.0f;   // score of the row
  if (!SURE && !a.sigmoid) {
    largest = s[0];
#pragma unroll
    for (int j = 1; j < VPL; j++) largest = fmaxf(largest, s[j]);
    largest = lanes_reduce<LPR>(largest, OpMax{});
  }
  if (a.groups > 1) {
    // the value of a group comes from the choices; with group_top 1 and no
    // bias the largest logit says the same
    const bool two = a.group_top == 2 && a.per > 1;
    const float off = a.sigmoid ? 8 * U : (9 + VPL / 2) * U * fminf(1.0f, 4.0f * largest);   // of one group
    auto value = [&](const Top2& t) {
      const float v = two ? t.m1 + t.m2 : t.m1;
      return v == v ? v : -INFINITY;   // inf - inf
    };
    auto error = [&](const Top2& t) { return off + 2 * U * (fabsf(t.m1) + (two ? fabsf(t.m2) : 0.0f)); };
    // biases next to the type's largest or lowest value: a sum that 32 bits do
    // not hold says nothing about its place among the others of its kind
    auto overflow = [&](const Top2& t) {
      return two && fabsf(t.m1) < INFINITY && fabsf(t.m2) < INFINITY && fabsf(t.m1 + t.m2) == INFINITY;
    };
    bool past = false;
    float low = INFINITY, high = -INFINITY;   // smallest an open group may be, largest a closed one
    if (l < 4 && a.groups + l < kMaxGroups) gval[a.groups + l] = -INFINITY;
    if (a.group_lanes) {   // in registers
      Top2 t{-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < VPL; j++) t.add(v[j]);
      if (a.group_lanes > 1) t.merge_dpp<0xB1>();
      if (a.group_lanes > 2) t.merge_dpp<0x4E>();
      if (a.group_lanes > 4) t.merge_dpp<0x141>();
      if (a.group_lanes > 8) t.merge_dpp<0x140>();
      const int g = l / a.group_lanes;
      const float mine = value(t);
      past = overflow(t);
      if (g < a.groups && (l & (a.group_lanes - 1)) == 0) gval[g] = mine;
      wave_lds_fence();
      const bool open = rank_of(gval, a.groups, g, mine) < a.top_groups;
      if (g < a.groups) {
        if (open) low = mine - error(t);
        else high = mine + error(t);
      }
#pragma unroll
      for (int j = 0; j < VPL; j++)
        if (!open && e0 + j < a.E) key[j] = 1;
    } else {               // through LDS
#pragma unroll
      for (int j = 0; j < VPL; j++) vals[e0 + j] = v[j];
      wave_lds_fence();
      int lg = 1;   // lanes per group, 16 at most
      while (lg < 16 && 2 * lg * a.groups <= LPR) lg *= 2;
      for (int g0 = 0; g0 < a.groups; g0 += LPR / lg) {
        const int g = g0 + l / lg;
        Top2 t{-INFINITY, -INFINITY};
        if (g < a.groups)
#pragma unroll 4
          for (int i = l & (lg - 1); i < a.per; i += lg) t.add(vals[g * a.per + i]);
        if (lg > 1) t.merge_dpp<0xB1>();
        if (lg > 2) t.merge_dpp<0x4E>();
        if (lg > 4) t.merge_dpp<0x141>();
        if (lg > 8) t.merge_dpp<0x140>();
        if (g < a.groups && (l & (lg - 1)) == 0) {
          gval[g] = value(t);
          keep[g] = __float_as_uint(error(t));
          past = past || overflow(t);
        }
      }
      wave_lds_fence();
      for (int g = l; g < a.groups; g += LPR) {
        const float mine = gval[g], e = __uint_as_float(keep[g]);
        const bool open = rank_of(gval, a.groups, g, mine) < a.top_groups;
        keep[g] = open;
        if (open) low = fminf(low, mine - e);
        else high = fmaxf(high, mine + e);
      }
      wave_lds_fence();
      int g = e0 / a.per, next = (g + 1) * a.per;
      uint32_t open = g < a.groups ? keep[g] : 0;
#pragma unroll
      for (int j = 0; j < VPL; j++) {
        if (e0 + j == next) {
          g++;
          next += a.per;
          open = g < a.groups ? keep[g] : 0;
        }
        if (!open && e0 + j < a.E) key[j] = 1;
      }
    }
    if (!SURE) {   // an infinite choice leaves NaN, which says nothing: infinities are equal in 64 bits too
      low = lanes_reduce<LPR>(fminf(low, INFINITY), OpMin{});
      high = lanes_reduce<LPR>(fmaxf(high, -INFINITY), OpMax{});
      doubt = past || low < high;
    }
    wave_lds_fence();
  }
#pragma unroll
  for (int j = 0; j < VPL; j++) vals[e0 + j] = s[j];
  // top_k rounds of the largest key, ties to the lowest lane and then the
  // lowest register, i.e. the lowest expert; one more round says how far the
  // first one left out is.
  const bool check = !SURE && a.bias;
  const int rounds = check && a.K < a.E ? a.K + 1 : a.K;
  for (int k = 0; k < rounds; k++) {
    uint32_t lm = key[0];
#pragma unroll
    for (int j = 1; j < VPL; j++) lm = key[j] > lm ? key[j] : lm;
    const uint32_t m = lanes_reduce<LPR>(lm, OpMax{});
    uint64_t who = __ballot(lm == m) >> seg;
    if (LPR < 64) who &= ((uint64_t)1 << (LPR & 63)) - 1;
    if (l == (int)__builtin_ctzll(who)) {
      int at = 0;
#pragma unroll
      for (int j = VPL - 1; j >= 0; j--) at = key[j] == m ? j : at;
#pragma unroll
      for (int j = 0; j < VPL; j++) key[j] = j == at ? 0 : key[j];
      pick[k] = u32x2{(uint32_t)(e0 + at), m};
    }
  }
  wave_lds_fence();
  if (check) {
    const float off = a.sigmoid ? 8 * U : (18 + VPL) * U * fminf(1.0f, 2.0f * largest);
    for (int k = l; k + 1 < rounds; k += LPR) {
      const uint32_t k0 = pick[k].y, k1 = pick[k + 1].y;
      const float v0 = value_of(k0), v1 = value_of(k1);
      doubt = doubt || (k1 > 2 && v0 - v1 <= off + 2 * U * fmaxf(fabsf(v0), fabsf(v1)));
    }
  }
  if constexpr (!SURE) {
    uint64_t any = __ballot(doubt) >> seg;
    if (LPR < 64) any &= ((uint64_t)1 << (LPR & 63)) - 1;
    doubt = any != 0;
  }
  float total = 0.0f;
  if (a.renorm) {
    for (int k = l; k < a.K; k += LPR) total += vals[pick[k].x];
    total = lanes_reduce<LPR>(total, OpAdd{});
  }
  const float r = a.renorm ? 1.0f / (total + 1e-20f) : 1.0f;
  if (live && !doubt)
    for (int k = l; k < a.K; k += LPR) {
      const int e = (int)pick[k].x;
      w_out[k] = vals[e] * r;
      id_out[k] = e;
    }
  wave_lds_fence();
  return doubt;
}

// One row again in 64 bits, on a whole wave: lane l holds experts l N .. + N - 1.
// The kernel waits for the last such row, so it is made short: one exp per
// expert (in a loop that turns the registers, as the code is fetched for it
// alone), groups by several lanes each, rounds on the keys' upper words.
template <int N, typename D>
__device__ __forceinline__ void route_exact(const RouteArgs& a, const typename D::T* __restrict__ row, char* lds,
                                            float* __restrict__ w_out, int32_t* __restrict__ id_out) {
  double* const vals = reinterpret_cast<double*>(lds);              // [64 N] choices, then scores
  double* const gval = vals + 64 * N;                               // [64]
  uint32_t* const keep = reinterpret_cast<uint32_t*>(gval + kMaxGroups);
  int32_t* const picked = reinterpret_cast<int32_t*>(keep + kMaxGroups);
  const int lane = threadIdx.x & 63, e0 = lane * N;
  float x[N], b[N];
#pragma unroll
  for (int j = 0; j < N; j++) {
    x[j] = e0 + j < a.E ? to_f32<D>(row[e0 + j]) : -INFINITY;
    b[j] = a.bias && e0 + j < a.E ? a.bias[e0 + j] : 0.0f;
  }
  float m = x[0];
#pragma unroll
  for (int j = 1; j < N; j++) m = fmaxf(m, x[j]);
  m = lanes_reduce<64>(m, OpMax{});
  if (m == -INFINITY) m = 0.0f;
  double s[N];
#pragma unroll 1
  for (int i = 0; i < N; i++) {
    const float first = x[0];
    double t = exp(a.sigmoid ? -(double)first : (double)first - (double)m);
    if (a.sigmoid) t = 1.0 / (1.0 + t);
#pragma unroll
    for (int j = 0; j + 1 < N; j++) {
      x[j] = x[j + 1];
      s[j] = s[j + 1];
    }
    x[N - 1] = first;
    s[N - 1] = t;
  }
  if (!a.sigmoid) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < N; j++) sum += s[j];
    sum = lanes_reduce<64>(sum, OpAdd{});
    const double r = sum == 0.0 ? 0.0 : 1.0 / sum;
#pragma unroll
    for (int j = 0; j < N; j++) s[j] *= r;
  }
  // without a bias the order is the logits' own
  uint64_t key[N];
#pragma unroll
  for (int j = 0; j < N; j++) key[j] = e0 + j >= a.E ? 0 : key_of(a.bias ? s[j] + (double)b[j] : (double)x[j]);
  if (a.groups > 1) {
#pragma unroll
    for (int j = 0; j < N; j++) vals[e0 + j] = s[j] + (double)b[j];
    wave_lds_fence();
    int lg = 1;   // lanes per group, 16 at most
    while (lg < 16 && 2 * lg * a.groups <= 64) lg *= 2;
    const int mine = lane / lg;
    double m1 = -INFINITY, m2 = -INFINITY;
    auto add = [&](double v1, double v2) {   // v1 >= v2
      const double less = v1 > m1 ? m1 : v1;
      m1 = v1 > m1 ? v1 : m1;
      m2 = v2 > m2 ? v2 : m2;
      m2 = less > m2 ? less : m2;
    };
    if (mine < a.groups)
#pragma unroll 2
      for (int i = lane & (lg - 1); i < a.per; i += lg) add(vals[mine * a.per + i], -INFINITY);
    if (lg > 1) add(dppx<double, 0xB1>(m1), dppx<double, 0xB1>(m2));
    if (lg > 2) add(dppx<double, 0x4E>(m1), dppx<double, 0x4E>(m2));
    if (lg > 4) add(dppx<double, 0x141>(m1), dppx<double, 0x141>(m2));
    if (lg > 8) add(dppx<double, 0x140>(m1), dppx<double, 0x140>(m2));
    if (mine < a.groups && (lane & (lg - 1)) == 0) {
      const double v = a.group_top == 2 && a.per > 1 ? m1 + m2 : m1;
      gval[mine] = v == v ? v : -INFINITY;   // inf - inf
    }
    wave_lds_fence();
    if (lane < a.groups) {
      const double v = gval[lane];
      int rank = 0;
#pragma unroll 4
      for (int h = 0; h < a.groups; h++) {
        const double o = gval[h];
        rank += o > v || (o == v && h < lane);
      }
      keep[lane] = rank < a.top_groups;
    }
    wave_lds_fence();
#pragma unroll
    for (int j = 0; j < N; j++)
      if (e0 + j < a.E && !keep[(e0 + j) / a.per]) key[j] = 1;
  }
#pragma unroll
  for (int j = 0; j < N; j++) vals[e0 + j] = s[j];
#pragma unroll 1
  for (int k = 0; k < a.K; k++) {
    uint64_t best = key[0];
#pragma unroll
    for (int j = 1; j < N; j++) best = key[j] > best ? key[j] : best;
    const uint32_t hi = (uint32_t)(best >> 32), top = lanes_reduce<64>(hi, OpMax{});
    uint64_t who = __ballot(hi == top);
    if (who & (who - 1)) {   // several lanes: by the lower words
      const uint32_t lo = hi == top ? (uint32_t)best : 0;
      const uint32_t low = lanes_reduce<64>(lo, OpMax{});
      who = __ballot(hi == top && lo == low);
    }
    if (lane == (int)__builtin_ctzll(who)) {
      int at = 0;
#pragma unroll
      for (int j = N - 1; j >= 0; j--) at = key[j] == best ? j : at;
#pragma unroll
      for (int j = 0; j < N; j++) key[j] = j == at ? 0 : key[j];
      picked[k] = e0 + at;
    }
  }
  wave_lds_fence();
  const int id = lane < a.K ? picked[lane] : 0;
  const double mine = lane < a.K ? vals[id] : 0.0;
  const double total = lanes_reduce<64>(mine, OpAdd{});
  if (lane < a.K) {
    w_out[lane] = (float)(a.renorm ? mine / (total + 1e-20) : mine);
    id_out[lane] = id;
  }
  wave_lds_fence();
}

// A wave holds 64 / LPR rows.  The choice is made in 32 bits; a row in which
// the order of two values is within the rounding (one in a few thousand with a
// bias) is chosen again in 64, which the kernel then waits 2.5 us for.  Bound by
// the rounds' latency for few rows (16 tokens, 256 experts, top 8: 3.1 us, 4.6
// with a bias and 8 groups) and by their instructions for many (16384 tokens, 128
// experts, top 8: softmax 6.1 us for 5 MB, 9.1 with a bias, sigmoid 5.8 and 7.1;
// 0.35 a round).
template <typename D, int LPR, int VPL, bool SURE>
__global__ __launch_bounds__(256) void moe_route_kernel(const typename D::T* __restrict__ logits, int64_t T, int64_t ld,
                                                        RouteArgs a, float* __restrict__ weights,
                                                        int32_t* __restrict__ ids) {
  typedef RouteLds<LPR, VPL> L;
  constexpr int ROWS = 256 / LPR, WROWS = 64 / LPR;
  constexpr int WAVE = SURE ? L::ROWS : L::WAVE;
  __shared__ __attribute__((aligned(16))) char lds[4][WAVE];
  const int l = threadIdx.x & (LPR - 1);
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t first = (int64_t)blockIdx.x * ROWS + w * WROWS;   // the wave's rows
  const int sub = (threadIdx.x & 63) / LPR;
  const int64_t t = first + sub;
  const bool live = t < T;   // rows past the end repeat the last one and write nothing
  const int64_t tr = live ? t : T - 1;
  float x[VPL];
  float bias[VPL];   // with the logits, so that one latency covers both
#pragma unroll
  for (int j = 0; j < VPL; j++) bias[j] = 0.0f;
  if (!SURE && a.bias) load_logits<VPL, Fp32>(a.bias, l * VPL, a.E, a.wide_bias, bias);
  load_logits<VPL, D>(logits + tr * ld, l * VPL, a.E, a.wide, x);
  const bool doubt =
      route_row<LPR, VPL, SURE>(a, x, bias, l, lds[w] + sub * L::ROW, weights + tr * a.K, ids + tr * a.K, live);
  if constexpr (!SURE) {
    uint64_t again = __ballot(doubt && live && l == 0);
#pragma unroll 1
    while (again) {
      const int64_t row = first + __builtin_ctzll(again) / LPR;
      again &= again - 1;
      route_exact<L::NV / 64, D>(a, logits + row * ld, lds[w], weights + row * a.K, ids + row * a.K);
    }
  }
}

// d logits of a row: with g' = dw of the chosen experts (renormalized weights:
// (g - <g, w>) / total), softmax d_j = s_j (g'_j - <g', s>), sigmoid
// d_j = g'_j s_j (1 - s_j) with s (1 - s) = e / (1 + e)^2, e = exp(-|x|).  Who is
// chosen goes through LDS, so that a lane looks at its own experts alone.  16384
// tokens, 128 experts: 6.0 us for 9 MB.
template <typename D, int LPR, int VPL>
__global__ __launch_bounds__(256) void moe_route_backward_kernel(const typename D::T* __restrict__ logits, int64_t T,
                                                                 int64_t ld, RouteArgs a,
                                                                 const int32_t* __restrict__ ids,
                                                                 const float* __restrict__ dw,
                                                                 typename D::T* __restrict__ out, bool wide_out) {
  constexpr int ROWS = 256 / LPR;
  __shared__ __attribute__((aligned(16))) uint16_t slot_of[ROWS][LPR * VPL];
  const int l = threadIdx.x & (LPR - 1);
  const int sub = threadIdx.x / LPR;
  const int64_t t = (int64_t)blockIdx.x * ROWS + sub;
  const bool live = t < T;
  const int64_t tr = live ? t : T - 1;
  const int e0 = l * VPL;
  float x[VPL];
  load_logits<VPL, D>(logits + tr * ld, e0, a.E, a.wide, x);
  uint16_t* slot = slot_of[sub];
#pragma unroll
  for (int j = 0; j < VPL; j++) slot[e0 + j] = 0;
  wave_lds_fence();
  for (int k = l; k < a.K; k += LPR) {
    const int e = ids[tr * a.K + k];
    if (e >= 0 && e < a.E) slot[e] = (uint16_t)(k + 1);
  }
  wave_lds_fence();
  float s[VPL], g[VPL];
  scores_of<LPR, VPL>(x, a.sigmoid, s);
  uint32_t chosen = 0;
  float total = 0.0f, gs = 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; j++) {
    const int k = slot[e0 + j];
    g[j] = k ? dw[tr * a.K + k - 1] : 0.0f;
    if (k) {
      chosen |= 1u << j;
      total += s[j];
      gs += g[j] * s[j];
    }
  }
  float dot = lanes_reduce<LPR>(gs, OpAdd{});
  if (a.renorm) {
    total = lanes_reduce<LPR>(total, OpAdd{}) + 1e-20f;
    const float r = 1.0f / total;
    const float gw = dot * r;
    gs = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; j++)
      if ((chosen >> j) & 1) {
        g[j] = (g[j] - gw) * r;
        gs += g[j] * s[j];
      }
    if (!a.sigmoid) dot = lanes_reduce<LPR>(gs, OpAdd{});
  }
#pragma unroll
  for (int j = 0; j < VPL; j++) {
    if (a.sigmoid) {
      const float e = exp_of(-fabsf(x[j]));
      const float q = rcp_of(1.0f + e);
      g[j] = ((chosen >> j) & 1) ? g[j] * (e * q * q) : 0.0f;
    } else {
      g[j] = s[j] * (g[j] - dot);
    }
  }
  if (!live) return;
  typename D::T* row = out + tr * a.E;
  constexpr int V = D::V;
  if (wide_out && e0 + VPL <= a.E) {
    if constexpr (VPL % V == 0) {
#pragma unroll
      for (int j = 0; j < VPL / V; j++) *reinterpret_cast<u32x4*>(row + e0 + V * j) = pack<D>(g + V * j);
    } else {
#pragma unroll
      for (int j = 0; j < VPL / 4; j++) {
        const float f[8] = {g[4 * j], g[4 * j + 1], g[4 * j + 2], g[4 * j + 3], 0.f, 0.f, 0.f, 0.f};
        const u32x4 d = pack<D>(f);
        *reinterpret_cast<u32x2*>(row + e0 + 4 * j) = u32x2{d.x, d.y};
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; j++)
      if (e0 + j < a.E) row[e0 + j] = from_f32<D>(g[j]);
  }
}

// Lanes per row and experts per lane: the fewest lanes whose registers hold
// the row (fewer lanes: more rows share a wave's selection rounds), but where a
// row per wave still leaves SIMDs without one, the most (fewer experts per lane:
// each round is shorter).
constexpr int64_t kFewRows = 512;
#define MOE_ROUTE_SHAPE(CALL)            \
  do {                                   \
    if (T <= kFewRows && a.E > 64) {     \
      if (a.E <= 256) CALL(64, 4);       \
      else if (a.E <= 512) CALL(64, 8);  \
      else CALL(64, 16);                 \
    } else if (a.E <= 64) CALL(16, 4);   \
    else if (a.E <= 128) CALL(16, 8);    \
    else if (a.E <= 256) CALL(32, 8);    \
    else if (a.E <= 384) CALL(32, 12);   \
    else CALL(64, 16);                   \
  } while (0)

static RouteArgs route_args(int64_t E, int32_t K, int32_t groups, int32_t top_groups, int32_t group_top, bool sigmoid,
                            bool renorm, const float* bias) {
  RouteArgs a;
  a.E = (int)E;
  a.K = K;
  a.groups = top_groups == groups ? 1 : groups;   // every group open: no groups
  a.top_groups = top_groups;
  a.group_top = group_top;
  a.per = (int)(E / groups);
  a.group_lanes = 0;
  a.sigmoid = sigmoid;
  a.renorm = renorm;
  a.wide = false;
  a.wide_bias = reinterpret_cast<uintptr_t>(bias) % 16 == 0;
  a.bias = bias;
  return a;
}

// Lanes of vpl experts that hold one group, where that is a power of two up to
// a DPP row (16384 tokens, 128 experts: 8 groups add 1.0 us, through LDS 2.2).
static int lanes_of_group(const RouteArgs& a, int vpl) {
  const int n = a.per % vpl ? 0 : a.per / vpl;
  return n <= 16 && (n & (n - 1)) == 0 ? n : 0;
}

// Whether rows of stride ld and lanes of vpl (a multiple of 4) can be read in
// whole vectors: 16 bytes, or the 8 of four two-byte elements.
static bool wide_rows(const void* p, int64_t ld, int esize, int vpl) {
  const int unit = esize == 4 ? 16 : vpl % 8 ? 8 : 16;
  return reinterpret_cast<uintptr_t>(p) % unit == 0 && (ld * esize) % unit == 0;
}

template <typename D>
static hipError_t route_t(const void* logits, int64_t T, int64_t ld, RouteArgs a, float* weights, int32_t* ids,
                          hipStream_t stream) {
  const auto* x = static_cast<const typename D::T*>(logits);
  const bool sure = !a.bias && (a.groups == 1 || a.group_top == 1 || a.per == 1);
#define MOE_CALL(L, V)                                                                                               \
  do {                                                                                                               \
    const unsigned grid = (unsigned)((T + 256 / L - 1) / (256 / L));                                                 \
    a.wide = wide_rows(logits, ld, sizeof(typename D::T), V);                                                        \
    a.group_lanes = lanes_of_group(a, V);                                                                            \
    if (sure)                                                                                                        \
      hipLaunchKernelGGL((moe_route_kernel<D, L, V, true>), dim3(grid), dim3(256), 0, stream, x, T, ld, a, weights, ids); \
    else                                                                                                             \
      hipLaunchKernelGGL((moe_route_kernel<D, L, V, false>), dim3(grid), dim3(256), 0, stream, x, T, ld, a, weights, ids); \
  } while (0)
  MOE_ROUTE_SHAPE(MOE_CALL);
#undef MOE_CALL
  return hipGetLastError();
}

template <typename D>
static hipError_t route_back_t(const void* logits, int64_t T, int64_t ld, RouteArgs a, const int32_t* ids,
                               const float* dw, void* dlogits, hipStream_t stream) {
  const auto* x = static_cast<const typename D::T*>(logits);
  auto* o = static_cast<typename D::T*>(dlogits);
#define MOE_CALL(L, V)                                                                                             \
  do {                                                                                                             \
    a.wide = wide_rows(logits, ld, sizeof(typename D::T), V);                                                      \
    hipLaunchKernelGGL((moe_route_backward_kernel<D, L, V>), dim3((unsigned)((T + 256 / L - 1) / (256 / L))), dim3(256), \
                       0, stream, x, T, ld, a, ids, dw, o, wide_rows(dlogits, a.E, sizeof(typename D::T), V));    \
  } while (0)
  MOE_ROUTE_SHAPE(MOE_CALL);
#undef MOE_CALL
  return hipGetLastError();
}

bool moe_route_grid_fits(int64_t T) { return grid_fits((T + 3) / 4, 1, 256); }

hipError_t launch_moe_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, const float* bias, int32_t K,
                            int32_t groups, int32_t top_groups, int32_t group_top, bool sigmoid, bool renorm,
                            float* weights, int32_t* ids, hipStream_t stream) {
  const RouteArgs a = route_args(E, K, groups, top_groups, group_top, sigmoid, renorm, bias);
  return dtype == 0 ? route_t<Fp32>(logits, T, ld, a, weights, ids, stream)
       : dtype == 1 ? route_t<Bf16>(logits, T, ld, a, weights, ids, stream)
                    : route_t<Fp16>(logits, T, ld, a, weights, ids, stream);
}

hipError_t launch_moe_route_backward(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld, const int32_t* ids,
                                     const float* dw, int32_t K, bool sigmoid, bool renorm, void* dlogits,
                                     hipStream_t stream) {
  const RouteArgs a = route_args(E, K, 1, 1, 1, sigmoid, renorm, nullptr);
  return dtype == 0 ? route_back_t<Fp32>(logits, T, ld, a, ids, dw, dlogits, stream)
       : dtype == 1 ? route_back_t<Bf16>(logits, T, ld, a, ids, dw, dlogits, stream)
                    : route_back_t<Fp16>(logits, T, ld, a, ids, dw, dlogits, stream);
}

// ------------------------------------------------------------------ dispatch
// Stable counting sort.  A workgroup owns a run of slots, each of its 8 or 16
// waves a part of that run.  A wave counts its part per expert in LDS; with the
// totals of the workgroups before it (and of all experts before this one) the
// count becomes the next free row of (wave, expert), and the wave walks its
// part 64 slots at a time: lanes of the same expert find each other with one
// ballot per bit of the id, a lane's rank is the number of such lanes below
// it, and the last of them moves the counter on.  Nothing depends on the order
// of waves or workgroups.  Up to kOneBlock slots a single workgroup does it
// all.  Up to kOneLaunch every workgroup counts the other runs itself (16384
// slots: 7.7 us, with a launch of counts before it 8.2 and the host's 2.7; 32768:
// 10.7 and 8.3).  Beyond that a first launch leaves every run's counts in the
// workspace and each workgroup of the second adds up what it needs of them (at
// most 256 runs, so that this stays a few hundred KB of L2 reads).  A few MB at
// most: latency decides, so ids are loaded four 64-slot pieces at a time and the
// first batch stays in registers between counting and placing.  128 slots: 2.8
// us; 4096: 5.6 (with eight waves 7.4); 131064: 2.7 + 6.6 us, of which 2 are the
// counts of all runs coming back from behind the other XCDs' L2, 1.5 the ranks
// (two or sixteen waves, 1024 or 4096 slots a run: within 5 %).
// Ids outside [0, E) are counted as expert E, whose rows come last.
constexpr int DW = 8;                    // waves
constexpr int DB = 4;                    // 64-slot pieces in a batch
constexpr int64_t kRun = 64 * DW * DB;   // slots of a workgroup with one batch a wave
constexpr int64_t kOneBlock = 2 * kRun;
constexpr int64_t kOneLaunch = 4 * kOneBlock;
constexpr int64_t kMaxRuns = 256;

__device__ __forceinline__ int bucket_of(int id, int E) { return id >= 0 && id < E ? id : E; }

__global__ __launch_bounds__(64 * DW) void moe_count_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t run, int E,
                                                            int32_t* __restrict__ counts) {
  extern __shared__ int32_t hist[];   // [E + 1]
  for (int e = threadIdx.x; e <= E; e += 64 * DW) hist[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * run, hi = lo + run < n ? lo + run : n;
  for (int64_t i0 = lo + threadIdx.x; i0 < hi; i0 += kRun) {
    int id[DB];
#pragma unroll
    for (int b = 0; b < DB; b++) id[b] = i0 + 64 * DW * b < hi ? ids[i0 + 64 * DW * b] : 0;
#pragma unroll
    for (int b = 0; b < DB; b++)
      if (i0 + 64 * DW * b < hi) atomicAdd(&hist[bucket_of(id[b], E)], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += 64 * DW) counts[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
}

template <bool ONE, int W>
__global__ __launch_bounds__(64 * W) void moe_place_kernel(const int32_t* __restrict__ ids, int64_t n, int64_t run, int E,
                                                            int32_t top_k, int bits, int runs,
                                                            const int32_t* __restrict__ counts,
                                                            int32_t* __restrict__ offsets, int32_t* __restrict__ token,
                                                            int32_t* __restrict__ position) {
  // next row of (wave, expert) [W][E + 1]; of all runs the total and of the
  // runs before this one the count per expert [E + 1] each
  extern __shared__ int32_t next[];
  __shared__ int32_t wave_sum[W];
  int32_t* const total = next + W * (E + 1);   // not with ONE
  int32_t* const before = total + (E + 1);
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t lo = blockIdx.x * run, hi = lo + run < n ? lo + run : n;
  const int64_t part = run / W;      // a multiple of a piece
  const int64_t plo = lo + w * part;
  const int64_t phi = plo + part < hi ? plo + part : hi;
  int first[DB];                      // the wave's first batch
#pragma unroll
  for (int b = 0; b < DB; b++) first[b] = plo + 64 * b + lane < phi ? bucket_of(ids[plo + 64 * b + lane], E) : 0;
  for (int i = tid; i < (ONE ? W : W + 2) * (E + 1); i += 64 * W) next[i] = 0;
  __syncthreads();
  if (!ONE && !counts) {   // every workgroup counts all other runs itself
    for (int64_t i0 = tid; i0 < n; i0 += 64 * W * 8) {
      int id[8];
#pragma unroll
      for (int b = 0; b < 8; b++) id[b] = i0 + 64 * W * b < n ? bucket_of(ids[i0 + 64 * W * b], E) : 0;
#pragma unroll
      for (int b = 0; b < 8; b++) {
        const int64_t i = i0 + 64 * W * b;
        if (i < n && (i < lo || i >= hi)) atomicAdd(&(i < lo ? before : total)[id[b]], 1);
      }
    }
  } else if (!ONE) {
    // threads in groups of a whole number of waves, each for every q-th run
    const int width = (E + 64) / 64 * 64;
    const int groups = width <= 64 * W ? 64 * W / width : 1;
    const int q = width <= 64 * W ? tid / width : 0;
    if (q < groups)
      for (int e = tid - q * width; e <= E; e += groups > 1 ? width : 64 * W) {
        int32_t all = 0, mine = 0;
        for (int r0 = q; r0 < runs; r0 += 32 * groups) {   // 32 loads under one latency
          int32_t c[32];
#pragma unroll
          for (int i = 0; i < 32; i++) c[i] = r0 + i * groups < runs ? counts[(int64_t)(r0 + i * groups) * (E + 1) + e] : 0;
#pragma unroll
          for (int i = 0; i < 32; i++) {
            all += c[i];
            mine += r0 + i * groups < (int)blockIdx.x ? c[i] : 0;
          }
        }
        atomicAdd(&total[e], all);
        atomicAdd(&before[e], mine);
      }
  }
  int32_t* const row = next + w * (E + 1);
  for (int64_t i0 = plo; i0 < phi; i0 += 64 * DB) {
    int id[DB];
#pragma unroll
    for (int b = 0; b < DB; b++) {
      const int64_t i = i0 + 64 * b + lane;
      id[b] = i0 == plo ? first[b] : i < phi ? bucket_of(ids[i], E) : 0;
    }
#pragma unroll
    for (int b = 0; b < DB; b++)
      if (i0 + 64 * b + lane < phi) atomicAdd(&row[id[b]], 1);
  }
  __syncthreads();
  // scan of the totals over the experts, 64 * W at a time; then the first row
  // of every wave
  int32_t carry = 0;
  for (int e0 = 0; e0 <= E; e0 += 64 * W) {
    const int e = e0 + tid;
    int32_t here[W], all = 0;
    if (e <= E) {
#pragma unroll
      for (int v = 0; v < W; v++) {
        here[v] = next[v * (E + 1) + e];
        if (ONE || !counts) all += here[v];
      }
      if (!ONE) all += counts ? total[e] : before[e] + total[e];
    }
    const int32_t incl = scan64(all, OpAdd{});
    if (lane == 63) wave_sum[w] = incl;
    __syncthreads();
    int32_t start = carry + incl - all;
#pragma unroll
    for (int v = 0; v < W; v++) {
      const int32_t c = wave_sum[v];
      if (v < w) start += c;
      carry += c;
    }
    if (e <= E) {
      if (blockIdx.x == 0) offsets[e] = start;
      int32_t at = start + (ONE ? 0 : before[e]);
#pragma unroll
      for (int v = 0; v < W; v++) {
        next[v * (E + 1) + e] = at;
        at += here[v];
      }
    }
    __syncthreads();
  }
  auto place = [&](int64_t i0, auto pieces) {
    constexpr int P = decltype(pieces)::value;
    int id[P];
    uint32_t lo32[P], hi32[P];   // lanes of the same id
#pragma unroll
    for (int b = 0; b < P; b++) {
      const int64_t i = i0 + 64 * b + lane;
      id[b] = i0 == plo ? first[b] : i < phi ? bucket_of(ids[i], E) : 0;
      const uint64_t m = __ballot(i < phi);
      lo32[b] = (uint32_t)m;
      hi32[b] = (uint32_t)(m >> 32);
    }
    for (int bit = 0; bit < bits; bit++)
#pragma unroll
      for (int b = 0; b < P; b++) {
        const uint32_t mine = (uint32_t)__builtin_amdgcn_sbfe(id[b], bit, 1);   // all bits of it
        const uint64_t m = __ballot(mine);
        lo32[b] &= ~((uint32_t)m ^ mine);
        hi32[b] &= ~((uint32_t)(m >> 32) ^ mine);
      }
#pragma unroll
    for (int b = 0; b < P; b++) {
      const int64_t i = i0 + 64 * b + lane;
      if (i < phi) {
        const int32_t at = row[id[b]] + __builtin_amdgcn_mbcnt_hi(hi32[b], __builtin_amdgcn_mbcnt_lo(lo32[b], 0));
        // i < 2^31
        token[at] = id[b] < E ? (int32_t)((uint32_t)i / (uint32_t)top_k) : -1;
        position[i] = id[b] < E ? at : -1;
        const uint64_t same = lo32[b] | (uint64_t)hi32[b] << 32;
        if ((same >> lane) == 1) row[id[b]] = at + 1;   // the last lane of this id
      }
      wave_lds_fence();
    }
  };
  for (int64_t i0 = plo; i0 < phi; i0 += 64 * DB) {
    if (phi - i0 <= 64) place(i0, std::integral_constant<int, 1>{});
    else if (phi - i0 <= 128) place(i0, std::integral_constant<int, 2>{});
    else place(i0, std::integral_constant<int, DB>{});
  }
}

// Waves of a workgroup: 16 where eight would have more than a piece each, as
// long as 64 KB of LDS hold their counters.
static int waves_of(int64_t n, int64_t E) { return n > 64 * DW && n <= kOneLaunch && E <= 900 ? 16 : DW; }

// Slots of a workgroup: one batch a wave, more batches beyond kMaxRuns runs; alone
// in whole pieces for every wave.
static int64_t dispatch_run(int64_t n, int64_t E) {
  if (n <= kOneBlock) {
    const int64_t unit = 64 * waves_of(n, E);
    return (n + unit - 1) / unit * unit;
  }
  return ((n + kMaxRuns - 1) / kMaxRuns + kRun - 1) / kRun * kRun;
}

size_t moe_dispatch_workspace(int64_t n, int64_t E) {
  if (n <= kOneLaunch) return 0;
  const int64_t run = dispatch_run(n, E);
  return (size_t)((n + run - 1) / run) * (size_t)(E + 1) * 4u;
}

hipError_t launch_moe_dispatch(const int32_t* ids, int64_t n, int64_t E, int32_t top_k, int32_t* offsets, int32_t* token,
                               int32_t* position, int32_t* ws, hipStream_t stream) {
  int bits = 1;
  while ((1ll << bits) <= E) bits++;   // ids 0 .. E
  const int64_t run = dispatch_run(n, E);
  const int runs = n <= kOneBlock ? 1 : (int)((n + run - 1) / run);
  const size_t counters = (size_t)(E + 1) * 4u;
  if (n <= kOneLaunch) {
#define MOE_ONE(ONE, W)                                                                                               \
  hipLaunchKernelGGL((moe_place_kernel<ONE, W>), dim3((unsigned)runs), dim3(64 * W), (ONE ? W : W + 2) * counters, stream, \
                     ids, n, run, (int)E, top_k, bits, runs, nullptr, offsets, token, position)
    if (n <= kOneBlock) { if (waves_of(n, E) == 16) MOE_ONE(true, 16); else MOE_ONE(true, DW); }
    else { if (waves_of(n, E) == 16) MOE_ONE(false, 16); else MOE_ONE(false, DW); }
#undef MOE_ONE
    return hipGetLastError();
  }
  hipLaunchKernelGGL(moe_count_kernel, dim3((unsigned)runs), dim3(64 * DW), counters, stream, ids, n, run,
                     (int)E, ws);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_place_kernel<false, DW>), dim3((unsigned)runs), dim3(64 * DW), (DW + 2) * counters, stream, ids, n, run, (int)E,
                     top_k, bits, runs, ws, offsets, token, position);
  return hipGetLastError();
}

// ------------------------------------------------------------------- combine
// out[t] = sum_k w[t][k] y[pos[t][k]]: one pass over the rows of y, bound by
// HBM.  A thread owns 16 bytes of a token's row (VEC; single elements where
// rows are not 16-byte aligned) and has the loads of eight slots in flight.
// tpt threads (a power of two, 64 .. 256, so that a wave has one token) share
// a token.  8191 tokens x 8 x 4096: 107 us for 604 MB, 5.6 TB/s.
template <typename D, bool VEC>
__global__ __launch_bounds__(256) void moe_combine_kernel(const typename D::T* __restrict__ y, int64_t rows, int64_t ldy,
                                                          const int32_t* __restrict__ pos, const float* __restrict__ w,
                                                          int64_t T, int K, int64_t H, typename D::T* __restrict__ out,
                                                          int tpt, int chunks) {
  constexpr int V = VEC ? D::V : 1;
  const int per = 256 / tpt;
  const int64_t tb = blockIdx.x / chunks;
  const int ch = (int)(blockIdx.x - tb * chunks);
  const int64_t t = tb * per + __builtin_amdgcn_readfirstlane((int)threadIdx.x / tpt);
  const int64_t h = ((int64_t)ch * tpt + (threadIdx.x & (tpt - 1))) * V;
  if (t >= T || h >= H) return;
  const int32_t* tp = pos + t * K;
  const float* tw = w + t * K;
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; i++) acc[i] = 0.0f;
  for (int k0 = 0; k0 < K; k0 += 8) {
    u32x4 v[8];
    typename D::T sv[8];
    bool ok[8];
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const int64_t p = k0 + k < K ? tp[k0 + k] : -1;
      ok[k] = p >= 0 && p < rows;
      if (ok[k]) {
        if constexpr (VEC) v[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(y + p * ldy + h));
        else sv[k] = y[p * ldy + h];
      }
    }
#pragma unroll
    for (int k = 0; k < 8; k++)
      if (ok[k]) {
        const float wk = tw[k0 + k];
        float f[V];
        if constexpr (VEC) unpack<D>(v[k], f);
        else f[0] = to_f32<D>(sv[k]);
#pragma unroll
        for (int i = 0; i < V; i++) acc[i] = fmaf(wk, f[i], acc[i]);
      }
  }
  if constexpr (VEC) *reinterpret_cast<u32x4*>(out + t * H + h) = pack<D>(acc);
  else out[t * H + h] = from_f32<D>(acc[0]);
}

// How often a row of y is named.  Up to kOneCount slots a workgroup counts the
// rows of its range in LDS and goes through all positions for that (a few
// hundred KB of L2 reads): one launch, and no atomics on memory.  65528 slots and
// rows: 6.7 us (between the launches of a graph; 8.1 by itself), with a clear and a
// launch of atomics 9.6; 262144: 22.9 and 16.0.
// Up to kNoCount slots nothing is counted ahead: the gradients' waves look through
// the positions themselves (256 x 4 x 1024, all gradients: 4.8 us, with a launch of
// counts 6.7; 1024 x 4: 12.7 and 8.5) and the host has a launch less.
constexpr int64_t kNoCount = 1024;
constexpr int64_t kOneCount = 1 << 17;
constexpr int kCountRange = 2048;
__global__ __launch_bounds__(1024) void moe_count_rows_kernel(const int32_t* __restrict__ pos, int n, int rows,
                                                              int32_t* __restrict__ count) {
  __shared__ int32_t hist[kCountRange];
  const int r0 = blockIdx.x * kCountRange;
  const int here = rows - r0 < kCountRange ? rows - r0 : kCountRange;
  for (int i = threadIdx.x; i < kCountRange; i += 1024) hist[i] = 0;
  __syncthreads();
  constexpr int U = 16;   // loads in flight
  for (int i0 = threadIdx.x; i0 < n; i0 += 1024 * U) {
    int p[U];
#pragma unroll
    for (int u = 0; u < U; u++) p[u] = i0 + 1024 * u < n ? pos[i0 + 1024 * u] : -1;
#pragma unroll
    for (int u = 0; u < U; u++) {
      const uint32_t at = (uint32_t)p[u] - (uint32_t)r0;   // below r0: far past the range
      if (p[u] >= 0 && at < (uint32_t)here) atomicAdd(&hist[at], 1);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < here; i += 1024) count[r0 + i] = hist[i];
}
__global__ __launch_bounds__(256) void moe_clear_kernel(int32_t* __restrict__ count, int64_t rows) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < rows) count[i] = 0;
}
__global__ __launch_bounds__(256) void moe_named_kernel(const int32_t* __restrict__ pos, int64_t n, int64_t rows,
                                                        int32_t* __restrict__ count) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int64_t p = pos[i];
  if (p >= 0 && p < rows) atomicAdd(&count[p], 1);
}

// Backward.  TPT threads (64: four tokens a workgroup, 256: one) own a token:
// they read dout once and the token's rows of y, write the rows of dy and
// reduce the dot products.  A row that one slot names is written here as
// w * dout; one that several name is summed by the lowest of its slots (which
// finds the others by going through the positions: right, and slow, for what
// no dispatch produces).  The workgroups behind the tokens' own zero the rows
// that nobody names.  8191 tokens x 8 x 4096: 217 us for 1.14 GB, 5.3 TB/s, and
// 8 us to count who names whom; 8071 x 2 x 304: 7 us (18 with each slot's
// position, weight and count read by itself).
template <typename D, bool VEC, int TPT>
__global__ __launch_bounds__(256) void moe_combine_backward_kernel(
    const typename D::T* __restrict__ y, int64_t rows, int64_t ldy, const int32_t* __restrict__ pos,
    const float* __restrict__ w, int64_t T, int K, int64_t H, const typename D::T* __restrict__ dout, int64_t ldd,
    typename D::T* __restrict__ dy, float* __restrict__ dw, const int32_t* __restrict__ count, int64_t token_blocks) {
  constexpr int V = VEC ? D::V : 1;
  constexpr int PER = 256 / TPT;
  __shared__ float part[4][8];
  __shared__ int32_t has_slot[256];
  const int lane = threadIdx.x & 63;
  if ((int64_t)blockIdx.x >= token_blocks) {   // rows without a slot; launched with dy alone
    const int64_t rb = ((int64_t)blockIdx.x - token_blocks) * 256, r0 = rb + (threadIdx.x & ~63);
    const bool in = r0 + lane < rows;
    if (count) {
      has_slot[threadIdx.x] = in ? count[r0 + lane] : 1;
    } else {
      has_slot[threadIdx.x] = !in;
      __syncthreads();
      for (int64_t i = threadIdx.x; i < T * K; i += 256) {
        const int64_t at = (int64_t)pos[i] - rb;
        if (at >= 0 && at < 256) has_slot[at] = 1;
      }
      __syncthreads();
    }
    uint64_t none = __ballot(has_slot[threadIdx.x] == 0);
    while (none) {
      const int64_t r = r0 + __builtin_ctzll(none);
      none &= none - 1;
      for (int64_t h = (int64_t)lane * V; h < H; h += 64 * V) {
        if constexpr (VEC) *reinterpret_cast<u32x4*>(dy + r * H + h) = u32x4{0u, 0u, 0u, 0u};
        else dy[r * H + h] = from_f32<D>(0.0f);
      }
    }
    return;
  }
  const int64_t t = (int64_t)blockIdx.x * PER + __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPT);
  const int l = threadIdx.x & (TPT - 1);
  if (t < T) {   // uniform in a wave, and in the workgroup where TPT is 256
    for (int k0 = 0; k0 < K; k0 += 8) {
      // lane k of every eight looks after slot k0 + k: two latencies for all of them
      const int64_t slot = t * K + k0 + (lane & 7);
      const bool in = k0 + (lane & 7) < K;
      int pv = in ? pos[slot] : -1;
      const float wv = in ? w[slot] : 0.0f;
      if (pv >= rows) pv = -1;
      int cv = dy && count && pv >= 0 ? count[pv] : 0;
      if (dy && !count) {   // the wave counts its rows among all positions itself
        int n[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int64_t i0 = 0; i0 < T * K; i0 += 256) {
          int q[4];
#pragma unroll
          for (int u = 0; u < 4; u++) q[u] = i0 + 64 * u + lane < T * K ? pos[i0 + 64 * u + lane] : -1;
#pragma unroll
          for (int k = 0; k < 8; k++) {
            if (k0 + k >= K) break;
            const int p = __builtin_amdgcn_readlane(pv, k);
#pragma unroll
            for (int u = 0; u < 4; u++) n[k] += __popcll(__ballot(q[u] == p));
          }
        }
#pragma unroll
        for (int k = 0; k < 8; k++) cv = pv >= 0 && (lane & 7) == k ? n[k] : cv;
      }
      const uint32_t named = (uint32_t)__ballot(pv >= 0) & 0xFFu;   // slots with a row,
      const uint32_t alone = (uint32_t)__ballot(cv == 1) & 0xFFu;   // that nobody else names,
      uint32_t shared = (uint32_t)__ballot(cv > 1) & 0xFFu;         // that others name too
      auto row_of = [&](int k) { return (int64_t)__builtin_amdgcn_readlane(pv, k); };
      auto weight_of = [&](int k) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wv), k)); };
      float acc[8];
#pragma unroll
      for (int k = 0; k < 8; k++) acc[k] = 0.0f;
      for (int64_t h = (int64_t)l * V; h < H; h += TPT * V) {
        u32x4 v[8], gv;
        typename D::T sv[8];
        float g[V];
        if constexpr (VEC) gv = *reinterpret_cast<const u32x4*>(dout + t * ldd + h);
        else g[0] = to_f32<D>(dout[t * ldd + h]);
        if (dw) {
#pragma unroll
          for (int k = 0; k < 8; k++)
            if ((named >> k) & 1) {
              if constexpr (VEC) v[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(y + row_of(k) * ldy + h));
              else sv[k] = y[row_of(k) * ldy + h];
            }
        }
        if constexpr (VEC) unpack<D>(gv, g);
        if (dw) {
#pragma unroll
          for (int k = 0; k < 8; k++)
            if ((named >> k) & 1) {
              float f[V];
              if constexpr (VEC) unpack<D>(v[k], f);
              else f[0] = to_f32<D>(sv[k]);
#pragma unroll
              for (int i = 0; i < V; i++) acc[k] = fmaf(g[i], f[i], acc[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < 8; k++)
          if ((alone >> k) & 1) {
            const float wk = weight_of(k);
            float f[V];
#pragma unroll
            for (int i = 0; i < V; i++) f[i] = wk * g[i];
            if constexpr (VEC) __builtin_nontemporal_store(pack<D>(f), reinterpret_cast<u32x4*>(dy + row_of(k) * H + h));
            else dy[row_of(k) * H + h] = from_f32<D>(f[0]);
          }
      }
      while (shared) {
        const int k = __builtin_ctz(shared);
        shared &= shared - 1;
        const int64_t p = row_of(k), me = t * K + k0 + k;
        bool earlier = false;
        for (int64_t i0 = 0; i0 < me && !earlier; i0 += 64)
          earlier = __any(i0 + lane < me && pos[i0 + lane < me ? i0 + lane : 0] == p);
        if (earlier) continue;
        for (int64_t h = (int64_t)l * V; h < H; h += TPT * V) {
          float f[V];
#pragma unroll
          for (int i = 0; i < V; i++) f[i] = 0.0f;
          // the loop over h leaves the wave's last lanes behind: positions by those at work
          const uint64_t at_work = __ballot(true);
          const int width = __popcll(at_work);   // lanes 0 .. width - 1
          for (int64_t i0 = me; i0 < T * K; i0 += width) {
            uint64_t hit = __ballot(i0 + lane < T * K && pos[i0 + lane < T * K ? i0 + lane : 0] == p);
            while (hit) {
              const int64_t i = i0 + __builtin_ctzll(hit);
              hit &= hit - 1;
              const int64_t ti = i / K;
              float g[V];
              if constexpr (VEC) unpack<D>(*reinterpret_cast<const u32x4*>(dout + ti * ldd + h), g);
              else g[0] = to_f32<D>(dout[ti * ldd + h]);
#pragma unroll
              for (int j = 0; j < V; j++) f[j] = fmaf(w[i], g[j], f[j]);
            }
          }
          if constexpr (VEC) *reinterpret_cast<u32x4*>(dy + p * H + h) = pack<D>(f);
          else dy[p * H + h] = from_f32<D>(f[0]);
        }
      }
      if (dw) {
        float mine = 0.0f;   // lane k: slot k's sum over the wave
#pragma unroll
        for (int k = 0; k < 8; k++)
          if ((named >> k) & 1) {
            const float sum = lanes_reduce<64>(acc[k], OpAdd{});
            mine = lane == k ? sum : mine;
          }
        if (TPT == 64) {
          if (lane < 8 && in) dw[slot] = mine;
        } else {
          if (lane < 8) part[threadIdx.x >> 6][lane] = mine;
          __syncthreads();
          if (threadIdx.x < 8 && in) dw[slot] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
          __syncthreads();
        }
      }
    }
  }
}

static bool vec_rows(const void* p, int64_t ld, int64_t H, int esize) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * esize) % 16 == 0 && (H * esize) % 16 == 0;
}

// The forward's grid: threads per token (a power of two, 64 .. 256), their
// repeats along the row, workgroups along the tokens.
struct CombineGrid {
  bool vec;
  int tpt;
  int64_t chunks, tb;
};
static CombineGrid combine_grid(const void* y, int es, int64_t ldy, int64_t T, int64_t H, const void* out) {
  CombineGrid g;
  g.vec = vec_rows(y, ldy, H, es) && vec_rows(out, H, H, es);
  const int64_t items = g.vec ? H * es / 16 : H;
  g.tpt = items > 128 ? 256 : items > 64 ? 128 : 64;
  g.chunks = (items + g.tpt - 1) / g.tpt;
  g.tb = (T + 256 / g.tpt - 1) / (256 / g.tpt);
  return g;
}

template <typename D>
static hipError_t combine_t(const void* y, int64_t rows, int64_t ldy, const int32_t* pos, const float* w, int64_t T, int K,
                            int64_t H, void* out, hipStream_t stream) {
  const auto [vec, tpt, chunks, tb] = combine_grid(y, sizeof(typename D::T), ldy, T, H, out);
  const auto* yy = static_cast<const typename D::T*>(y);
  auto* o = static_cast<typename D::T*>(out);
  if (vec)
    hipLaunchKernelGGL((moe_combine_kernel<D, true>), dim3((unsigned)(tb * chunks)), dim3(256), 0, stream, yy, rows, ldy, pos,
                       w, T, K, H, o, tpt, (int)chunks);
  else
    hipLaunchKernelGGL((moe_combine_kernel<D, false>), dim3((unsigned)(tb * chunks)), dim3(256), 0, stream, yy, rows, ldy,
                       pos, w, T, K, H, o, tpt, (int)chunks);
  return hipGetLastError();
}

bool moe_combine_grid_fits(const void* y, int dtype, int64_t ldy, int64_t T, int64_t H, const void* out) {
  const CombineGrid g = combine_grid(y, dtype == 0 ? 4 : 2, ldy, T, H, out);
  return g.chunks <= 0x7FFFFFFF && grid_fits(g.tb, g.chunks, 256);
}
bool moe_combine_backward_grid_fits(int64_t T, int64_t K, int64_t rows) {
  return grid_fits(T + (rows + 255) / 256, 1, 256) && grid_fits((T * K + 255) / 256, 1, 256);
}

hipError_t launch_moe_combine(const void* y, int dtype, int64_t rows, int64_t ldy, const int32_t* pos, const float* w,
                              int64_t T, int K, int64_t H, void* out, hipStream_t stream) {
  return dtype == 0 ? combine_t<Fp32>(y, rows, ldy, pos, w, T, K, H, out, stream)
       : dtype == 1 ? combine_t<Bf16>(y, rows, ldy, pos, w, T, K, H, out, stream)
                    : combine_t<Fp16>(y, rows, ldy, pos, w, T, K, H, out, stream);
}

template <typename D>
static hipError_t combine_back_t(const void* y, int64_t rows, int64_t ldy, const int32_t* pos, const float* w, int64_t T,
                                 int K, int64_t H, const void* dout, int64_t ldd, void* dy, float* dw, int32_t* count,
                                 hipStream_t stream) {
  const int es = sizeof(typename D::T);
  const bool vec = vec_rows(dout, ldd, H, es) && (!dw || vec_rows(y, ldy, H, es)) && (!dy || vec_rows(dy, H, H, es));
  const int64_t items = vec ? H / D::V : H;
  const auto* yy = static_cast<const typename D::T*>(y);
  const auto* g = static_cast<const typename D::T*>(dout);
  auto* o = static_cast<typename D::T*>(dy);
  if (T * K <= kNoCount) {
    count = nullptr;
  } else if (dy && rows <= 2 * kOneCount && T * K <= kOneCount) {
    hipLaunchKernelGGL(moe_count_rows_kernel, dim3((unsigned)((rows + kCountRange - 1) / kCountRange)), dim3(1024), 0, stream,
                       pos, (int)(T * K), (int)rows, count);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  } else if (dy) {
    hipLaunchKernelGGL(moe_clear_kernel, dim3((unsigned)((rows + 255) / 256)), dim3(256), 0, stream, count, rows);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (T * K > 0)
      hipLaunchKernelGGL(moe_named_kernel, dim3((unsigned)((T * K + 255) / 256)), dim3(256), 0, stream, pos, T * K, rows,
                         count);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int tpt = items > 128 ? 256 : 64;
  const int64_t tb = (T + 256 / tpt - 1) / (256 / tpt);
  const int64_t blocks = tb + (dy ? (rows + 255) / 256 : 0);
  if (blocks == 0) return hipSuccess;
#define MOE_BACK(VE, TP)                                                                                                 \
  hipLaunchKernelGGL((moe_combine_backward_kernel<D, VE, TP>), dim3((unsigned)blocks), dim3(256), 0, stream, yy, rows, ldy, \
                     pos, w, T, K, H, g, ldd, o, dw, count, tb)
  if (vec) { if (tpt == 256) MOE_BACK(true, 256); else MOE_BACK(true, 64); }
  else { if (tpt == 256) MOE_BACK(false, 256); else MOE_BACK(false, 64); }
#undef MOE_BACK
  return hipGetLastError();
}

hipError_t launch_moe_combine_backward(const void* y, int dtype, int64_t rows, int64_t ldy, const int32_t* pos,
                                       const float* w, int64_t T, int K, int64_t H, const void* dout, int64_t ldd,
                                       void* dy, float* dw, int32_t* count, hipStream_t stream) {
  return dtype == 0 ? combine_back_t<Fp32>(y, rows, ldy, pos, w, T, K, H, dout, ldd, dy, dw, count, stream)
       : dtype == 1 ? combine_back_t<Bf16>(y, rows, ldy, pos, w, T, K, H, dout, ldd, dy, dw, count, stream)
                    : combine_back_t<Fp16>(y, rows, ldy, pos, w, T, K, H, dout, ldd, dy, dw, count, stream);
}

}  // namespace mx
