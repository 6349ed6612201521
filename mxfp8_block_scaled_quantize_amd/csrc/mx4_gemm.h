// Device code shared by the MXFP4 GEMM's tiled kernels.
#pragma once

#include "mx_device.h"
#include "wave_scan.h"

namespace mx {
namespace mx4 {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) uint32_t lds_u32;

constexpr int STEP = 128;                        // bytes of a row in a K step: 256 elements
constexpr uint32_t RSRC_FLAGS = 0x00020000u;     // raw buffer, 32-bit data
constexpr uint32_t HOLE = 0x40000000u;           // past every buffer (at most 2^29 bytes)

template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }
// The compiler may not move memory accesses across; what must have landed is
// waited for explicitly in front of it.
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
template <int V>
struct ic {
  static constexpr int value = V;
};
__device__ __forceinline__ v8i operand(u32x4 d) {   // an FP4 operand takes the low four registers
  v8i r;
  r.lo = __builtin_bit_cast(v4i, d);
  return r;
}
__device__ __forceinline__ u32x2 bf16x4(const float* v) {
  const bf16x2 h0 = {(__bf16)v[0], (__bf16)v[1]};
  const bf16x2 h1 = {(__bf16)v[2], (__bf16)v[3]};
  return u32x2{__builtin_bit_cast(uint32_t, h0), __builtin_bit_cast(uint32_t, h1)};
}

// Workgroup -> tile.  Ids are dealt to the 8 XCDs in turn: each XCD gets a
// contiguous range of tiles, walked in groups of 4 along the larger side
// (grouped: along N, so that an expert's B is read once), which share an
// operand in the XCD's L2.
template <bool GROUPED>
__device__ __forceinline__ void tile_of_block(int64_t tiles_m, int64_t tiles_n, int64_t* tm, int64_t* tn) {
  constexpr int GROUP = 4;
  const int64_t nblk = tiles_m * tiles_n;
  const int64_t bid = blockIdx.x;
  const int64_t full = (nblk / 8) * 8;
  const int64_t lid = bid < full ? (bid & 7) * (full >> 3) + (bid >> 3) : bid;
  if (!(GROUPED || tiles_n > tiles_m)) {
    const int64_t per = (int64_t)GROUP * tiles_n;
    const int64_t first = lid / per * GROUP;
    const int64_t n = (tiles_m - first) < GROUP ? (tiles_m - first) : GROUP;
    const int64_t rem = lid % per;
    *tm = first + rem % n;
    *tn = rem / n;
  } else {
    const int64_t per = (int64_t)GROUP * tiles_m;
    const int64_t first = lid / per * GROUP;
    const int64_t n = (tiles_n - first) < GROUP ? (tiles_n - first) : GROUP;
    const int64_t rem = lid % per;
    *tn = first + rem % n;
    *tm = rem / n;
  }
}

// Bound on the row tiles of G groups in M rows: a group with rows, of which there
// are M at most, ends BM - 1 rows into a tile at worst.
inline int64_t group_tiles(int64_t M, int64_t G, int64_t BM) { return (M + (G < M ? G : M) * (BM - 1)) / BM; }

// Row tile tm (of TM rows) among the groups' tiles, 64 groups at a time: bounds
// clamped into [0, M] and raised to the running maximum, a prefix sum of the
// tile counts, and the lane whose range holds tm.  Returns the group (-1: past
// the last tile) and the tile's rows [lo, hi) to the group's end.  Every wave
// of the workgroup computes the same.
template <int TM>
__device__ __forceinline__ int group_of_tile(const int32_t* __restrict__ offsets, int G, int64_t M, int64_t tm, int64_t* m_lo,
                                             int64_t* m_hi) {
  const int lane = threadIdx.x & 63;
  const int end = (int)M;
  int carry = 0;
  for (int g0 = 0; g0 < G; g0 += 64) {
    const int g = g0 + lane;
    int lo = 0, hi = 0;
    if (g < G) {
      const int l = offsets[g], h = offsets[g + 1];
      lo = l < 0 ? 0 : (l > end ? end : l);
      hi = h < 0 ? 0 : (h > end ? end : h);
    }
    lo = lo > carry ? lo : carry;
    lo = scan64(lo, [](int a, int b) { return a > b ? a : b; });
    hi = hi > lo ? hi : lo;
    carry = __builtin_amdgcn_readlane(hi, 63);
    const int nt = (int)(((unsigned)(hi - lo) + TM - 1) / TM);
    const int incl = scan64(nt, [](int a, int b) { return a + b; });
    const int total = __builtin_amdgcn_readlane(incl, 63);
    if (tm < total) {
      const int fl = __builtin_ctzll(__ballot(incl > tm));
      const int before = __builtin_amdgcn_readlane(incl - nt, fl);
      *m_lo = (int64_t)__builtin_amdgcn_readlane(lo, fl) + (tm - before) * TM;
      *m_hi = (int64_t)__builtin_amdgcn_readlane(hi, fl);
      return g0 + fl;
    }
    tm -= total;
  }
  return -1;
}

}  // namespace mx4
}  // namespace mx
