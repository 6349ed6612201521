// MXFP4 quantization and dequantization kernels for gfx950.
//
// A block of 32 BF16 values has the scale 2^X, X = floor(log2 amax) - 2 (so
// that the largest magnitude lands in [4, 8) and saturates at 6), and the E2M1
// codes of x / 2^X.  The amax is an integer maximum on the BF16 magnitude
// bits; its exponent field gives the scale byte without arithmetic on values;
// v_cvt_scalef32_pk_fp4_bf16 divides by the scale, rounds to nearest even and
// saturates.  Every kernel is one pass bound by HBM: 2 bytes in and 17/32 byte
// out per element and copy (the reverse for dequantize).
#include "mx_device.h"
#include "launch.h"

namespace mx {

// E8M0 byte of a block from the 15-bit magnitude pattern of its amax:
// floor(log2 amax) - 2 + 127 is (exponent field - 2); zero, subnormal and tiny
// amaxes clamp to byte 0.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 7);
  return (uint32_t)(e > 2 ? e - 2 : 0);
}

// Pair `i` of a code word: two BF16 values -> byte i.
#define MX4_CVT(word, pair, scale, i) \
  (uint32_t) __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16((word), __builtin_bit_cast(bf16x2, (uint32_t)(pair)), (scale), (i))

// Eight consecutive BF16 values of one block -> eight E2M1 codes.
__device__ __forceinline__ uint32_t fp4_codes8(uint4 v, uint32_t byte) {
  const float f = __uint_as_float(byte << 23);
  uint32_t w = 0;
  w = MX4_CVT(w, v.x, f, 0);
  w = MX4_CVT(w, v.y, f, 1);
  w = MX4_CVT(w, v.z, f, 2);
  w = MX4_CVT(w, v.w, f, 3);
  return w;
}

// The four bytes of lanes 0, 4, 8, 12 of a 16-lane row as one word (valid in
// the row's first lane).  All lanes of the row must execute it.
__device__ __forceinline__ uint32_t word_of_row(uint32_t byte) {
  const uint32_t b1 = (uint32_t)__builtin_amdgcn_mov_dpp((int)byte, 0x104, 0xF, 0xF, true);
  const uint32_t b2 = (uint32_t)__builtin_amdgcn_mov_dpp((int)byte, 0x108, 0xF, 0xF, true);
  const uint32_t b3 = (uint32_t)__builtin_amdgcn_mov_dpp((int)byte, 0x10C, 0xF, 0xF, true);
  return byte | (b1 << 8) | (b2 << 16) | (b3 << 24);
}

// ---- rowwise: 4 waves own 4 * RW rows x 512 columns; a wave reads a row's
// 512 columns at once (16 bytes a lane: 1 KB), all RW rows before the first is
// used.  A block is a DPP quad, a scale word a 16-lane DPP row; the words are
// gathered in LDS so that they leave as runs along the rows.  RW = 8 where
// that gives the chip enough workgroups, else 2 (short inputs: the latency of
// one load decides, not the width of the word stores): 32 x 4096 2.6 us, a launch
// and one latency.  8192 x 4096 takes 16.2 us for 85 MB, 5.2 TB/s.
constexpr int RQ_C = 512;

template <int RW, bool PACKED, bool GATHER>
__global__ __launch_bounds__(256) void mx4_quantize_row_kernel(const uint16_t* __restrict__ x, int64_t x_rows,
                                                               int64_t R, int64_t C, int64_t ldx,
                                                               const int32_t* __restrict__ index,
                                                               uint8_t* __restrict__ q, void* __restrict__ s,
                                                               int64_t tiles_c) {
  constexpr int TR = 4 * RW;
  __shared__ uint32_t words[4][TR + 1];
  const int lane = threadIdx.x & 63;
  const int w = threadIdx.x >> 6;
  const int64_t tr = blockIdx.x / tiles_c;
  const int64_t tc = blockIdx.x - tr * tiles_c;
  const int64_t r0 = tr * TR + w * RW;
  const int64_t c = tc * RQ_C + 8 * lane;
  const bool cval = c < C;   // C % 32 == 0: whole quads are valid
  uint4 v[RW];
#pragma unroll
  for (int i = 0; i < RW; i++) {
    const int64_t r = r0 + i;
    int64_t src = r;
    bool ok = cval && r < R;
    if (GATHER) {
      src = r < R ? (int64_t)index[r] : -1;
      ok = ok && src >= 0 && src < x_rows;
    }
    v[i] = ok ? load_nt16(x + src * ldx + c) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < RW; i++) {
    const int64_t r = r0 + i;
    uint32_t m = pk_max_u16(pk_max_u16(abs_bits2(v[i].x), abs_bits2(v[i].y)),
                            pk_max_u16(abs_bits2(v[i].z), abs_bits2(v[i].w)));
    m = quad_max(max(m & 0xFFFFu, m >> 16));
    const uint32_t byte = fp4_scale_byte(m);
    const uint32_t codes = fp4_codes8(v[i], byte);
    if (cval && r < R) *reinterpret_cast<uint32_t*>(q + r * (C / 2) + c / 2) = codes;
    if (PACKED) {
      const uint32_t word = word_of_row(byte);
      if ((lane & 15) == 0) words[lane >> 4][w * RW + i] = word;
    } else if (cval && r < R && (lane & 3) == 0) {
      static_cast<uint8_t*>(s)[r * (C / 32) + c / 32] = (uint8_t)byte;
    }
  }
  if (PACKED) {
    __syncthreads();
    for (int k = threadIdx.x; k < 4 * TR; k += 256) {
      const int t = k / TR, rr = k % TR;
      const int64_t kt = tc * 4 + t, r = tr * TR + rr;
      if (kt < C / 128 && r < R) static_cast<uint32_t*>(s)[kt * R + r] = words[t][rr];
    }
  }
}

// ---- columnwise, or both copies in one pass: 8 waves own 256 rows x 128
// columns, wave w the 32 rows 32 w .. + 31, i.e. one columnwise block per
// column; a lane the 8 x 8 sub-block rows 8 (lane / 16), columns 8 (lane % 16).
// Rowwise blocks are DPP quads, columnwise ones the four lanes 16 apart.  A
// byte permute pairs two rows of a column for the convert; the lane's dword of
// a column (8 rows) goes to a transposed LDS tile whose 16-byte chunks are
// XOR-swizzled by the lane's column group (all 16 lanes that write one
// register would else hit one bank), and leaves as 128-byte runs of q_colT.
// 8192 x 4096, both copies: 21.5 us for 103 MB, 4.8 TB/s (the transposed copy
// alone 16.5 us for 85 MB).  Measured and not kept: 8 waves a SIMD (64
// registers, 24.8 us), non-temporal q_colT stores (22.4 us), groups of 8 row
// tiles dealt to one XCD (22.3 us; 62 instead of 64.5 us at 16384 x 7168).
constexpr int CQ_R = 256, CQ_C = 128;

template <bool ROW, bool PACKED>
__global__ __launch_bounds__(512) void mx4_quantize_tile_kernel(const uint16_t* __restrict__ x, int64_t R, int64_t C,
                                                                int64_t ldx, uint8_t* __restrict__ q_row,
                                                                void* __restrict__ s_row, uint8_t* __restrict__ q_colT,
                                                                void* __restrict__ s_colT, int64_t tiles_c) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[CQ_C * (CQ_R / 8)];
  __shared__ __attribute__((aligned(16))) uint8_t col_scale[CQ_C][8];
  __shared__ __attribute__((aligned(16))) uint8_t row_scale[CQ_R][4];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int w = tid >> 6;
  const int cg = lane & 15, rg = lane >> 4;
  const int64_t tr = blockIdx.x / tiles_c;
  const int64_t r0 = tr * CQ_R;
  const int64_t c0 = (blockIdx.x - tr * tiles_c) * CQ_C;
  const int64_t rb = r0 + 32 * w + 8 * rg;
  const int64_t cb = c0 + 8 * cg;
  const bool val = cb < C && rb < R;   // R % 32 == 0: all 8 rows are valid or none is
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = val ? load_nt16(x + (rb + i) * ldx + cb) : make_uint4(0u, 0u, 0u, 0u);

  if (ROW) {
#pragma unroll
    for (int i = 0; i < 8; i++) {
      uint32_t m = pk_max_u16(pk_max_u16(abs_bits2(v[i].x), abs_bits2(v[i].y)),
                              pk_max_u16(abs_bits2(v[i].z), abs_bits2(v[i].w)));
      m = quad_max(max(m & 0xFFFFu, m >> 16));
      const uint32_t byte = fp4_scale_byte(m);
      const uint32_t codes = fp4_codes8(v[i], byte);
      if (val) *reinterpret_cast<uint32_t*>(q_row + (rb + i) * (C / 2) + cb / 2) = codes;
      if ((cg & 3) == 0) row_scale[32 * w + 8 * rg + i][cg >> 2] = (uint8_t)byte;
    }
  }
  // block amaxes of the lane's eight columns, two to a register
  uint32_t cm[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; i++) {
    cm[0] = pk_max_u16(cm[0], abs_bits2(v[i].x));
    cm[1] = pk_max_u16(cm[1], abs_bits2(v[i].y));
    cm[2] = pk_max_u16(cm[2], abs_bits2(v[i].z));
    cm[3] = pk_max_u16(cm[3], abs_bits2(v[i].w));
  }
#pragma unroll
  for (int j = 0; j < 4; j++) {
    cm[j] = pk_max_u16(cm[j], (uint32_t)__shfl_xor((int)cm[j], 16, 64));
    cm[j] = pk_max_u16(cm[j], (uint32_t)__shfl_xor((int)cm[j], 32, 64));
  }
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const uint32_t byte = fp4_scale_byte((k & 1) ? cm[k >> 1] >> 16 : cm[k >> 1] & 0xFFFFu);
    const float f = __uint_as_float(byte << 23);
    uint32_t pair[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const uint4 lo4 = v[2 * i], hi4 = v[2 * i + 1];
      const uint32_t lo = (k >> 1) == 0 ? lo4.x : (k >> 1) == 1 ? lo4.y : (k >> 1) == 2 ? lo4.z : lo4.w;
      const uint32_t hi = (k >> 1) == 0 ? hi4.x : (k >> 1) == 1 ? hi4.y : (k >> 1) == 2 ? hi4.z : hi4.w;
      // halves k & 1 of rows 2 i (low) and 2 i + 1 (high)
      pair[i] = __builtin_amdgcn_perm(hi, lo, (k & 1) ? 0x07060302u : 0x05040100u);
    }
    uint32_t word = 0;
    word = MX4_CVT(word, pair[0], f, 0);
    word = MX4_CVT(word, pair[1], f, 1);
    word = MX4_CVT(word, pair[2], f, 2);
    word = MX4_CVT(word, pair[3], f, 3);
    // column 8 cg + k, dword 4 w + rg of its 32; chunk w swizzled by cg
    tile[(8 * cg + k) * 32 + 4 * (w ^ (cg & 7)) + rg] = word;
    if (rg == 0) col_scale[8 * cg + k][w] = (uint8_t)byte;
  }
  __syncthreads();
#pragma unroll
  for (int k = tid; k < CQ_C * 8; k += 512) {
    const int col = k >> 3, ch = k & 7;
    const int64_t cc = c0 + col, rr = r0 + 32 * ch;
    if (cc < C && rr < R) {
      const u32x4 d = *reinterpret_cast<const u32x4*>(&tile[col * 32 + 4 * (ch ^ ((col >> 3) & 7))]);
      *reinterpret_cast<u32x4*>(q_colT + cc * (R / 2) + rr / 2) = d;
    }
  }
  if (PACKED) {
    if (tid < 256) {
      const int h = tid >> 7, col = tid & 127;
      const int64_t t = r0 / 128 + h;
      if (t < R / 128 && c0 + col < C)
        static_cast<uint32_t*>(s_colT)[t * C + c0 + col] = *reinterpret_cast<const uint32_t*>(&col_scale[col][4 * h]);
    } else if (ROW) {
      const int r = tid - 256;
      if (r0 + r < R)
        static_cast<uint32_t*>(s_row)[(c0 / 128) * R + r0 + r] = *reinterpret_cast<const uint32_t*>(row_scale[r]);
    }
  } else {
    for (int k = tid; k < CQ_C * 8; k += 512) {
      const int col = k >> 3, ch = k & 7;
      if (c0 + col < C && r0 + 32 * ch < R)
        static_cast<uint8_t*>(s_colT)[(c0 + col) * (R / 32) + r0 / 32 + ch] = col_scale[col][ch];
    }
    if (ROW)
      for (int k = tid; k < CQ_R * 4; k += 512) {
        const int r = k >> 2, b = k & 3;
        if (r0 + r < R && c0 + 32 * b < C)
          static_cast<uint8_t*>(s_row)[(r0 + r) * (C / 32) + c0 / 32 + b] = row_scale[r][b];
      }
  }
}

// ---- dequantize: 4 waves own 4 * RW rows x 512 columns as in the rowwise
// quantizer; a lane turns a code word of 8 elements into 16 bytes of BF16.
// The conversion multiplies the E2M1 value by 2^(byte - 127), exactly (BF16
// subnormals included).  8192 x 4096: 14.0 us for 85 MB, 6.1 TB/s.
template <int RW, bool PACKED>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint8_t* __restrict__ q, const void* __restrict__ s,
                                                             int64_t R, int64_t C, uint16_t* __restrict__ out,
                                                             int64_t ldo, int64_t tiles_c) {
  const int lane = threadIdx.x & 63;
  const int w = threadIdx.x >> 6;
  const int64_t tr = blockIdx.x / tiles_c;
  const int64_t r0 = (tr * 4 + w) * RW;
  const int64_t c = (blockIdx.x - tr * tiles_c) * RQ_C + 8 * lane;
  if (c >= C) return;
  uint32_t code[RW], byte[RW];
#pragma unroll
  for (int i = 0; i < RW; i++) {
    const int64_t r = r0 + i < R ? r0 + i : R - 1;
    code[i] = *reinterpret_cast<const uint32_t*>(q + r * (C / 2) + c / 2);
    byte[i] = PACKED ? (static_cast<const uint32_t*>(s)[(c >> 7) * R + r] >> (8 * ((lane >> 2) & 3))) & 0xFFu
                     : static_cast<const uint8_t*>(s)[r * (C / 32) + c / 32];
  }
#pragma unroll
  for (int i = 0; i < RW; i++) {
    if (r0 + i >= R) break;
    const float f = __uint_as_float(byte[i] << 23);
    uint4 o;
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[i], f, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[i], f, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[i], f, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[i], f, 3));
    *reinterpret_cast<uint4*>(out + (r0 + i) * ldo + c) = o;
  }
}

// Rows per wave of the row kernels: 8, or 2 where 8 would leave compute units
// without a workgroup.
static int rows_per_wave(int64_t R, int64_t tiles_c) { return ((R + 31) / 32) * tiles_c >= 512 ? 8 : 2; }

bool mx4_quantize_grid_fits(int64_t R, int64_t C) { return grid_fits((R + 7) / 8, (C + 127) / 128, 512); }

hipError_t launch_mx4_quantize(const uint16_t* x, int64_t x_rows, int64_t R, int64_t C, int64_t ldx,
                               const int32_t* index, bool row, bool col, bool packed, uint8_t* q_row, void* s_row,
                               uint8_t* q_colT, void* s_colT, hipStream_t stream) {
  if (col) {
    const int64_t tc = (C + CQ_C - 1) / CQ_C, tr = (R + CQ_R - 1) / CQ_R;
#define MX4_TILE(RO, PA) \
  hipLaunchKernelGGL((mx4_quantize_tile_kernel<RO, PA>), dim3((unsigned)(tr * tc)), dim3(512), 0, stream, x, R, C, ldx, \
                     q_row, s_row, q_colT, s_colT, tc)
    if (row) { if (packed) MX4_TILE(true, true); else MX4_TILE(true, false); }
    else { if (packed) MX4_TILE(false, true); else MX4_TILE(false, false); }
#undef MX4_TILE
    return hipGetLastError();
  }
  const int64_t tc = (C + RQ_C - 1) / RQ_C;
  const int rw = rows_per_wave(R, tc);
  const int64_t tr = (R + 4 * rw - 1) / (4 * rw);
#define MX4_ROW(RW, PA, GA) \
  hipLaunchKernelGGL((mx4_quantize_row_kernel<RW, PA, GA>), dim3((unsigned)(tr * tc)), dim3(256), 0, stream, x, x_rows, \
                     R, C, ldx, index, q_row, s_row, tc)
#define MX4_ROW_W(PA, GA) do { if (rw == 8) MX4_ROW(8, PA, GA); else MX4_ROW(2, PA, GA); } while (0)
  if (packed) { if (index) MX4_ROW_W(true, true); else MX4_ROW_W(true, false); }
  else { if (index) MX4_ROW_W(false, true); else MX4_ROW_W(false, false); }
#undef MX4_ROW_W
#undef MX4_ROW
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const uint8_t* q, const void* s, int64_t R, int64_t C, bool packed, uint16_t* out,
                                 int64_t ldo, hipStream_t stream) {
  const int64_t tc = (C + RQ_C - 1) / RQ_C;
  const int rw = rows_per_wave(R, tc);
  const int64_t tr = (R + 4 * rw - 1) / (4 * rw);
#define MX4_DEQ(RW, PA) \
  hipLaunchKernelGGL((mx4_dequantize_kernel<RW, PA>), dim3((unsigned)(tr * tc)), dim3(256), 0, stream, q, s, R, C, out, \
                     ldo, tc)
  if (packed) { if (rw == 8) MX4_DEQ(8, true); else MX4_DEQ(2, true); }
  else { if (rw == 8) MX4_DEQ(8, false); else MX4_DEQ(2, false); }
#undef MX4_DEQ
  return hipGetLastError();
}

}  // namespace mx
