// The MXFP4 GEMM's 256 x 256 tile, for products with enough tiles to fill the
// chip: bound by the matrix cores' rate at the clock that the chip's power leaves
// them, and by each tile's start and output.
//
// Operand layout of V_MFMA_SCALE_F32_32X32X64_F8F6F4 with E2M1 on both sides:
// lane l holds row l % 32, K = 32 (l / 32) + [0, 32) in its 16 bytes, i.e. one
// scale block, whose scale byte it supplies (byte chosen by op_sel).  Result
// register i of lane l is row 8 (i / 4) + 4 (l / 32) + i % 4 of the first
// operand, row l % 32 of the second; B goes first, so a lane holds runs of four
// consecutive columns of one row of C.
//
// One workgroup of 4 waves, one per SIMD; wave (wm, wn) owns 128 x 128 = 4 x 4
// MFMA blocks (256 fp32 accumulators a lane).  K moves in steps of 256 elements
// = 128 bytes a row through a ring of two LDS slots (68 KB each: 256 rows of A
// and of B and the step's two scale words per row) filled by buffer -> LDS DMA.
// A step is two halves of two 64-wide K slices with fragment registers of
// their own: the first half's MFMAs cover the LDS reads of the second half;
// then one barrier makes the next step's slot visible and frees this one; the
// second half's MFMAs cover the next step's first reads and the DMA of the step
// after it.  The order (two MFMAs, one 16-byte read, at most one DMA) is pinned
// with scheduling barriers.  16-byte chunks of an LDS row are XOR-swizzled by
// (row >> 1) & 7, which spreads a fragment read over all banks.  K of an odd
// number of 128 ends in a half step whose second half reads as zero.
//
// Rows past the end of an operand read as zero (buffer range check), results
// past the end are not stored.
//
// 8192 x 14336 x 4096 takes 229 us, 4.2 PFLOP/s; MFMAs on operands that never
// leave the registers reach 5.8 PFLOP/s on this grid (166 us), and codes that
// toggle more bits slow both down (uniformly random ones: 256 us).  A tile's start
// and output cost about 6 us in which nothing is multiplied (40 of the 229: seven
// rounds of tiles), a step 1.6 us under full load and 1.1 on an otherwise idle
// chip.  Counters on this grid, matrix cores busy and clock: K = 1024 25 % of the
// cycles at 2.25 GHz, K = 4096 49 % at 1.85; 8192 x 8192 x 16384 64 % at 1.63 (4.6
// PFLOP/s under the profiler, 4.9 without): the busier they are, the lower the
// clock.  Measured and not kept: a workgroup that stays and loads the next tile's
// first steps during its last ones, its output through a staging area of its own
// (254 us: more scalar registers than there are, and output rows in 128-byte
// instead of 512-byte pieces); cached instead of non-temporal stores (247 us);
// 6, 7, 8 or 14 tiles to a group (257 .. 268 us where 4 took 256).
#include "launch.h"
#include "mx4_gemm.h"

namespace mx {

using namespace mx4;

namespace {

constexpr int TM = 256, TNB = 256;               // rows of A and of B in a tile
constexpr int A_BYTES = TM * STEP, B_BYTES = TNB * STEP;
constexpr int SA_OFF = A_BYTES + B_BYTES;        // two words for each of 256 rows
constexpr int SB_OFF = SA_OFF + 2 * TM * 4;
constexpr int SLOT = SB_OFF + 2 * TNB * 4;       // 69632
constexpr int LDS_BYTES = 2 * SLOT;
constexpr int C_STRIDE = 2 * TNB + 16;           // staged BF16 output row
constexpr int SW_COLS = 128;                     // SwiGLU: output columns of a tile
constexpr int SW_STRIDE = 2 * SW_COLS + 16;
static_assert(TM * C_STRIDE <= LDS_BYTES && LDS_BYTES <= 160 * 1024, "LDS");

}  // namespace

template <bool GROUPED, int EPI>   // EPI 0 none, 1 accumulate, 2 SwiGLU
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(1, 1))) void mx4_gemm_tile_kernel(
    const uint8_t* __restrict__ A, const uint32_t* __restrict__ Ap, const uint8_t* __restrict__ B,
    const uint32_t* __restrict__ Bp, uint16_t* __restrict__ C, int64_t ldc, int64_t M, int64_t N, int64_t K,
    const int32_t* __restrict__ offsets, int32_t G, int64_t tiles_m, int64_t tiles_n) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_raw[];
  lds_u8* smem = (lds_u8*)smem_raw;
  constexpr bool SW = EPI == 2;
  constexpr int64_t BMUL = SW ? 2 : 1;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t Kb = K / 2;

  int64_t tm, tn;
  tile_of_block<GROUPED>(tiles_m, tiles_n, &tm, &tn);
  int64_t m_lo = tm * TM, m_hi = M, b_row0 = 0;
  if (GROUPED) {
    const int g = group_of_tile<TM>(offsets, G, M, tm, &m_lo, &m_hi);
    if (g < 0) return;   // the whole workgroup
    b_row0 = (int64_t)g * N * BMUL;
  }
  const int64_t n0 = tn * (SW ? SW_COLS : TNB);
  const int64_t brows = (GROUPED ? (int64_t)G : 1) * N * BMUL;
  const int rows_a = (int)((m_hi - m_lo) < TM ? (m_hi - m_lo) : TM);
  const int rows_b = (int)((N - n0) < TNB ? (N - n0) : TNB);

  // DMA instruction i of a wave brings LDS rows 64 wave + 8 i + lane / 8, chunk
  // slot lane % 8, which holds chunk c (the swizzle).
  uint32_t dma_off[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int r = 64 * wave + 8 * i + (lane >> 3);
    const int c = (lane & 7) ^ ((4 * i + (lane >> 4)) & 7);
    dma_off[i] = (uint32_t)r * (uint32_t)Kb + 16u * (uint32_t)c;
  }
  // Half step: chunks 4 .. 7 lie past the row; of instruction i that is bit 2
  // of the lane, flipped for odd i.  They read as zero in both operands.  (The
  // range check may leave out a load's scalar offset, here the step's: what has
  // to read as zero is past the range by its lane offset alone, and an empty
  // range goes with a scalar offset of zero.)
  const uint32_t hole_even = (lane & 4) ? HOLE : 0u, hole_odd = (lane & 4) ? 0u : HOLE;
  // Scale words: position p = 128 half + 4 lr + i holds row 128 half + 32 i + lr,
  // so that a lane's four words are one 16-byte read; rows past the end repeat
  // a valid one (their data is zero).
  const int sp = 64 * wave + lane;
  const int srow = (sp & ~127) + 32 * (sp & 3) + ((sp & 127) >> 2);
  const int sra = srow < rows_a ? srow : rows_a - 1;
  int srb;
  if (SW) {   // 64-row segments: gate rows (even), up rows (odd) of the same 64 columns
    const int s = srow >> 6;
    const int64_t oc = n0 + 64 * (s >> 1) + (srow & 63);
    srb = (int)((s & 1) * N + (oc < N ? oc : N - 1));
  } else {
    srb = srow < rows_b ? srow : rows_b - 1;
  }
  const int nk = (int)((K + 255) / 256);
  const int words = (int)(K / 128);
  const bool half_end = (K & 128) != 0;
  const __amdgpu_buffer_rsrc_t ra_v =
      __builtin_amdgcn_make_buffer_rsrc((void*)(A + m_lo * Kb), 0, (int)((int64_t)rows_a * Kb), RSRC_FLAGS);
  __amdgpu_buffer_rsrc_t rb_v;
  bool have_b = true;   // whether the wave's rows of B begin before its end
  if (SW) {
    // wave w fills rows 64 w .. of the slot: its resource starts 64 w rows
    // before the segment's first row, so that the shared offsets land on it
    const int64_t oc0 = n0 + 64 * (wave >> 1);
    const int64_t seg = N - oc0 < 0 ? 0 : (N - oc0 < 64 ? N - oc0 : 64);
    const int64_t src = b_row0 + (wave & 1) * N + oc0;
    have_b = seg > 0;
    rb_v = __builtin_amdgcn_make_buffer_rsrc((void*)((uintptr_t)B + (uintptr_t)((src - 64 * wave) * Kb)), 0,
                                             seg ? (int)((64 * wave + seg) * Kb) : 0, RSRC_FLAGS);
  } else {
    rb_v = __builtin_amdgcn_make_buffer_rsrc((void*)(B + (b_row0 + n0) * Kb), 0, (int)((int64_t)rows_b * Kb), RSRC_FLAGS);
  }
  const __amdgpu_buffer_rsrc_t r_none = __builtin_amdgcn_make_buffer_rsrc((void*)A, 0, 0, RSRC_FLAGS);

  // Piece q of step s: 0 .. 7 A, 8 .. 15 B, 16 / 17 A's scale words, 18 / 19 B's.
  // Steps past the end touch no memory (empty ranges) and fill a slot that
  // adds nothing.
  auto dma_piece = [&](int s, auto SL, int q) {
    lds_u8* base = smem + decltype(SL)::value * SLOT;
    const bool valid = s < nk;
    const int k0 = valid ? s * STEP : 0;
    if (q < 16) {
      const bool cut = half_end && s == nk - 1;
      const uint32_t off = dma_off[q & 7] + (cut ? ((q & 1) ? hole_odd : hole_even) : 0u);
      if (q < 8)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(valid ? ra_v : r_none, (lds_void*)(base + 1024 * (8 * wave + q)), 16, off, k0,
                                                 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(valid ? rb_v : r_none, (lds_void*)(base + A_BYTES + 1024 * (8 * wave + q - 8)),
                                                 16, off, have_b ? k0 : 0, 0, 0);
    } else {
      const int t = 2 * s + (q & 1);
      const bool have = t < words;
      const int64_t tt = have ? t : 0;
      if (q < 18) {
        const __amdgpu_buffer_rsrc_t r =
            __builtin_amdgcn_make_buffer_rsrc((void*)(Ap + tt * M + m_lo), 0, have ? rows_a * 4 : 0, RSRC_FLAGS);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(base + SA_OFF + 1024 * (q & 1) + 256 * wave), 4,
                                                 4u * (uint32_t)sra, 0, 0, 0);
      } else {
        const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
            (void*)(Bp + tt * brows + b_row0 + (SW ? 0 : n0)), 0, have ? (SW ? (int)(8 * N) : rows_b * 4) : 0, RSRC_FLAGS);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(base + SB_OFF + 1024 * (q & 1) + 256 * wave), 4,
                                                 4u * (uint32_t)srb, 0, 0, 0);
      }
    }
  };

  const int lr = lane & 31;
  const int lg = lane >> 5;
  const int swz = (lr >> 1) & 7;
  const int a_row = (wm * 128 + lr) * STEP;
  const int b_row = A_BYTES + (wn * 128 + lr) * STEP;
  const uint32_t sh = 8u * (uint32_t)lg;
  u32x4 fa[2][2][4], fb[2][2][4];          // [half][slice][block]
  uint32_t sa[2][4], sb[2][4], na[2][4], nb[2][4];
  v16f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < 4; j++) acc[i][j] = v16f{};

  // Fragment piece qq of half h, in the order of use: slice 0 (A0, B0 .. B3,
  // A1 .. A3), then slice 1.
  auto read_piece = [&](auto SL, auto H, int qq) {
    constexpr int h = decltype(H)::value;
    constexpr int order[8] = {0, 4, 5, 6, 7, 1, 2, 3};
    const int sl = qq >> 3, f = order[qq & 7];
    const lds_u8* base = smem + decltype(SL)::value * SLOT;
    const int p = 16 * ((4 * h + 2 * sl + lg) ^ swz);
    if (f < 4) fa[h][sl][f] = *(lds_u32x4*)(base + a_row + f * 32 * STEP + p);
    else fb[h][sl][f - 4] = *(lds_u32x4*)(base + b_row + (f - 4) * 32 * STEP + p);
  };
  auto read_scales = [&](auto SL, uint32_t (*ra)[4], uint32_t (*rb)[4]) {
    const lds_u8* base = smem + decltype(SL)::value * SLOT;
#pragma unroll
    for (int j = 0; j < 2; j++) {
      const u32x4 a4 = *(lds_u32x4*)(base + SA_OFF + 1024 * j + 16 * (wm * 32 + lr));
      const u32x4 b4 = *(lds_u32x4*)(base + SB_OFF + 1024 * j + 16 * (wn * 32 + lr));
#pragma unroll
      for (int i = 0; i < 4; i++) {
        ra[j][i] = a4[i];
        rb[j][i] = b4[i];
      }
    }
  };
  // MFMA q of half h: slice q / 16, block (q / 4 % 4, q % 4).  The scale words
  // are shifted by 8 (lane / 32) once a step, so that byte 0 (2) of a lane is
  // the scale of its block in the half's first (second) slice.
  auto mfma_one = [&](auto H, int q) {
    constexpr int h = decltype(H)::value;
    const int sl = q >> 4, i = (q >> 2) & 3, j = q & 3;
    if (sl == 0)
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fb[h][0][j]), operand(fa[h][0][i]), acc[i][j], 4, 4,
                                                                  0, (int)sb[h][j], 0, (int)sa[h][i]);
    else
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fb[h][1][j]), operand(fa[h][1][i]), acc[i][j], 4, 4,
                                                                  2, (int)sb[h][j], 2, (int)sa[h][i]);
  };
  auto kstep = [&](int t, auto SL) {
    constexpr int slot = decltype(SL)::value;
#pragma unroll
    for (int q = 0; q < 16; q++) {
      mfma_one(ic<0>{}, 2 * q);
      read_piece(SL, ic<1>{}, q);
      mfma_one(ic<0>{}, 2 * q + 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_vm<0>();
    wait_lds();
    barrier();
#pragma unroll
    for (int q = 16; q < 20; q++) dma_piece(t + 2, SL, q);
    read_scales(ic<1 - slot>{}, na, nb);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < 16; q++) {
      mfma_one(ic<1>{}, 2 * q);
      read_piece(ic<1 - slot>{}, ic<0>{}, q);
      mfma_one(ic<1>{}, 2 * q + 1);
      dma_piece(t + 2, SL, q);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        sa[j][i] = na[j][i] >> sh;
        sb[j][i] = nb[j][i] >> sh;
      }
  };
  if (nk > 0) {
#pragma unroll
    for (int q = 0; q < 20; q++) dma_piece(0, ic<0>{}, q);
#pragma unroll
    for (int q = 0; q < 20; q++) dma_piece(1, ic<1>{}, q);
    wait_vm<20>();
    barrier();
    read_scales(ic<0>{}, sa, sb);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < 16; q++) {
      read_piece(ic<0>{}, ic<0>{}, q);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
      for (int i = 0; i < 4; i++) {
        sa[j][i] >>= sh;
        sb[j][i] >>= sh;
      }
    for (int t = 0; t < nk; t += 2) {   // an odd count runs one step of zeros
      kstep(t, ic<0>{});
      kstep(t + 1, ic<1>{});
    }
  }
  wait_vm<0>();   // the tail's empty DMA, before the ring is used again
  wait_lds();
  barrier();

  // Epilogue: BF16 through a row-major LDS tile, then 16-byte stores of whole
  // row segments.  The lane id is derived anew so that nothing of it stays live
  // over the main loop.
  const int el = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
  const bool full_rows = m_lo + TM <= m_hi;
  if constexpr (SW) {
    // blocks j = 0, 1 hold the gate and j + 2 the up sums of the same columns
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int row = wm * 128 + 32 * i + (el & 31);
#pragma unroll
      for (int j = 0; j < 2; j++)
#pragma unroll
        for (int g = 0; g < 4; g++) {
          const int col = wn * 64 + 32 * j + 8 * g + 4 * (el >> 5);
          float v[4];
#pragma unroll
          for (int t = 0; t < 4; t++) v[t] = silu_f32(acc[i][j][4 * g + t]) * acc[i][j + 2][4 * g + t];
          *(lds_u32x2*)(smem + row * SW_STRIDE + 2 * col) = bf16x4(v);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_lds();
    barrier();
    const int ch = el & 15, row0 = 4 * wave + (el >> 4);
    const int64_t col = n0 + 8 * ch;
    if (col < N) {
      u32x4 v[16];
#pragma unroll
      for (int k = 0; k < 16; k++) v[k] = *(lds_u32x4*)(smem + (row0 + 16 * k) * SW_STRIDE + 16 * ch);
#pragma unroll
      for (int k = 0; k < 16; k++) {
        const int64_t r = m_lo + row0 + 16 * k;
        if (full_rows || r < m_hi) store_nt16(C + r * ldc + col, make_uint4(v[k].x, v[k].y, v[k].z, v[k].w));
      }
    }
    return;
  }
  const int ch = el & 31, row0 = 2 * wave + (el >> 5);
  const int64_t col = n0 + 8 * ch;
  if (EPI == 1) {   // stage the old C first: all loads before the first LDS write
    u32x4 v[32];
#pragma unroll
    for (int k = 0; k < 32; k++) {
      const int64_t r = m_lo + row0 + 8 * k;
      v[k] = u32x4{0u, 0u, 0u, 0u};
      if (col < N && r < m_hi) v[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(C + r * ldc + col));
    }
#pragma unroll
    for (int k = 0; k < 32; k++) *(lds_u32x4*)(smem + (row0 + 8 * k) * C_STRIDE + 16 * ch) = v[k];
    wait_lds();
    barrier();
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int row = wm * 128 + 32 * i + (el & 31);
#pragma unroll
    for (int j = 0; j < 4; j++)
#pragma unroll
      for (int g = 0; g < 4; g++) {
        lds_u32x2* p = (lds_u32x2*)(smem + row * C_STRIDE + 2 * (wn * 128 + 32 * j + 8 * g + 4 * (el >> 5)));
        float v[4];
#pragma unroll
        for (int t = 0; t < 4; t++) v[t] = acc[i][j][4 * g + t];
        if (EPI == 1) {
          const u32x2 o = *p;
#pragma unroll
          for (int t = 0; t < 4; t++) v[t] += bf16_half2(o, t);
        }
        *p = bf16x4(v);
      }
    __builtin_amdgcn_sched_barrier(0);
  }
  wait_lds();
  barrier();
  if (col < N) {
#pragma unroll
    for (int kb = 0; kb < 32; kb += 16) {
      u32x4 v[16];
#pragma unroll
      for (int k = 0; k < 16; k++) v[k] = *(lds_u32x4*)(smem + (row0 + 8 * (kb + k)) * C_STRIDE + 16 * ch);
#pragma unroll
      for (int k = 0; k < 16; k++) {
        const int64_t r = m_lo + row0 + 8 * (kb + k);
        if (full_rows || r < m_hi) store_nt16(C + r * ldc + col, make_uint4(v[k].x, v[k].y, v[k].z, v[k].w));
      }
    }
  }
}

static int64_t tile_cols(const Mx4Gemm& g) { return g.epilogue == 2 ? SW_COLS : TNB; }
static int64_t tiles_n(const Mx4Gemm& g) { return (g.N + tile_cols(g) - 1) / tile_cols(g); }
static int64_t tiles_m(const Mx4Gemm& g) { return g.offsets ? group_tiles(g.M, g.G, TM) : (g.M + TM - 1) / TM; }
// An expert's scale words (SwiGLU: 2N of them) lie in one buffer of 32-bit offsets.
bool mx4_gemm_tile_fits(const Mx4Gemm& g) {
  return (g.epilogue != 2 || g.N < (int64_t(1) << 28)) && grid_fits(tiles_m(g), tiles_n(g), 256);
}

// More than 64 KB of dynamic LDS has to be asked for, once per kernel and device
// (the stream's, made current for it); `done` holds a bit per device below 64.
hipError_t allow_dynamic_lds(const void* kernel, int bytes, std::atomic<uint64_t>* done, hipStream_t stream) {
  int dev = 0;
  hipError_t e = stream ? hipStreamGetDevice(stream, &dev) : hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (bit && (done->load(std::memory_order_acquire) & bit)) return hipSuccess;
  int cur = 0;
  e = hipGetDevice(&cur);
  if (e != hipSuccess) return e;
  if (cur != dev && (e = hipSetDevice(dev)) != hipSuccess) return e;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (cur != dev) {
    const hipError_t back = hipSetDevice(cur);
    if (e == hipSuccess) e = back;
  }
  if (e == hipSuccess) done->fetch_or(bit, std::memory_order_release);
  return e;
}

template <bool GROUPED, int EPI>
static hipError_t launch_tile(const Mx4Gemm& g, hipStream_t stream) {
  static std::atomic<uint64_t> done{0};
  const hipError_t e =
      allow_dynamic_lds(reinterpret_cast<const void*>(&mx4_gemm_tile_kernel<GROUPED, EPI>), LDS_BYTES, &done, stream);
  if (e != hipSuccess) return e;
  const int64_t tm = tiles_m(g), tn = tiles_n(g);
  hipLaunchKernelGGL((mx4_gemm_tile_kernel<GROUPED, EPI>), dim3((unsigned)(tm * tn)), dim3(256), LDS_BYTES, stream, g.a, g.ap,
                     g.b, g.bp, g.c, g.ldc, g.M, g.N, g.K, g.offsets, g.G, tm, tn);
  return hipGetLastError();
}

hipError_t launch_mx4_gemm_tile(const Mx4Gemm& g, hipStream_t stream) {
  if (g.offsets)
    return g.epilogue == 2 ? launch_tile<true, 2>(g, stream)
         : g.epilogue == 1 ? launch_tile<true, 1>(g, stream)
                           : launch_tile<true, 0>(g, stream);
  return g.epilogue == 2 ? launch_tile<false, 2>(g, stream)
       : g.epilogue == 1 ? launch_tile<false, 1>(g, stream)
                         : launch_tile<false, 0>(g, stream);
}

}  // namespace mx
