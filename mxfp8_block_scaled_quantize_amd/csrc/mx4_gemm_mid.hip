// The MXFP4 GEMM's smaller tiles, for products whose 256 x 256 tiles would
// leave compute units without work.
//
// The same scheme as the large tile (32x32x64 MFMA, B first, 256-element K
// steps DMAd into LDS, chunks swizzled by (row >> 1) & 7) with BM x BN tiles,
// 2 x 2 waves of (BM / 2) x (BN / 2), and a ring of NS slots, unrolled so that
// every slot is a constant.  A step waits for its own slot's loads, reads all its
// fragments, asks for the step NS - 1 further on and multiplies.  Few tiles: the
// time is the steps' own latency (barrier, LDS reads, MFMA chain: 0.24 us a step
// of 64 x 64), and two workgroups of a compute unit fill each other's gaps.
// K = 4096: 512 x 4096 10.0 us with 64 x 64, 1024 x 4096 15.3 with 128 x 128.
// Measured and not kept: deeper rings (64 x 64 with six slots 8.6 us where three
// took 8.3; 128 x 128 with four, one workgroup a compute unit, 60 us where two
// took 45), fragments read one step ahead into a second set of registers (7.1 us
// where 6.3), 128 x 256 tiles (51 us where 128 x 128 takes 45); over 600 products:
// two slots for the two smaller tiles (5 % slower), a second barrier a step that
// frees its slot for one more step of loads (1 to 3 % slower).
#include "launch.h"
#include "mx4_gemm.h"

namespace mx {

using namespace mx4;

constexpr uint32_t PAST = 0xF8000000u;   // past every buffer (below 0xF0000000 bytes), with any step's offset added

template <int BM, int BN, int NS>
struct MidTile {
  static constexpr int A_BYTES = BM * STEP, B_BYTES = BN * STEP;
  static constexpr int SA_OFF = A_BYTES + B_BYTES;       // two words for each row of A,
  static constexpr int SB_OFF = SA_OFF + 2 * BM * 4;     // of B
  static constexpr int DATA = (BM + BN) / 8 / 4;                 // 1 KB DMA instructions of a wave and step
  static constexpr int WORDS = (2 * (BM + BN) / 64 + 3) / 4;     // 64-word ones (some past the last word, empty)
  static constexpr int SLOT = SA_OFF + 4 * WORDS * 256;
  static constexpr int LDS = NS * SLOT;
  static constexpr int PIECES = DATA + WORDS;
  static constexpr int C_STRIDE = 2 * BN + 16;
  static_assert(BM * C_STRIDE <= LDS && LDS <= 160 * 1024, "LDS");
};

template <int BM, int BN, int NS, bool GROUPED, int EPI>   // EPI 0 none, 1 accumulate, 2 SwiGLU
__global__ __launch_bounds__(256) void mx4_gemm_mid_kernel(const uint8_t* __restrict__ A, const uint32_t* __restrict__ Ap,
                                                           const uint8_t* __restrict__ B, const uint32_t* __restrict__ Bp,
                                                           uint16_t* __restrict__ C, int64_t ldc, int64_t M, int64_t N,
                                                           int64_t K, const int32_t* __restrict__ offsets, int32_t G,
                                                           int64_t tiles_m, int64_t tiles_n) {
  typedef MidTile<BM, BN, NS> T;
  constexpr bool SW = EPI == 2;
  constexpr int WM = BM / 64, WN = BN / 64;   // 32-row blocks of a wave
  static_assert(!SW || WN % 2 == 0, "gate and up blocks of a wave");
  constexpr int COLS = SW ? BN / 2 : BN;      // output columns of a tile
  constexpr int64_t BMUL = SW ? 2 : 1;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_raw[];
  lds_u8* smem = (lds_u8*)smem_raw;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t Kb = K / 2;
  int64_t tm, tn;
  tile_of_block<GROUPED>(tiles_m, tiles_n, &tm, &tn);
  int64_t m_lo = tm * BM, m_hi = M, b_row0 = 0;
  if (GROUPED) {
    const int g = group_of_tile<BM>(offsets, G, M, tm, &m_lo, &m_hi);
    if (g < 0) return;   // the whole workgroup
    b_row0 = (int64_t)g * N * BMUL;
  }
  const int64_t n0 = tn * COLS;
  const int64_t brows = (GROUPED ? (int64_t)G : 1) * N * BMUL;
  const int rows_a = (int)((m_hi - m_lo) < BM ? (m_hi - m_lo) : BM);

  // LDS row r of B holds tensor row b_row(r): plain n0 + r; SwiGLU: the wave's
  // BN / 2 rows are BN / 4 gate rows and the same columns' up rows.  Rows past
  // the end get an offset past the buffer and read as zero (B), or a valid row
  // (scale words, whose data rows are zero).
  auto b_row = [&](int r, bool* ok) -> int64_t {
    if (SW) {
      const int half = r / (BN / 2), up = r / (BN / 4) & 1;
      const int64_t oc = n0 + half * (BN / 4) + r % (BN / 4);
      *ok = oc < N;
      return b_row0 + up * N + (oc < N ? oc : N - 1);
    }
    *ok = n0 + r < N;
    return b_row0 + (n0 + r < N ? n0 + r : N - 1);
  };
  // Buffers start at the tile's first row of each operand (SwiGLU: the
  // expert's first gate row); offsets stay below 2^32.
  const int64_t b_base = SW ? b_row0 : b_row0 + n0;
  const int64_t b_span = SW ? 2 * N : (N - n0 < BN ? N - n0 : BN);
  uint32_t off[T::DATA];   // instruction i of a wave: LDS rows 8 (4 i + wave) + lane / 8, A's for i < BM / 32, then B's
  // The second half of a half step reads as zero: its lanes' own offsets are put
  // past the buffer (the range check may leave out the step's scalar offset).
  // The lane's chunk is the same in every instruction: 32 rows further on the
  // swizzle repeats.
  const bool late = ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7)) & 4;
#pragma unroll
  for (int i = 0; i < T::DATA; i++) {
    const int r = 8 * (4 * i + wave) + (lane >> 3);
    const int c = (lane & 7) ^ ((r >> 1) & 7);
    if (i < BM / 32) {
      off[i] = r < rows_a ? (uint32_t)r * (uint32_t)Kb + 16u * (uint32_t)c : PAST;
    } else {
      bool ok;
      const int64_t row = b_row(r - BM, &ok);
      off[i] = ok ? (uint32_t)((row - b_base) * Kb) + 16u * (uint32_t)c : PAST;
    }
  }
  // Scale instruction i of a wave: 64 words of one operand and one of its two
  // words of a step, from words(i) on, two words of K further each step.
  uint32_t soff[T::WORDS];
  const uint32_t* words[T::WORDS];
  int64_t stride[T::WORDS];
  int sbytes[T::WORDS], second[T::WORDS];
#pragma unroll
  for (int i = 0; i < T::WORDS; i++) {
    const int first = 64 * (4 * i + wave);   // word index in the slot's scale area, uniform
    const int at = first + lane;
    const bool is_a = first < 2 * BM, none = first >= 2 * (BM + BN);
    if (is_a) {
      const int r = at % BM;
      soff[i] = 4u * (uint32_t)(r < rows_a ? r : rows_a - 1);
      second[i] = first / BM;
    } else {
      bool ok;
      soff[i] = 4u * (uint32_t)(b_row((at - 2 * BM) % BN, &ok) - b_base);
      second[i] = (first - 2 * BM) / BN;
    }
    stride[i] = is_a ? M : brows;
    words[i] = (is_a ? Ap + m_lo : Bp + b_base) + (none ? 0 : second[i] * stride[i]);
    sbytes[i] = none ? 0 : is_a ? rows_a * 4 : (int)(b_span * 4);
    stride[i] = none ? 0 : 2 * stride[i];
  }
  const int nk = (int)((K + 255) / 256);
  const bool half_end = (K & 128) != 0;
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc((void*)(A + m_lo * Kb), 0, (int)((int64_t)rows_a * Kb), RSRC_FLAGS);
  const __amdgpu_buffer_rsrc_t rb =
      __builtin_amdgcn_make_buffer_rsrc((void*)(B + b_base * Kb), 0, (int)(uint32_t)(b_span * Kb), RSRC_FLAGS);
  auto issue = [&](int s, int slot) {   // in the order of steps
    lds_u8* base = smem + slot * T::SLOT;
    const int k0 = s * STEP;
    const bool cut = half_end && s == nk - 1;
    const bool skip = cut && late;
#pragma unroll
    for (int i = 0; i < T::DATA; i++) {
      lds_void* to = (lds_void*)(base + 1024 * (4 * i + wave));
      const uint32_t o = skip ? PAST : off[i];
      if (i < BM / 32) __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, to, 16, o, k0, 0, 0);
      else __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, to, 16, o, k0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < T::WORDS; i++) {
      const uint32_t o = soff[i];
      const __amdgpu_buffer_rsrc_t r =
          __builtin_amdgcn_make_buffer_rsrc((void*)words[i], 0, cut && second[i] ? 0 : sbytes[i], RSRC_FLAGS);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(base + T::SA_OFF + 256 * (4 * i + wave)), 4, o, 0, 0, 0);
      words[i] += stride[i];
    }
  };

  const int lr = lane & 31, lg = lane >> 5;
  const int swz = (lr >> 1) & 7;
  const int a_row = (wm * (BM / 2) + lr) * STEP;
  const int b_rowo = T::A_BYTES + (wn * (BN / 2) + lr) * STEP;
  const int sa_at = T::SA_OFF + 4 * (wm * (BM / 2) + lr);
  const int sb_at = T::SB_OFF + 4 * (wn * (BN / 2) + lr);
  v16f acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; i++)
#pragma unroll
    for (int j = 0; j < WN; j++) acc[i][j] = v16f{};
#pragma unroll
  for (int s = 0; s < NS - 1; s++)
    if (s < nk) issue(s, s);
  // Step t in slot u (a constant: every LDS address is a register plus an
  // immediate).  What the step reads is asked for first, then the loads of the
  // step NS - 1 further on, into the slot that every wave has left.
  auto step = [&](int t, auto SL) {
    constexpr int u = decltype(SL)::value;
    if (t + NS - 2 < nk) wait_vm<(NS - 2) * T::PIECES>();   // NS - 2 later steps are under way
    else wait_vm<0>();
    wait_lds();      // this wave's reads of the slot that is filled next
    barrier();
    const lds_u8* base = smem + u * T::SLOT;
    uint32_t sa[2][WM], sb[2][WN];
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int i = 0; i < WM; i++) sa[h][i] = *(lds_u32*)(base + sa_at + 4 * BM * h + 128 * i);
#pragma unroll
      for (int j = 0; j < WN; j++) sb[h][j] = *(lds_u32*)(base + sb_at + 4 * BN * h + 128 * j);
    }
    u32x4 fa[4][WM], fb[4][WN];
#pragma unroll
    for (int sl = 0; sl < 4; sl++) {
      const int p = 16 * ((2 * sl + lg) ^ swz);
#pragma unroll
      for (int i = 0; i < WM; i++) fa[sl][i] = *(lds_u32x4*)(base + a_row + 32 * STEP * i + p);
#pragma unroll
      for (int j = 0; j < WN; j++) fb[sl][j] = *(lds_u32x4*)(base + b_rowo + 32 * STEP * j + p);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (t + NS - 1 < nk) issue(t + NS - 1, (u + NS - 1) % NS);
#pragma unroll
    for (int h = 0; h < 2; h++) {
#pragma unroll
      for (int i = 0; i < WM; i++) sa[h][i] >>= 8 * lg;
#pragma unroll
      for (int j = 0; j < WN; j++) sb[h][j] >>= 8 * lg;
    }
#pragma unroll
    for (int sl = 0; sl < 4; sl++)
#pragma unroll
      for (int i = 0; i < WM; i++)
#pragma unroll
        for (int j = 0; j < WN; j++) {
          if (sl & 1)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fb[sl][j]), operand(fa[sl][i]), acc[i][j], 4, 4,
                                                                        2, (int)sb[sl >> 1][j], 2, (int)sa[sl >> 1][i]);
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(fb[sl][j]), operand(fa[sl][i]), acc[i][j], 4, 4,
                                                                        0, (int)sb[sl >> 1][j], 0, (int)sa[sl >> 1][i]);
        }
    __builtin_amdgcn_sched_barrier(0);
  };
  int t = 0;
  for (; t + NS <= nk; t += NS) {
    step(t, ic<0>{});
    step(t + 1, ic<1>{});
    if constexpr (NS > 2) step(t + 2, ic<2>{});
  }
  if (t < nk) step(t, ic<0>{});
  if constexpr (NS > 2)
    if (t + 1 < nk) step(t + 1, ic<1>{});
  wait_lds();
  barrier();

  // BF16 through a row-major LDS tile, then 16-byte stores
  constexpr int CH = COLS / 8;              // 16-byte chunks of an output row
  constexpr int PASS = 256 / CH;            // rows of a pass over the tile
  constexpr int STRIDE = 2 * COLS + 16;
  const int ch = tid % CH, row0 = tid / CH;
  const int64_t col = n0 + 8 * ch;
  if (EPI == 1) {
#pragma unroll
    for (int k = 0; k < BM / PASS; k++) {
      const int64_t r = m_lo + row0 + PASS * k;
      u32x4 v = u32x4{0u, 0u, 0u, 0u};
      if (col < N && r < m_hi) v = *reinterpret_cast<const u32x4*>(C + r * ldc + col);
      *(lds_u32x4*)(smem + (row0 + PASS * k) * STRIDE + 16 * ch) = v;
    }
    wait_lds();
    barrier();
  }
#pragma unroll
  for (int i = 0; i < WM; i++) {
    const int row = wm * (BM / 2) + 32 * i + lr;
#pragma unroll
    for (int j = 0; j < (SW ? WN / 2 : WN); j++)
#pragma unroll
      for (int g = 0; g < 4; g++) {
        lds_u32x2* p = (lds_u32x2*)(smem + row * STRIDE + 2 * (wn * (COLS / 2) + 32 * j + 8 * g + 4 * lg));
        float v[4];
#pragma unroll
        for (int t = 0; t < 4; t++) {
          v[t] = acc[i][j][4 * g + t];
          if (SW) v[t] = silu_f32(v[t]) * acc[i][SW ? j + WN / 2 : j][4 * g + t];
        }
        if (EPI == 1) {
          const u32x2 o = *p;
#pragma unroll
          for (int t = 0; t < 4; t++) v[t] += bf16_half2(o, t);
        }
        *p = bf16x4(v);
      }
  }
  wait_lds();
  barrier();
  if (col < N) {
#pragma unroll
    for (int k = 0; k < BM / PASS; k++) {
      const int64_t r = m_lo + row0 + PASS * k;
      if (r < m_hi) *reinterpret_cast<u32x4*>(C + r * ldc + col) = *(lds_u32x4*)(smem + (row0 + PASS * k) * STRIDE + 16 * ch);
    }
  }
}

template <int BM, int BN>
static void mid_tiles(const Mx4Gemm& g, int64_t* tm, int64_t* tn) {
  const int cols = g.epilogue == 2 ? BN / 2 : BN;
  *tm = g.offsets ? group_tiles(g.M, g.G, BM) : (g.M + BM - 1) / BM;
  *tn = (g.N + cols - 1) / cols;
}

// B's offsets inside a tile's buffer are 32 bits, below the mark of a row past
// the end; so are the scale words' of an expert.
bool mx4_gemm_mid_fits(const Mx4Gemm& g) {
  const int64_t rows = g.epilogue == 2 ? 2 * g.N : 256;
  int64_t tm, tn;
  mid_tiles<64, 64>(g, &tm, &tn);
  return rows * (g.K / 2) < 0xF0000000ll && g.N < (int64_t(1) << 27) && grid_fits(tm, tn, 256);
}

template <int BM, int BN, int NS, bool GROUPED, int EPI>
static hipError_t launch_mid_t(const Mx4Gemm& g, hipStream_t stream) {
  typedef MidTile<BM, BN, NS> T;
  if (T::LDS > 65536) {
    static std::atomic<uint64_t> done{0};
    const hipError_t e = allow_dynamic_lds(reinterpret_cast<const void*>(&mx4_gemm_mid_kernel<BM, BN, NS, GROUPED, EPI>),
                                           T::LDS, &done, stream);
    if (e != hipSuccess) return e;
  }
  int64_t tm, tn;
  mid_tiles<BM, BN>(g, &tm, &tn);
  hipLaunchKernelGGL((mx4_gemm_mid_kernel<BM, BN, NS, GROUPED, EPI>), dim3((unsigned)(tm * tn)), dim3(256), T::LDS, stream, g.a,
                     g.ap, g.b, g.bp, g.c, g.ldc, g.M, g.N, g.K, g.offsets, g.G, tm, tn);
  return hipGetLastError();
}

template <int BM, int BN, int NS>
static hipError_t launch_mid(const Mx4Gemm& g, hipStream_t stream) {
  if constexpr (BN > 64)   // a wave of SwiGLU holds gate and up blocks
    if (g.epilogue == 2)
      return g.offsets ? launch_mid_t<BM, BN, NS, true, 2>(g, stream) : launch_mid_t<BM, BN, NS, false, 2>(g, stream);
  if (g.epilogue == 1)
    return g.offsets ? launch_mid_t<BM, BN, NS, true, 1>(g, stream) : launch_mid_t<BM, BN, NS, false, 1>(g, stream);
  return g.offsets ? launch_mid_t<BM, BN, NS, true, 0>(g, stream) : launch_mid_t<BM, BN, NS, false, 0>(g, stream);
}

hipError_t launch_mx4_gemm_mid(const Mx4Gemm& g, Mx4Tile tile, hipStream_t stream) {
  return tile == Mx4Tile::k64x64   ? launch_mid<64, 64, 3>(g, stream)
       : tile == Mx4Tile::k64x128 ? launch_mid<64, 128, 3>(g, stream)
                                  : launch_mid<128, 128, 2>(g, stream);
}

}  // namespace mx
