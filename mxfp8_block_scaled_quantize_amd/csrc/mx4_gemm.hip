// Block-scaled MXFP4 GEMM (TN) on the gfx950 scaled FP4 matrix instructions.
//
//   C[m][n] = bf16( sum_k dq(A)[m][k] dq(B)[n][k] ), fp32 accumulation.
//
// Operand layout of V_MFMA_SCALE_F32_16X16X128_F8F6F4 with E2M1 on both sides:
// lane l holds row l % 16, K = 32 (l / 16) + [0, 32) in its 16 bytes (one scale
// block), and supplies that block's scale byte.  Result register i of lane l is
// row 4 (l / 16) + i of the first operand, row l % 16 of the second.  The
// kernels pass B first: a lane holds four consecutive columns of one row of C.
#include "launch.h"
#include "mx4_gemm.h"

namespace mx {

using namespace mx4;
typedef float v4f __attribute__((ext_vector_type(4)));

// ---- few rows per group: bound by the stream of B.  W waves share 16 NB rows
// of B (SwiGLU: 16 gate rows and their 16 up rows) and 16 MB rows of A of one
// group, each wave a part of K.  Both operands go from global memory straight
// to registers in the matrix instructions' layout (16 rows x 64 bytes a load),
// several K slices in flight; the waves' sums meet in LDS.  One row x 14336 columns, K = 4096: 7.3 us
// for 31 MB, of which 2 are the launch; 148 rows of 32 experts, 27 with rows, through
// 2048 x 4096 weights (SwiGLU): 23.4 us for the 130 MB that the counters see, 5.5 TB/s
// (row sums of 4 GB read 6.4).
enum { EPI_NONE = 0, EPI_ACC = 1, EPI_SWIGLU = 2 };

template <int MB, int NB, int W, bool GROUPED, int EPI>
__global__ __launch_bounds__(64 * W) void mx4_gemm_rows_kernel(const uint8_t* __restrict__ A, const uint32_t* __restrict__ Ap,
                                                               const uint8_t* __restrict__ B, const uint32_t* __restrict__ Bp,
                                                               uint16_t* __restrict__ C, int64_t ldc, int64_t M, int64_t N,
                                                               int64_t K, const int32_t* __restrict__ offsets, int32_t G) {
  constexpr bool SW = EPI == EPI_SWIGLU;
  static_assert(!SW || NB == 2, "gate and up rows");
  constexpr int TN = SW ? 16 : 16 * NB;
  constexpr int U = 8 / NB;   // K slices of 128 in flight
  __shared__ v4f red[W][MB][NB][64];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int r = lane & 15, kg = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * TN;
  int64_t m0 = (int64_t)blockIdx.y * 16 * MB, hi = M, b_row0 = 0;
  if (GROUPED) {
    const int g = group_of_tile<16 * MB>(offsets, G, M, blockIdx.y, &m0, &hi);
    if (g < 0) return;   // the whole workgroup
    b_row0 = (int64_t)g * N * (SW ? 2 : 1);
  }
  const int64_t b_rows = (GROUPED ? (int64_t)G : 1) * N * (SW ? 2 : 1);
  const int nsl = (int)(K / 128);
  const int per = ((nsl + W - 1) / W + 1) & ~1;   // even: two slices are one 128-byte line
  const int s0 = w * per < nsl ? w * per : nsl;
  const int s1 = s0 + per < nsl ? s0 + per : nsl;
  const uint8_t* bp[NB];
  const uint32_t* bs[NB];
#pragma unroll
  for (int nb = 0; nb < NB; nb++) {
    const int64_t row = b_row0 + (SW ? nb * N + n0 : n0 + 16 * nb) + r;
    bp[nb] = B + row * (K / 2) + 16 * kg;
    bs[nb] = Bp + row;
  }
  v4f acc[MB][NB];
#pragma unroll
  for (int i = 0; i < MB; i++)
#pragma unroll
    for (int j = 0; j < NB; j++) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  int64_t arow[MB];   // rows past the end repeat the last one; their results are not stored
#pragma unroll
  for (int i = 0; i < MB; i++) arow[i] = m0 + 16 * i + r < hi ? m0 + 16 * i + r : hi - 1;
  for (int s = s0; s < s1; s += U) {
    u32x4 b[U][NB];
    uint32_t sb[U][NB];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int64_t k = s + u < s1 ? s + u : s1 - 1;
#pragma unroll
      for (int j = 0; j < NB; j++) {
        b[u][j] = *reinterpret_cast<const u32x4*>(bp[j] + k * 64);
        sb[u][j] = bs[j][k * b_rows];
      }
    }
#pragma unroll
    for (int i = 0; i < MB; i++) {
      if (m0 + 16 * i >= hi) break;
      u32x4 a[U];
      uint32_t sa[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int64_t k = s + u < s1 ? s + u : s1 - 1;
        a[u] = *reinterpret_cast<const u32x4*>(A + arow[i] * (K / 2) + k * 64 + 16 * kg);
        sa[u] = Ap[k * M + arow[i]];
      }
#pragma unroll
      for (int u = 0; u < U; u++)
        if (s + u < s1) {
#pragma unroll
          for (int j = 0; j < NB; j++)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                operand(b[u][j]), operand(a[u]), acc[i][j], 4, 4, 0, (int)(sb[u][j] >> (8 * kg)), 0,
                (int)(sa[u] >> (8 * kg)));
        }
    }
  }
#pragma unroll
  for (int i = 0; i < MB; i++)
#pragma unroll
    for (int j = 0; j < NB; j++) red[w][i][j][lane] = acc[i][j];
  __syncthreads();
  for (int x = threadIdx.x; x < MB * (SW ? 1 : NB) * 64; x += 64 * W) {
    const int i = x / ((SW ? 1 : NB) * 64), j = SW ? 0 : x / 64 % NB, ln = x & 63;
    const int64_t row = m0 + 16 * i + (ln & 15);
    v4f v = red[0][i][j][ln];
#pragma unroll
    for (int q = 1; q < W; q++) v += red[q][i][j][ln];
    if (SW) {
      v4f up = red[0][i][NB - 1][ln];
#pragma unroll
      for (int q = 1; q < W; q++) up += red[q][i][NB - 1][ln];
#pragma unroll
      for (int t = 0; t < 4; t++) v[t] = silu_f32(v[t]) * up[t];
    }
    if (row < hi) {
      u32x2* out = reinterpret_cast<u32x2*>(C + row * ldc + n0 + 16 * j + 4 * (ln >> 4));
      if (EPI == EPI_ACC) {
        const u32x2 o = *out;
#pragma unroll
        for (int t = 0; t < 4; t++) v[t] += bf16_half2(o, t);
      }
      const bf16x2 h0 = {(__bf16)v[0], (__bf16)v[1]};
      const bf16x2 h1 = {(__bf16)v[2], (__bf16)v[3]};
      *out = u32x2{__builtin_bit_cast(uint32_t, h0), __builtin_bit_cast(uint32_t, h1)};
    }
  }
}

static int64_t row_blocks(const Mx4Gemm& g, int64_t bm) { return g.offsets ? group_tiles(g.M, g.G, bm) : (g.M + bm - 1) / bm; }

template <int MB, int NB, int W, bool GROUPED, int EPI>
static hipError_t launch_rows(const Mx4Gemm& g, hipStream_t stream) {
  const int64_t tn = g.N / (EPI == EPI_SWIGLU ? 16 : 16 * NB);
  const int64_t ty = row_blocks(g, 16 * MB);
  hipLaunchKernelGGL((mx4_gemm_rows_kernel<MB, NB, W, GROUPED, EPI>), dim3((unsigned)tn, (unsigned)ty), dim3(64 * W), 0, stream,
                     g.a, g.ap, g.b, g.bp, g.c, g.ldc, g.M, g.N, g.K, g.offsets, g.G);
  return hipGetLastError();
}

// Whether workgroups take 16 columns instead of 32: where they are still at most
// one a compute unit, and K is so long that a wave's part of it is in flight at
// once with 16 columns (8 slices) and not with 32 (4).  5 x 256 x 7168: 5.3 us, with
// 32 columns 6.9; 29 x 1024 x 6144: 6.6 and 8.4; K = 4096 and less: 7 % slower.
static bool narrow_rows(const Mx4Gemm& g, int64_t bm) {
  return !g.offsets && g.epilogue != EPI_SWIGLU && g.K > 4096 && g.N / 16 * row_blocks(g, bm) <= 256;
}

// ---- choice of the kernel by estimated time.  Every variant was timed, as
// launches in a graph, on 1500 products: 1 .. 16384 rows, 256 .. 16384 columns,
// K 256 .. 8192, dense and in 2 .. 64 ragged groups, with and without SwiGLU.  The
// constants below are fitted to those times (microseconds; 7 to 10 % off, and the
// variant with the smallest estimate takes 1.6 % longer than the fastest one on
// average, 1.4 times as long at worst).  With b workgroups per compute unit and K
// in steps of 256:
//   64 x 64 .. 128 x 128  several workgroups fill each other's gaps: the longer of
//                         one workgroup's time and b times its share of the unit;
//   256 x 256             one workgroup a unit: rounds times (start and output +
//                         steps), a step slower the more units are busy;
//   few rows              a first round bound by latency, the others by loads.
// Dense products go by whole rounds, ragged groups by b and a part.  Each takes at
// least as long as the reading of B (the tiles: and the writing of C).  E.g.
// K = 4096, 512 x 4096: 10 us with 64 x 64 (512 tiles), 14 with 128 x 128, 24 with
// 256 x 256, 26 with the few-rows kernel; 4096 x 4096: 60, 43, 38 and over 200.
// 12126 rows in 7 groups, 2 x 576 x 768: 17 us with 128 x 128, 27 with 256 x 256.
struct Choice {
  Mx4Tile tile;
  int mb;   // few rows: blocks of 16 rows
};

static Choice choose(const Mx4Gemm& g) {
  const bool sw = g.epilogue == EPI_SWIGLU, ragged = g.offsets != nullptr;
  const double groups = ragged ? (double)(g.G < g.M ? g.G : g.M) : 1;   // that can have rows
  const double rows = (double)g.M / groups;                             // of a group, on average
  const int64_t n = sw ? 2 * g.N : g.N;
  const double steps = (double)((g.K + 255) / 256), k = (double)g.K / 4096;
  const double b_mb = groups * (double)n * (double)g.K * (17.0 / 32 / 1e6), c_mb = (double)g.M * (double)g.N * (2 / 1e6);
  // workgroups per compute unit; ragged groups end half a block early on average
  auto blocks = [&](int bm, int bn, bool few) {
    double down = (double)((g.M + bm - 1) / bm);
    if (ragged) {
      down = few && rows <= bm ? groups * (1 + 0.5 * rows / bm) : (double)g.M / bm + 0.5 * groups;
      const double least = few ? groups : 1;
      if (down < least) down = least;
    }
    return down * (double)((n + bn - 1) / bn) / 256;
  };
  auto rounds = [&](double b, double part) {
    const double r = ragged ? b + part : b < 6 ? (double)(int64_t)(b + 0.999) : b + 0.5;
    return r > 1 ? r : 1;
  };
  auto longer = [](double a, double b) { return a > b ? a : b; };
  Choice best{Mx4Tile::k256x256, 0};
  double least = 1e30;
  auto offer = [&](Mx4Tile tile, int mb, double us) {
    if (us < least) {
      least = us;
      best = Choice{tile, mb};
    }
  };
  static const struct { double call, k, fill, part, more_k, more_fill, tb_s; double start; } few[2] = {
      {3.30, 1.36, 0.82, 1.10, 1.27, 1.17, 6.72, 0.22}, {3.27, 1.35, 1.80, 1.09, 0.91, 2.14, 6.83, 0.32}};
  for (int i = 0; i < 2; i++) {
    const int bm = 16 << i;
    if (row_blocks(g, bm) > 65535) continue;   // the grid's second dimension
    const auto& f = few[i];
    const double fill = rows < bm ? rows / bm : 1;
    const double us = (f.start + k * (f.k + fill * f.fill)) * (narrow_rows(g, bm) ? 0.62 : 1) +
                      (rounds(blocks(bm, 32, true), f.part) - 1) * (f.start + k * (f.more_k + fill * f.more_fill));
    offer(Mx4Tile::kRows, 1 << i, f.call + longer(us, b_mb / f.tb_s));
  }
  static const struct { Mx4Tile tile; int bm, bn; double call, start, step, more_start, more_step, tb_s, part, swiglu; } mid[3] = {
      {Mx4Tile::k64x64, 64, 64, 3.63, 0.05, 0.238, 0.476, 0.234, 5.56, 0.69, 0},
      {Mx4Tile::k64x128, 64, 128, 3.93, -0.15, 0.427, 0.909, 0.416, 5.83, 0.43, 0.11},
      {Mx4Tile::k128x128, 128, 128, 4.65, -0.68, 0.748, 1.375, 0.669, 5.20, 0.19, 0.07}};
  if (mx4_gemm_mid_fits(g))
    for (const auto& t : mid) {
      if (sw && t.tile == Mx4Tile::k64x64) continue;
      const double b = blocks(t.bm, t.bn, false) + (ragged ? t.part : 0);
      const double us = longer(t.start + steps * t.step, b * (t.more_start + (sw ? t.swiglu : 0) + steps * t.more_step));
      offer(t.tile, 0, t.call + longer(us, (b_mb + c_mb) / t.tb_s));
    }
  if (mx4_gemm_tile_fits(g)) {
    const double b = blocks(256, 256, false), load = b < 1 ? b : 1;
    const double us = rounds(b, 0.53) * (7.3 + (sw ? 0.56 : 0) + steps * (0.953 + 0.777 * load));
    offer(Mx4Tile::k256x256, 0, 1.45 + longer(us, (b_mb + c_mb) / 3.47));
  }
  return best;
}

// Whether the chosen kernel's grid can be launched (where no variant's can, the
// choice is the largest tile).
bool mx4_gemm_grid_fits(const Mx4Gemm& g) {
  const Choice c = choose(g);
  if (c.tile == Mx4Tile::k256x256) return mx4_gemm_tile_fits(g);
  if (c.tile != Mx4Tile::kRows) return true;   // offered where it fits
  // a grid's dimensions are limited one by one: 2^32 - 1 work-items, 65535 workgroups of the second
  return grid_fits(g.N / 16, 1, 512) && row_blocks(g, 16 * c.mb) <= 65535;
}

template <int MB, int W, bool GROUPED>
static hipError_t launch_rows_e(const Mx4Gemm& g, hipStream_t stream) {
  return g.epilogue == EPI_SWIGLU ? launch_rows<MB, 2, W, GROUPED, EPI_SWIGLU>(g, stream)
       : g.epilogue == EPI_ACC   ? launch_rows<MB, 2, W, GROUPED, EPI_ACC>(g, stream)
                                 : launch_rows<MB, 2, W, GROUPED, EPI_NONE>(g, stream);
}
template <int MB>
static hipError_t launch_rows_w(const Mx4Gemm& g, hipStream_t stream) {
  if (narrow_rows(g, 16 * MB))
    return g.epilogue == EPI_ACC ? launch_rows<MB, 1, 8, false, EPI_ACC>(g, stream)
                                 : launch_rows<MB, 1, 8, false, EPI_NONE>(g, stream);
  // eight waves where K is long enough to be split and workgroups are few (one
  // row x 2048 columns, K = 8192: 6.3 us, with four waves 6.8; K = 1024, 256 x
  // 4096: 10.4 and 9.8; 32 experts of 2048 x 4096: 23 and 20)
  const int64_t tn = g.N / (g.epilogue == EPI_SWIGLU ? 16 : 32);
  if (g.K >= 2048 && tn * row_blocks(g, 16 * MB) < 1024) return g.offsets ? launch_rows_e<MB, 8, true>(g, stream) : launch_rows_e<MB, 8, false>(g, stream);
  return g.offsets ? launch_rows_e<MB, 4, true>(g, stream) : launch_rows_e<MB, 4, false>(g, stream);
}

hipError_t launch_mx4_gemm(const Mx4Gemm& g, hipStream_t stream) {
  const Choice c = choose(g);
  if (c.tile == Mx4Tile::k256x256) return launch_mx4_gemm_tile(g, stream);
  if (c.tile != Mx4Tile::kRows) return launch_mx4_gemm_mid(g, c.tile, stream);
  return c.mb == 1 ? launch_rows_w<1>(g, stream) : launch_rows_w<2>(g, stream);
}

}  // namespace mx
