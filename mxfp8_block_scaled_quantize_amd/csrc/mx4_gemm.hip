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

// Rows [lo, hi) of group g: e_i = max over j <= i of offsets[j] clamped into
// [0, M]; every wave of the workgroup computes the same.
__device__ __forceinline__ void group_rows(const int32_t* __restrict__ offsets, int g, int64_t M, int64_t* lo, int64_t* hi) {
  const int lane = threadIdx.x & 63;
  int m = 0;
  for (int j = lane; j <= g; j += 64) {
    const int v = offsets[j];
    m = v > m ? v : m;
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const int o = __shfl_xor(m, d, 64);
    m = m > o ? m : o;
  }
  m = __builtin_amdgcn_readfirstlane(m);
  const int h = __builtin_amdgcn_readfirstlane(offsets[g + 1]);
  const int64_t l = m < M ? m : M;
  const int64_t u = h < M ? h : M;
  *lo = l;
  *hi = u > l ? u : l;
}

// ---- few rows per group: bound by the stream of B.  W waves share 16 NB rows
// of B (SwiGLU: 16 gate rows and their 16 up rows) and up to 16 MB rows of A at
// a time, each wave a part of K.  Both operands go from global memory straight
// to registers in the matrix instructions' layout (16 rows x 64 bytes a load),
// several K slices in flight; the waves' sums meet in LDS.  Groups of more rows
// repeat the walk with B then in L2.  One row x 14336 columns, K = 4096: 7.4 us
// for 31 MB, of which 2 are the launch; 148 rows of 32 experts through 2048 x 4096
// weights (SwiGLU): 22.8 us for the 142 MB of all experts, 6.2 TB/s.
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
  int64_t lo, hi, b_row0 = 0;
  if (GROUPED) {
    // fewer workgroups than groups: one for each group that can have rows
    int g = blockIdx.y;
    if (gridDim.y < (unsigned)G) g = group_of_tile<0>(offsets, G, M, blockIdx.y, &lo, &hi);
    else group_rows(offsets, g, M, &lo, &hi);
    if (g < 0) return;
    b_row0 = (int64_t)g * N * (SW ? 2 : 1);
  } else {
    lo = (int64_t)blockIdx.y * 16 * MB;
    hi = lo + 16 * MB < M ? lo + 16 * MB : M;
  }
  if (lo >= hi) return;
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
  for (int64_t m0 = lo; m0 < hi; m0 += 16 * MB) {
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
    __syncthreads();
  }
}

template <int MB, int NB, int W, bool GROUPED, int EPI>
static hipError_t launch_rows(const Mx4Gemm& g, hipStream_t stream) {
  const int64_t tn = g.N / (EPI == EPI_SWIGLU ? 16 : 16 * NB);
  const int64_t ty = GROUPED ? (g.G < g.M ? g.G : g.M) : (g.M + 16 * MB - 1) / (16 * MB);
  hipLaunchKernelGGL((mx4_gemm_rows_kernel<MB, NB, W, GROUPED, EPI>), dim3((unsigned)tn, (unsigned)ty), dim3(64 * W), 0, stream,
                     g.a, g.ap, g.b, g.bp, g.c, g.ldc, g.M, g.N, g.K, g.offsets, g.G);
  return hipGetLastError();
}

// ---- choice of the kernel.  Every variant was timed over M x N (1 .. 4096
// rows, 512 .. 14336 columns) and over ragged groups, K 512 .. 8192, as launches
// in a graph.  A tile's time follows
//   K steps * max(one workgroup's time for a step,
//                 a full compute unit's time for it * tiles / 256),
// or that of reading B where it is longer, and the variant with the smallest
// estimate is taken.  In microseconds for a 256-element step (latency / share):
// 64 x 64 0.27 / 0.25, 64 x 128 0.45 / 0.43, 128 x 128 0.66 / 0.65; 256 x 256
// 1.3 for a lone tile, 2.2 for a full round of 256.  E.g. K = 4096, 512 x 4096:
// 10 us with 64 x 64 (512 tiles), 14 with 128 x 128, 24 with 256 x 256, 26 with
// the few-rows kernel; 4096 x 4096: 60, 43, 38 and over 200.  The few-rows
// kernel (16 MB rows x 32 columns a workgroup) takes per 256 workgroups a part
// for the columns and one that grows with the rows in a block: 128 rows x 1024
// columns 5.3 us, 6.3 with 64 x 64.  It streams B faster too (32 experts of 2048
// x 4096, one row each: 20 us, 28 with 64 x 128).
struct Choice {
  Mx4Tile tile;
  int mb;   // few rows: blocks of 16 rows
};

static Choice choose(const Mx4Gemm& g) {
  const bool sw = g.epilogue == EPI_SWIGLU;
  const double groups = g.offsets ? g.G : 1;
  const double rows = (double)g.M / groups;   // of a group, on average
  const double n = sw ? 2 * (double)g.N : (double)g.N;
  // workgroups per compute unit.  Ragged groups end half a block early on
  // average; the few-rows kernel, whose workgroup goes through all blocks of
  // its group, waits for the largest ones (`spread`).
  auto blocks = [&](int bm, int bn, int spread = 1) {
    double down = g.offsets ? spread * rows / bm + 0.5 : (double)((g.M + bm - 1) / bm);
    if (down < 1) down = 1;
    return groups * down * (double)(int64_t)((n + bn - 1) / bn) / 256;
  };
  const double steps = (double)((g.K + 255) / 256), k = steps / 16;
  const double b_bytes = groups * n * (double)g.K * 17 / 32;
  Choice best{Mx4Tile::k256x256, 0};
  double least = 1e30;
  auto offer = [&](Mx4Tile tile, int mb, double work, double read) {
    const double us = work > read ? work : read;
    if (us < least) {
      least = us;
      best = Choice{tile, mb};
    }
  };
  const double few[2][4] = {{0.45, 1.85, 0.75, -0.15}, {0.55, 1.7, 0.78, 0.77}};
  for (int i = 1; i >= 0; i--) {   // the larger block where both wait for B: ragged groups pass 16 rows
    const int bm = 16 << i;
    if (g.offsets || (g.M + bm - 1) / bm <= 65535) {   // the grid's second dimension
      const double b = blocks(bm, 32, 2), fill = rows < bm ? rows / bm : 1;
      const double* f = few[i];
      offer(Mx4Tile::kRows, 1 << i, (f[0] + f[1] * k + fill * (f[2] + f[3] * k)) * (b > 1 ? b : 1), b_bytes / 6.5e6);
    }
  }
  auto tiled = [&](Mx4Tile tile, double latency, double share, double b) {
    offer(tile, 0, steps * (latency > share * b ? latency : share * b), b_bytes / 5.2e6);
  };
  if (mx4_gemm_mid_fits(g)) {
    if (!sw) tiled(Mx4Tile::k64x64, 0.27, 0.25, blocks(64, 64));
    tiled(Mx4Tile::k64x128, 0.45, 0.43, blocks(64, 128));
    tiled(Mx4Tile::k128x128, 0.66, 0.65, blocks(128, 128));
  }
  if (mx4_gemm_tile_fits(g)) {
    const double b = blocks(256, 256);
    const double rounds = g.offsets ? b + 0.25 : (double)(int64_t)(b + 0.999);
    offer(Mx4Tile::k256x256, 0, steps * (b <= 1 ? 1.3 + 0.9 * b : 2.1 * rounds), b_bytes / 5.2e6);
  }
  return best;
}

bool mx4_gemm_grid_fits(const Mx4Gemm& g) {
  // a grid's dimensions are limited one by one: 2^32 - 1 work-items, 65535 workgroups of the second
  return choose(g).tile != Mx4Tile::kRows || (grid_fits(g.N / 16, 1, 512) && (g.offsets || (g.M + 15) / 16 <= 65535));
}

template <int MB, int W, bool GROUPED>
static hipError_t launch_rows_e(const Mx4Gemm& g, hipStream_t stream) {
  return g.epilogue == EPI_SWIGLU ? launch_rows<MB, 2, W, GROUPED, EPI_SWIGLU>(g, stream)
       : g.epilogue == EPI_ACC   ? launch_rows<MB, 2, W, GROUPED, EPI_ACC>(g, stream)
                                 : launch_rows<MB, 2, W, GROUPED, EPI_NONE>(g, stream);
}
template <int MB>
static hipError_t launch_rows_w(const Mx4Gemm& g, hipStream_t stream) {
  // eight waves where K is long enough to be split and workgroups are few (one
  // row x 2048 columns, K = 8192: 6.3 us, with four waves 6.8; K = 1024, 256 x
  // 4096: 10.4 and 9.8; 32 experts of 2048 x 4096: 23 and 20)
  const int64_t tn = g.N / (g.epilogue == EPI_SWIGLU ? 16 : 32);
  const int64_t groups = g.offsets ? (g.G < g.M ? g.G : g.M) : (g.M + 16 * MB - 1) / (16 * MB);
  if (g.K >= 2048 && tn * groups < 1024) return g.offsets ? launch_rows_e<MB, 8, true>(g, stream) : launch_rows_e<MB, 8, false>(g, stream);
  return g.offsets ? launch_rows_e<MB, 4, true>(g, stream) : launch_rows_e<MB, 4, false>(g, stream);
}

hipError_t launch_mx4_gemm(const Mx4Gemm& g, hipStream_t stream) {
  const Choice c = choose(g);
  if (c.tile == Mx4Tile::k256x256) return launch_mx4_gemm_tile(g, stream);
  if (c.tile != Mx4Tile::kRows) return launch_mx4_gemm_mid(g, c.tile, stream);
  return c.mb == 1 ? launch_rows_w<1>(g, stream) : launch_rows_w<2>(g, stream);
}

}  // namespace mx
