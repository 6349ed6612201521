// Block-scaled MXFP4 GEMM (TN) on the gfx950 scaled FP4 matrix instructions.
//
//   C[m][n] = bf16( sum_k dq(A)[m][k] dq(B)[n][k] ), fp32 accumulation.
//
// Operand layout of V_MFMA_SCALE_F32_16X16X128_F8F6F4 with E2M1 on both sides:
// lane l holds row l % 16, K = 32 (l / 16) + [0, 32) in its 16 bytes (one scale
// block), and supplies that block's scale byte.  Result register i of lane l is
// row 4 (l / 16) + i of the first operand, row l % 16 of the second.  The
// kernels pass B first: a lane holds four consecutive columns of one row of C.
#include "mx_device.h"
#include "launch.h"

namespace mx {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v8i fp4_operand(u32x4 d) {   // an FP4 operand takes the low four registers
  v8i r;
  r.lo = __builtin_bit_cast(v4i, d);
  return r;
}

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
// repeat the walk with B then in L2.
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
    group_rows(offsets, blockIdx.y, M, &lo, &hi);
    b_row0 = (int64_t)blockIdx.y * N * (SW ? 2 : 1);
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
                  fp4_operand(b[u][j]), fp4_operand(a[u]), acc[i][j], 4, 4, 0, (int)(sb[u][j] >> (8 * kg)), 0,
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
  const int64_t ty = GROUPED ? g.G : (g.M + 16 * MB - 1) / (16 * MB);
  hipLaunchKernelGGL((mx4_gemm_rows_kernel<MB, NB, W, GROUPED, EPI>), dim3((unsigned)tn, (unsigned)ty), dim3(64 * W), 0, stream,
                     g.a, g.ap, g.b, g.bp, g.c, g.ldc, g.M, g.N, g.K, g.offsets, g.G);
  return hipGetLastError();
}

// Rows of a group on average (dense: all rows).
static int64_t rows_per_group(const Mx4Gemm& g) { return g.offsets ? (g.M + g.G - 1) / g.G : g.M; }
static bool few_rows(const Mx4Gemm& g) { return rows_per_group(g) <= 256; }

bool mx4_gemm_grid_fits(const Mx4Gemm& g) { return few_rows(g) ? grid_fits(g.M + g.G, g.N / 16, 256) : mx4_gemm_tile_fits(g); }

hipError_t launch_mx4_gemm(const Mx4Gemm& g, hipStream_t stream) {
  if (!few_rows(g)) return launch_mx4_gemm_tile(g, stream);
  const bool grouped = g.offsets != nullptr;
  if (grouped) {
    if (g.epilogue == EPI_SWIGLU) return launch_rows<2, 2, 4, true, EPI_SWIGLU>(g, stream);
    if (g.epilogue == EPI_ACC) return launch_rows<2, 2, 4, true, EPI_ACC>(g, stream);
    return launch_rows<2, 2, 4, true, EPI_NONE>(g, stream);
  }
  if (g.epilogue == EPI_SWIGLU) return launch_rows<2, 2, 4, false, EPI_SWIGLU>(g, stream);
  if (g.epilogue == EPI_ACC) return launch_rows<2, 2, 4, false, EPI_ACC>(g, stream);
  return launch_rows<2, 2, 4, false, EPI_NONE>(g, stream);
}

}  // namespace mx
