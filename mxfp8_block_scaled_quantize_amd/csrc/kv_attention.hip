// Attention of a few queries over the paged MXFP4 cache, the joining of partial
// sums, and the choice of the kernel.
//
// Few rows: bound by the stream of the cache.  A wave takes 16 NB rows against 32
// keys at a time, all of it in registers: of 16 keys a lane loads 16 bytes of codes
// (32 values of one key) for the scores, and 16 bytes of value codes (4 keys x 8
// values).  Lane (c, g) = (l % 16, l / 16) gets the scores of row c and keys 4 g ..
// 4 g + 3 of each 16, which is where the second product wants them: its reduction
// runs over the keys in the order (4 g + 0..3 of the first 16, then of the second)
// for lane group g, and the values' codes stand in groups of four keys for that.
// The four waves of a workgroup take every fourth 32 keys; their maxima, sums and
// outputs meet in LDS at the end.
#include "kv_attention.h"

namespace mx {

using namespace kv;

namespace {

constexpr int WAVES = 4;

// Sum, or maximum, over the four lane groups (lanes 16 apart).
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float group_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// 32 keys of one head as a lane loads them.
template <int D>
struct Keys {
  static constexpr int KB = D == 256 ? 2 : 1;   // 16-byte pieces of a key (of 4 keys' values) a lane takes
  u32x4 k[2][KB], v[2][KB];
  uint32_t ks[2][KB], vs[2][KB];
  bool there[2];   // wave-uniform: the page is one

  __device__ __forceinline__ void load(const Args& a, const Tile& t, int head, int key, int end) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int page_size = 1 << a.page_shift;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int at = key + 16 * i;
      const uint8_t* r = at < end ? record_of(a, t, head, at) : nullptr;
      there[i] = r != nullptr;
      if (!r) r = a.cache;   // any record: what comes is not used
      const int o = at & (page_size - 1);
      const uint8_t* v0 = r + page_size * (D / 2);
      const uint8_t* ks0 = r + page_size * D;
      const uint8_t* vs0 = ks0 + page_size * (D / 32);
#pragma unroll
      for (int b = 0; b < KB; b++) {
        const int kb = D == 64 ? (g & 1) : g + 4 * b;              // block of 32 of the key
        const int vd = D == 64 ? (c & 7) : c + 16 * b;             // eight values
        k[i][b] = *reinterpret_cast<const u32x4*>(r + (o + c) * (D / 2) + 16 * kb);
        ks[i][b] = ks0[(o + c) * (D / 32) + kb];
        v[i][b] = *reinterpret_cast<const u32x4*>(v0 + ((o >> 2) + g) * (2 * D) + 16 * vd);
        vs[i][b] = *reinterpret_cast<const uint32_t*>(vs0 + (vd >> 2) * page_size + o + 4 * g);
      }
    }
  }
};

template <int D, int NB>
__global__ __launch_bounds__(64 * WAVES) void kv_attention_rows_kernel(Args a) {
  constexpr int TM = 16 * NB;
  constexpr int KB = Keys<D>::KB;
  constexpr int DT = D / 16;         // 16-row blocks of O^T
  constexpr int TERMS = D == 64 ? 1 : 2;
  __shared__ float meet[WAVES][4][64][4];
  __shared__ float stats[WAVES][NB][16][2];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int head = (int)(blockIdx.x % (unsigned)a.kv_heads);
  const int rest = (int)(blockIdx.x / (unsigned)a.kv_heads);
  const int part = rest % a.parts;
  Tile t;
  if (!find_tile<TM>(a, rest / a.parts, &t)) return;   // the whole workgroup
  const int rows = t.rows < TM ? t.rows : TM;
  const int64_t all_rows = (int64_t)a.tokens * a.heads;

  // keys of the tile's first and last query
  int first_lo, first_hi, last_lo, last_hi;
  seen(a, t, t.row0 / a.group, &first_lo, &first_hi);
  seen(a, t, (t.row0 + rows - 1) / a.group, &last_lo, &last_hi);
  const int begin = first_lo & ~31, end = last_hi;
  const int steps = (end - begin + 31) / 32;
  int each = (steps + a.parts - 1) / a.parts;
  each = (each + WAVES - 1) / WAVES * WAVES;
  const int s0 = part * each, s1 = s0 + each < steps ? s0 + each : steps;

  // the lane's rows: column c of each block
  int64_t token[NB];
  int q_head[NB], lo[NB], hi[NB];
  v8i qh[NB][KB], ql[NB][KB];
  int qs[NB];
#pragma unroll
  for (int n = 0; n < NB; n++) {
    const int row = 16 * n + c;
    const bool valid = row < rows;
    const int x = (t.row0 + (valid ? row : 0)) / a.group;
    token[n] = t.first_token + x;
    q_head[n] = head * a.group + (t.row0 + (valid ? row : 0)) - x * a.group;
    seen(a, t, x, &lo[n], &hi[n]);
    if (!valid) lo[n] = hi[n] = 0;
    const uint16_t* q = a.q + token[n] * a.q_token + q_head[n] * a.q_head;
    // bytes 0 .. 15 of the FP8 operand are dimensions 16 g + (0 .. 15), the others 64 + 16 g + ..;
    // for 64 dimensions the second half is `lo` of the same ones
    uint4 v[2 * KB][2];
    uint32_t m = 0;
#pragma unroll
    for (int b = 0; b < (D == 64 ? 1 : 2 * KB); b++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        v[b][i] = valid ? *reinterpret_cast<const uint4*>(q + 64 * b + 16 * g + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
        m = max(m, amax8(v[b][i]));
      }
    m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
    qs[n] = query_scale(m);
#pragma unroll
    for (int b = 0; b < KB; b++)
#pragma unroll
      for (int h = 0; h < (D == 64 ? 1 : 2); h++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
          uint32_t x2[2], y2[2];
          split8(v[2 * b + h][i], qs[n], x2, y2);
#pragma unroll
          for (int j = 0; j < 2; j++) {
            qh[n][b][4 * h + 2 * i + j] = (int)x2[j];
            if (D == 64) qh[n][b][4 + 2 * i + j] = (int)y2[j];
            else ql[n][b][4 * h + 2 * i + j] = (int)y2[j];
          }
        }
    if (D == 64 && g >= 2) qs[n] -= 4;   // blocks 2 and 3 of the operand are `lo`
  }

  v4f o[NB][DT];
  float top[NB], sum[NB];
#pragma unroll
  for (int n = 0; n < NB; n++) {
    top[n] = -INFINITY;
    sum[n] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; d++) o[n][d] = v4f{0.f, 0.f, 0.f, 0.f};
  }

  Keys<D> now, next;
  if (s0 + w < s1) now.load(a, t, head, begin + 32 * (s0 + w), end);
  for (int s = s0 + w; s < s1; s += WAVES) {
    const int key = begin + 32 * s;
    if (s + WAVES < s1) next.load(a, t, head, key + 32 * WAVES, end);
    // values of places that no query sees are taken as zeros, whatever they hold
    if (key + 32 > end || !now.there[0] || !now.there[1]) {
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int b = 0; b < KB; b++)
#pragma unroll
          for (int j = 0; j < 4; j++)
            if (!now.there[i] || key + 16 * i + 4 * g + j >= end) {
              now.v[i][b][j] = 0;
              now.vs[i][b] &= ~(0xFFu << (8 * j));
            }
    }
    bf16x8 p[NB];
#pragma unroll
    for (int n = 0; n < NB; n++) {
      v4f x[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        x[i] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < KB; b++) {
          v8i k{};
          k.lo = __builtin_bit_cast(v4i, now.k[i][b]);
          if (TERMS == 2)
            x[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, ql[n][b], x[i], 4, 0, 0, (int)now.ks[i][b], 0, qs[n] - 4);
          x[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, qh[n][b], x[i], 4, 0, 0, (int)now.ks[i][b], 0, qs[n]);
        }
      }
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const int at = key + 16 * i + 4 * g + j;
          x[i][j] = now.there[i] && at >= lo[n] && at < hi[n] ? x[i][j] * a.scale2 : -INFINITY;
          mx = fmaxf(mx, x[i][j]);
        }
      mx = group_max(mx);
      if (__any(mx > top[n])) {
        const float higher = fmaxf(mx, top[n]);
        const float shrink = higher > -INFINITY ? __builtin_amdgcn_exp2f(top[n] - higher) : 1.0f;
        top[n] = higher;
        sum[n] *= shrink;
#pragma unroll
        for (int d = 0; d < DT; d++) o[n][d] *= shrink;
      }
      const float base = top[n] > -INFINITY ? top[n] : 0.0f;
      float e[8];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        e[j] = __builtin_amdgcn_exp2f(x[j >> 2][j & 3] - base);
        sum[n] += e[j];
        p[n][j] = (__bf16)e[j];
      }
    }
#pragma unroll
    for (int b = 0; b < KB; b++) {
      uint32_t val[2][4][4];   // BF16 pairs of each key
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          // for 64 values lanes c and c + 8 take the halves of a word
          const uint32_t codes = D == 64 ? now.v[i][b][j] >> (c & 8 ? 16 : 0) : now.v[i][b][j];
          bf16_of(codes, scale_of(now.vs[i][b], j), val[i][j]);
        }
#pragma unroll
      for (int d = 0; d < (D == 64 ? 4 : 8); d++) {
        u32x4 word;
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
          for (int j = 0; j < 2; j++)
            word[2 * i + j] = (d & 1) ? highs(val[i][2 * j][d >> 1], val[i][2 * j + 1][d >> 1])
                                      : lows(val[i][2 * j][d >> 1], val[i][2 * j + 1][d >> 1]);
#pragma unroll
        for (int n = 0; n < NB; n++)
          o[n][8 * b + d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, word), p[n], o[n][8 * b + d], 0, 0, 0);
      }
    }
    now = next;
  }

  // the waves' sums meet
#pragma unroll
  for (int n = 0; n < NB; n++) {
    sum[n] = group_sum(sum[n]);
    if (g == 0) {
      stats[w][n][c][0] = top[n];
      stats[w][n][c][1] = sum[n];
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NB; n++) {
    float all = -INFINITY, total = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; i++) all = fmaxf(all, stats[i][n][c][0]);
    const float base = all > -INFINITY ? all : 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; i++) total += stats[i][n][c][1] * __builtin_amdgcn_exp2f(stats[i][n][c][0] - base);
    const float mine = __builtin_amdgcn_exp2f(top[n] - base);
    const bool valid = 16 * n + c < rows;
    const int64_t row = token[n] * a.heads + q_head[n];
    const float factor = a.sums ? 1.0f : (total > 0.0f || total != total ? 1.0f / total : 0.0f);
    if (valid && w == 0 && g == 0) {
      if (a.sums) {
        float* ml = a.sums + a.parts * all_rows * D + (part * all_rows + row) * 2;
        ml[0] = all;
        ml[1] = total;
      } else if (a.lse) {
        a.lse[row] = total > 0.0f || total != total ? (all + __builtin_amdgcn_logf(total)) * kLn2 : -INFINITY;
      }
    }
    if (a.sums && s0 >= s1) continue;   // the whole workgroup: nothing but the statistics
    // four blocks of O^T at a time: lane (c, g) of wave j then adds up registers j of
    // row c's blocks, four neighbouring dimensions
#pragma unroll
    for (int q = 0; q < DT / 4; q++) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; i++) *reinterpret_cast<v4f*>(meet[w][i][lane]) = o[n][4 * q + i] * mine;
      __syncthreads();
      float r[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {
        r[i] = 0.0f;
#pragma unroll
        for (int u = 0; u < WAVES; u++) r[i] += meet[u][i][lane][w];
        r[i] *= factor;
      }
      const int m = 4 * g + w;   // row of the blocks: (eight values, or half of them)
      const int d0 = D == 64 ? 8 * (m & 7) + 4 * (m >> 3) : 128 * (q >> 1) + 8 * m + 4 * (q & 1);
      if (valid) {
        if (a.sums) {
          *reinterpret_cast<v4f*>(a.sums + (part * all_rows + row) * D + d0) = v4f{r[0], r[1], r[2], r[3]};
        } else {
          *reinterpret_cast<u32x2*>(a.out + row * D + d0) = u32x2{bf16_pair(r[0], r[1]), bf16_pair(r[2], r[3])};
        }
      }
    }
  }
}

// ---- joining the parts of a row: a wave for each part in turn, a workgroup a row.
template <int D>
__global__ __launch_bounds__(64 * WAVES) void kv_join_kernel(Args a) {
  __shared__ float meet[WAVES][D];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t row = blockIdx.x, all_rows = (int64_t)a.tokens * a.heads;
  const int token = (int)(row / a.heads);
  if (a.offsets && (token < a.offsets[0] || token >= a.offsets[a.sequences])) return;
  const float* ml = a.sums + a.parts * all_rows * D + row * 2;
  float all = -INFINITY;
  for (int p = lane; p < a.parts; p += 64) all = fmaxf(all, ml[p * all_rows * 2]);
#pragma unroll
  for (int x = 32; x; x >>= 1) all = fmaxf(all, __shfl_xor(all, x, 64));
  const float base = all > -INFINITY ? all : 0.0f;
  float total = 0.0f;
  for (int p = lane; p < a.parts; p += 64) total += ml[p * all_rows * 2 + 1] * __builtin_amdgcn_exp2f(ml[p * all_rows * 2] - base);
#pragma unroll
  for (int x = 32; x; x >>= 1) total += __shfl_xor(total, x, 64);
  float r[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; i++) r[i] = 0.0f;
  for (int p = w; p < a.parts; p += WAVES) {
    const float m = ml[p * all_rows * 2], l = ml[p * all_rows * 2 + 1];
    if (l == 0.0f) continue;   // nothing there, not even zeros
    const float f = __builtin_amdgcn_exp2f(m - base);
    const float* o = a.sums + (p * all_rows + row) * D;
#pragma unroll
    for (int i = 0; i < D / 64; i++) r[i] += f * o[64 * i + lane];
  }
#pragma unroll
  for (int i = 0; i < D / 64; i++) meet[w][64 * i + lane] = r[i];
  __syncthreads();
  const bool some = total > 0.0f || total != total;
  if (threadIdx.x < D / 2) {
    float x = 0.0f, y = 0.0f;
#pragma unroll
    for (int u = 0; u < WAVES; u++) {
      x += meet[u][2 * threadIdx.x];
      y += meet[u][2 * threadIdx.x + 1];
    }
    const float factor = some ? 1.0f / total : 0.0f;
    reinterpret_cast<uint32_t*>(a.out + row * D)[threadIdx.x] = bf16_pair(x * factor, y * factor);
  }
  if (a.lse && threadIdx.x == 0) a.lse[row] = some ? (all + __builtin_amdgcn_logf(total)) * kLn2 : -INFINITY;
}

int64_t group_of(const KvAttention& a) { return a.heads / a.cache.heads; }

// Rows of a tile: 16 or 32 for a run of queries that fits, else 128 (the kernel for
// many queries).
int64_t rows_of(const KvAttention& a) {
  const int64_t rows = a.max_queries < 65536 ? a.max_queries * group_of(a) : 65536;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
}

// Parts that the keys of a tile are cut into.
int64_t parts_of(const KvAttention& a) {
  const int64_t tm = rows_of(a), blocks = kv_tiles(a, tm) * a.cache.heads;
  int64_t keys = a.table_width * a.cache.page_size;
  if (a.window > 0 && a.window + a.max_queries < keys) keys = a.window + a.max_queries;
  int64_t parts = (tm == 128 ? 512 : 1024) / (blocks > 0 ? blocks : 1);
  const int64_t most = keys / (tm == 128 ? 512 : 256);
  parts = parts < most ? parts : most;
  return parts < 1 ? 1 : parts > 64 ? 64 : parts;
}

template <int D>
hipError_t launch_all(const KvAttention& a, int64_t parts, hipStream_t stream) {
  const Args g = kv_args(a, parts);
  const int64_t tm = rows_of(a);
  const dim3 grid((unsigned)(kv_tiles(a, tm) * parts * a.cache.heads));
  hipError_t e = hipSuccess;
  if (tm == 128) {
    e = launch_kv_attention_tile(a, parts, stream);
  } else {
    if (tm == 16) hipLaunchKernelGGL((kv_attention_rows_kernel<D, 1>), grid, dim3(64 * WAVES), 0, stream, g);
    else hipLaunchKernelGGL((kv_attention_rows_kernel<D, 2>), grid, dim3(64 * WAVES), 0, stream, g);
    e = hipGetLastError();
  }
  if (e == hipSuccess && parts > 1) {
    hipLaunchKernelGGL(kv_join_kernel<D>, dim3((unsigned)(a.tokens * a.heads)), dim3(64 * WAVES), 0, stream, g);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

kv::Args kv_args(const KvAttention& a, int64_t parts) {
  kv::Args g{};
  g.q = a.q;
  g.q_token = a.q_token;
  g.q_head = a.q_head;
  g.cache = a.cache.data;
  g.record = a.cache.record();
  g.table = a.table;
  g.ld_table = a.ld_table;
  g.lengths = a.lengths;
  g.offsets = a.offsets;
  g.out = a.out;
  g.lse = a.lse;
  g.sums = parts > 1 ? a.workspace : nullptr;
  g.tokens = (int32_t)a.tokens;
  g.heads = a.heads;
  g.kv_heads = a.cache.heads;
  g.group = (int32_t)group_of(a);
  g.sequences = (int32_t)a.sequences;
  g.pages = (int32_t)a.cache.pages;
  g.page_shift = a.cache.page_shift;
  g.keys_most = (int32_t)(a.table_width * a.cache.page_size);
  g.window = a.window > 0x7FFFFFFF ? 0 : (int32_t)a.window;
  g.parts = (int32_t)parts;
  g.scale2 = a.scale * kLog2e;
  return g;
}

size_t kv_attention_workspace(const KvAttention& a) {
  const int64_t parts = parts_of(a);
  return parts > 1 ? (size_t)parts * (size_t)a.tokens * (size_t)a.heads * (size_t)(a.cache.head_dim + 2) * 4 : 0;
}

bool kv_attention_grid_fits(const KvAttention& a) {
  return grid_fits(kv_tiles(a, rows_of(a)) * parts_of(a), a.cache.heads, 64 * WAVES) && grid_fits(a.tokens, a.heads, 64 * WAVES);
}

hipError_t launch_kv_attention(const KvAttention& a, hipStream_t stream) {
  const int64_t parts = parts_of(a);
  if (a.cache.head_dim == 64) return launch_all<64>(a, parts, stream);
  if (a.cache.head_dim == 128) return launch_all<128>(a, parts, stream);
  return launch_all<256>(a, parts, stream);
}

}  // namespace mx
