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
//
// Measured (32 heads, 8 of keys, of 128): 64 sequences of up to 8192 tokens, 358 MB in 66 us,
// 5.4 TB/s (a plain sum over as many bytes reaches 6.3; this kernel's loads alone take 64);
// one of 131071, 143 MB in 26 us, and 4 for the join.  Two steps of a wave are on their
// way, with 4 waves a SIMD: three steps, or fewer waves, were slower.  Of the chip's time the
// matrix cores work 12 %, the vector unit 30; with 64 values 7 and 29 (16 sequences of 16384
// keys, 143 MB in 39 us: a workgroup a compute unit then has half the bytes on their way).
#include "kv_attention.h"

namespace mx {

using namespace kv;

namespace {

constexpr int WAVES = 4, DEPTH = 2;   // DEPTH: steps on their way
// Codes are read once: non-temporal loads (64 sequences of up to 8192 tokens: 70 us, 77 without).
constexpr int NT = 2;

// Maximum, or sum, over the four lane groups (lanes 16 apart): swapping rows of 16
// (of 32) between two copies leaves each lane with its own and its partner's value.
__device__ __forceinline__ float group_max(float v) {
  const uint32_t x = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  const uint32_t y = __float_as_uint(fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1])));
  const auto b = __builtin_amdgcn_permlane32_swap(y, y, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float group_sum(float v) {
  const uint32_t x = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  const uint32_t y = __float_as_uint(__uint_as_float(a[0]) + __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(y, y, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Page numbers of a step's two runs of 16 keys.
struct Pages {
  int p[2];
  __device__ __forceinline__ void find(const Args& a, const Tile& t, int key, int end) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int at = key + 16 * i < end ? key + 16 * i : end - 1;
      p[i] = a.table[t.sequence * a.ld_table + (at >> a.page_shift)];
    }
  }
};

// 32 keys of one head as a lane loads them.
template <int D>
struct Keys {
  static constexpr int KB = D == 256 ? 2 : 1;   // 16-byte pieces of a key (of 4 keys' values) a lane takes
  u32x4 k[2][KB], v[2][KB];
  uint32_t ks[2][KB], vs[2][KB];
  bool there[2];   // wave-uniform: the page is one

  // No branch, so that the compiler can wait for one step's loads among those of the
  // next ones: what is not there (no page, or `wanted` false) is an empty buffer,
  // which reads as zeros.
  __device__ __forceinline__ void load(const Args& a, const Pages& pages, int head, int key, bool wanted) {
    const uint32_t lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const uint32_t page_size = 1u << a.page_shift;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      there[i] = (unsigned)pages.p[i] < (unsigned)a.pages;
      const int page = there[i] ? pages.p[i] : 0;
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t*>(record_of(a, head, page)), 0, there[i] && wanted ? (int)a.record : 0,
          0x00020000);
      const int o = (key + 16 * i) & (int)(page_size - 1);
      const int k0 = o * (D / 2), v0 = page_size * (D / 2) + (o >> 2) * (2 * D);
      const int ks0 = page_size * D + o * (D / 32), vs0 = page_size * (D + D / 32) + o;
#pragma unroll
      for (int b = 0; b < KB; b++) {
        const uint32_t kb = D == 64 ? (g & 1) : g + 4 * b;              // block of 32 of the key
        const uint32_t vd = D == 64 ? (c & 7) : c + 16 * b;             // eight values
        k[i][b] = __builtin_amdgcn_raw_buffer_load_b128(r, c * (D / 2) + 16 * kb, k0, NT);
        ks[i][b] = __builtin_amdgcn_raw_buffer_load_b8(r, c * (D / 32) + kb, ks0, 0);
        v[i][b] = __builtin_amdgcn_raw_buffer_load_b128(r, g * (2 * D) + 16 * vd, v0, NT);
        vs[i][b] = __builtin_amdgcn_raw_buffer_load_b32(r, (vd >> 2) * page_size + 4 * g, vs0, 0);
      }
    }
  }
};

template <int D, int NB>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 3 - NB : NB == 1 ? 4 : D == 64 ? 3 : 2) void kv_attention_rows_kernel(Args a) {
  constexpr int TM = 16 * NB;
  constexpr int KB = Keys<D>::KB;
  constexpr int DT = D / 16;         // 16-row blocks of O^T
  constexpr int TERMS = D == 64 ? 1 : 2;
  constexpr int CH = DT < 8 ? DT : 8;   // blocks that meet at a time
  __shared__ __attribute__((aligned(16))) float meet[WAVES][CH][64][4];
  __shared__ float stats[WAVES][16][2];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const Place place(a);
  const int head = place.head, part = place.part;
  Tile t;
  if (!find_tile<TM>(a, place.tile, &t)) return;   // the whole workgroup
  const int rows = t.rows < TM ? t.rows : TM;
  const int64_t all_rows = (int64_t)a.tokens * a.heads;

  // keys of the tile's first and last query
  int first_lo, first_hi, last_lo, last_hi;
  seen(a, t, t.row0 / a.group, &first_lo, &first_hi);
  seen(a, t, (t.row0 + rows - 1) / a.group, &last_lo, &last_hi);
  const int end = last_hi, begin = first_lo < end ? first_lo & ~31 : 0;   // (behind the table first_lo may be near 2^31)
  const int steps = first_lo < end ? (end - begin + 31) / 32 : 0;
  const int each = steps ? (part_steps<32>(a, steps) + WAVES - 1) / WAVES * WAVES : 1;
  const int used = (steps + each - 1) / each;
  if (part > 0 && part >= used) return;
  const bool whole = used <= 1;   // the outputs are written here
  const int s0 = part * each, s1 = s0 + each < steps ? s0 + each : steps;

  // the lane's rows: column c of each block
  int64_t token[NB];
  int q_head[NB], lo[NB], hi[NB];
  uint4 qv[NB][2 * KB][2];
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
#pragma unroll
    for (int b = 0; b < (D == 64 ? 1 : 2 * KB); b++)
#pragma unroll
      for (int i = 0; i < 2; i++) qv[n][b][i] = *reinterpret_cast<const uint4*>(q + 64 * b + 16 * g + 8 * i);
  }

  // DEPTH steps of the wave are on their way, and the page numbers of one more
  Keys<D> ring[DEPTH];
  Pages pages;
  const int stride = 32 * WAVES, first = begin + 32 * (s0 + w), last = s0 < s1 ? begin + 32 * s1 : 0;
  if (steps > 0) {
    pages.find(a, t, first, end);
#pragma unroll
    for (int u = 0; u < DEPTH; u++) {
      ring[u].load(a, pages, head, first + u * stride, first + u * stride < last);
      pages.find(a, t, first + (u + 1) * stride, end);
      __builtin_amdgcn_sched_barrier(0);   // the steps' loads in the order of the loop
    }
  }

  v8i qh[NB][KB], ql[NB][KB];
  int qs[NB];
#pragma unroll
  for (int n = 0; n < NB; n++) {
    const bool valid = 16 * n + c < rows;
    uint32_t m = 0;
#pragma unroll
    for (int b = 0; b < (D == 64 ? 1 : 2 * KB); b++)
#pragma unroll
      for (int i = 0; i < 2; i++) {
        if (!valid) qv[n][b][i] = make_uint4(0u, 0u, 0u, 0u);
        m = max(m, amax8(qv[n][b][i]));
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
          split8(qv[n][2 * b + h][i], qs[n], x2, y2);
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

  // what every query of the tile sees: nothing where one sees none, whose lo is no less than its hi
  const int full_lo = last_lo, full_hi = first_hi;
  auto step = [&](Keys<D>& now, const int key) {
    // values of places that no query of the tile sees, in front of its first one's window or
    // behind its last one, are taken as zeros, whatever they hold
    if (key < first_lo || key + 32 > end) {
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int b = 0; b < KB; b++)
#pragma unroll
          for (int j = 0; j < 4; j++)
            if (key + 16 * i + 4 * g + j < first_lo || key + 16 * i + 4 * g + j >= end) {
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
      if (!(key >= full_lo && key + 32 <= full_hi && now.there[0] && now.there[1])) {
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const int at = key + 16 * i + 4 * g + j;
            if (!(now.there[i] && at >= lo[n] && at < hi[n])) x[i][j] = -INFINITY;
          }
      }
#pragma unroll
      for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) mx = fmaxf(mx, x[i][j]);
      mx = group_max(mx * a.scale2);
      if (__any(mx > top[n] + 8.0f)) {   // the maximum may be 8 too low: see kv_attention.h
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
        e[j] = __builtin_amdgcn_exp2f(fmaf(x[j >> 2][j & 3], a.scale2, -base));
        sum[n] += e[j];
        p[n][j] = (__bf16)e[j];
      }
    }
#pragma unroll
    for (int b = 0; b < KB; b++) {
#pragma unroll
      for (int x = 0; x < (D == 64 ? 2 : 4); x++) {   // two of the eight (four) values at a time
        uint32_t val[2][4];
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
          for (int j = 0; j < 4; j++) {
            // for 64 values lanes c and c + 8 take the halves of a word
            const uint32_t codes = D == 64 ? now.v[i][b][j] >> (c & 8 ? 16 : 0) : now.v[i][b][j];
            val[i][j] = bf16_pair_of(codes, scale_of(now.vs[i][b], j), x);
          }
        const u32x4 even = {lows(val[0][0], val[0][1]), lows(val[0][2], val[0][3]), lows(val[1][0], val[1][1]), lows(val[1][2], val[1][3])};
        const u32x4 odd = {highs(val[0][0], val[0][1]), highs(val[0][2], val[0][3]), highs(val[1][0], val[1][1]), highs(val[1][2], val[1][3])};
#pragma unroll
        for (int n = 0; n < NB; n++) {
          v4f &o0 = o[n][8 * b + 2 * x], &o1 = o[n][8 * b + 2 * x + 1];
          o0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, even), p[n], o0, 0, 0, 0);
          o1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, odd), p[n], o1, 0, 0, 0);
        }
      }
    }
  };

  for (int key = first; key < last; key += DEPTH * stride) {
#pragma unroll
    for (int u = 0; u < DEPTH; u++) {
      const int at = key + u * stride, to = at + DEPTH * stride;
      if (at < last) step(ring[u], at);
      ring[u].load(a, pages, head, to, to < last);
      pages.find(a, t, to + stride, end);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // the waves' sums meet: lane (c, g) of wave j adds up registers j of row c's blocks of
  // O^T, four at a time, which are neighbouring dimensions
#pragma unroll
  for (int n = 0; n < NB; n++) {
    sum[n] = group_sum(sum[n]);
    if (n) __syncthreads();
    if (g == 0) {
      stats[w][c][0] = top[n];
      stats[w][c][1] = sum[n];
    }
    const bool valid = 16 * n + c < rows;
    const int64_t row = token[n] * a.heads + q_head[n];
    float part_of[WAVES], factor = 1.0f;
#pragma unroll
    for (int d0 = 0; d0 < DT; d0 += CH) {
      if (d0) __syncthreads();
#pragma unroll
      for (int d = 0; d < CH; d++) *reinterpret_cast<v4f*>(meet[w][d][lane]) = o[n][d0 + d];
      __syncthreads();
      if (d0 == 0) {
        float all = -INFINITY, total = 0.0f;
#pragma unroll
        for (int u = 0; u < WAVES; u++) all = fmaxf(all, stats[u][c][0]);
        const float base = all > -INFINITY ? all : 0.0f;
#pragma unroll
        for (int u = 0; u < WAVES; u++) {
          part_of[u] = __builtin_amdgcn_exp2f(stats[u][c][0] - base);
          total += stats[u][c][1] * part_of[u];
        }
        const bool some = total > 0.0f || total != total;
        if (whole) factor = some ? 1.0f / total : 0.0f;
        if (valid && w == 0 && g == 0) {
          if (!whole) {
            float* ml = a.sums + a.parts * all_rows * D + (part * all_rows + row) * 2;
            ml[0] = all;
            ml[1] = total;
          } else if (a.lse) {
            a.lse[row] = some ? (all + __builtin_amdgcn_logf(total)) * kLn2 : -INFINITY;
          }
          if (a.sums && part == 0) a.used[row] = used;
        }
      }
      if (valid) {
#pragma unroll
        for (int q = 0; q < CH / 4; q++) {
          float r[4];
#pragma unroll
          for (int i = 0; i < 4; i++) {
            r[i] = 0.0f;
#pragma unroll
            for (int u = 0; u < WAVES; u++) r[i] += meet[u][4 * q + i][lane][w] * part_of[u];
            r[i] *= factor;
          }
          const int m = 4 * g + w;   // row of the blocks: (eight values, or half of them)
          const int to = D == 64 ? 8 * (m & 7) + 4 * (m >> 3) : 16 * d0 + 8 * m + 4 * q;
          if (!whole) *reinterpret_cast<v4f*>(a.sums + (part * all_rows + row) * D + to) = v4f{r[0], r[1], r[2], r[3]};
          else *reinterpret_cast<u32x2*>(a.out + row * D + to) = u32x2{bf16_pair(r[0], r[1]), bf16_pair(r[2], r[3])};
        }
      }
    }
  }
}

// ---- joining the parts of a row: bound by the stream of the parts' sums for many rows, by
// three loads' latency for few.  G waves have a row (4 / G rows a workgroup), lane p part p's
// maximum and sum (64 parts at most), every lane 2 (of 256: 4) of the outputs.  What the
// places behind a row's parts hold is not loaded, but for the statistics, which are not taken.
// 16000 rows of 4 parts of 128: 10 us, 39 MB; 32 rows of 32 parts: 4.4.
template <int D, int G>
__global__ __launch_bounds__(64 * WAVES) void kv_join_kernel(Args a) {
  constexpr int V = D == 256 ? 4 : 2, PER = 64 * V / D, AHEAD = 4;   // outputs of a lane; parts that a wave's lanes take at a time
  typedef float vec __attribute__((ext_vector_type(V)));
  __shared__ __attribute__((aligned(16))) float meet[G == 1 ? 1 : WAVES][D];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t row = G == 1 ? (int64_t)blockIdx.x * WAVES + w : blockIdx.x, all_rows = (int64_t)a.tokens * a.heads;
  if (row >= all_rows) return;
  const int token = (int)(row / a.heads);
  if (a.offsets) {   // rows of no sequence; the offsets' running maximum is what counts
    if (token < a.offsets[0]) return;
    int end = a.offsets[a.sequences];
    if (token >= end) {
      for (int i = lane; i < a.sequences; i += 64) end = max(end, a.offsets[i]);
      if (!__any(token < end)) return;   // the same for all waves of the row
    }
  }
  const f32x2* const ml = reinterpret_cast<const f32x2*>(a.sums + a.parts * all_rows * D) + row;
  f32x2 stat = {-INFINITY, 0.0f};
  if (lane < a.parts) stat = ml[lane * all_rows];
  const int used = __builtin_amdgcn_readfirstlane(a.used[row]);   // the row's, in all lanes
  if (used <= 1) return;
  const int at = (lane & (D / V - 1)) * V, mine = lane / (D / V), step = G * PER;
  const float* const o = a.sums + row * D + at;
  auto load = [&](vec* x, int p0) {
#pragma unroll
    for (int u = 0; u < AHEAD; u++) x[u] = *reinterpret_cast<const vec*>(o + min(p0 + u * step + mine, used - 1) * all_rows * D);
  };
  vec x[AHEAD], r;
  const int first = (G == 1 ? 0 : w) * PER;
  load(x, first);
  if (lane >= used) stat = f32x2{-INFINITY, 0.0f};
  float all = stat.x;
#pragma unroll
  for (int i = 32; i; i >>= 1) all = fmaxf(all, __shfl_xor(all, i, 64));
  const float base = all > -INFINITY ? all : 0.0f;
  // a part that the row sees nothing of is not taken: -1
  const float f = stat.y == 0.0f ? -1.0f : __builtin_amdgcn_exp2f(stat.x - base);
  float total = stat.y == 0.0f ? 0.0f : stat.y * f;
#pragma unroll
  for (int i = 32; i; i >>= 1) total += __shfl_xor(total, i, 64);
#pragma unroll
  for (int i = 0; i < V; i++) r[i] = 0.0f;
  for (int p0 = first; p0 < used; p0 += AHEAD * step) {
    if (p0 > first) load(x, p0);
#pragma unroll
    for (int u = 0; u < AHEAD; u++) {
      const int p = p0 + u * step + mine;
      const float fp = __shfl(f, p < used ? p : 0, 64);
      const bool take = p < used && !(fp < 0.0f);   // NaN too
#pragma unroll
      for (int i = 0; i < V; i++) r[i] = take ? fmaf(fp, x[u][i], r[i]) : r[i];
    }
  }
  if (PER == 2)
#pragma unroll
    for (int i = 0; i < V; i++) r[i] += __shfl_xor(r[i], 32, 64);
  if (G > 1) {
    if (mine == 0) *reinterpret_cast<vec*>(&meet[w][at]) = r;
    __syncthreads();
    if (w > 0) return;
    r = *reinterpret_cast<const vec*>(&meet[0][at]);
#pragma unroll
    for (int u = 1; u < WAVES; u++) r += *reinterpret_cast<const vec*>(&meet[u][at]);
  }
  const bool some = total > 0.0f || total != total;
  const float factor = some ? 1.0f / total : 0.0f;
  if (mine == 0)
#pragma unroll
    for (int i = 0; i < V; i += 2) reinterpret_cast<uint32_t*>(a.out + row * D + at)[i / 2] = bf16_pair(r[i] * factor, r[i + 1] * factor);
  if (a.lse && lane == 0) a.lse[row] = some ? (all + __builtin_amdgcn_logf(total)) * kLn2 : -INFINITY;
}

int64_t group_of(const KvAttention& a) { return a.heads / a.cache.heads; }

// Places for parts, a lane each in kv_join_kernel, and bytes of their sums: 512 tiles of 128
// rows of 256 values, which fill the chip, take 68 MB.  Workgroups for places that nothing but
// the table's width asks for: 64 sequences of up to 8192 tokens in a table of 2^20 take 66 us
// with one place, 68 with 8, 84 with 64.
constexpr int64_t MOST_PARTS = 64, MOST_BYTES = 80ll << 20, MOST_BLOCKS = 8192;

// Keys that a tile can see.
int64_t keys_of(const KvAttention& a) {
  const int64_t keys = a.table_width * a.cache.page_size;
  return a.window > 0 && a.window + a.max_queries < keys ? a.window + a.max_queries : keys;
}
// Tiles of tm rows: as many as runs of max_queries have, if that is less than what any offsets
// can give; and those times heads.
int64_t likely_tiles(const KvAttention& a, int64_t tm) {
  const int64_t tiles = kv_tiles(a, tm);
  if (!a.offsets || a.max_queries >= 65536) return tiles;
  const int64_t likely = a.sequences * ((a.max_queries * group_of(a) + tm - 1) / tm);
  return tiles < likely ? tiles : likely;
}
int64_t blocks_of(const KvAttention& a, int64_t tm) { return likely_tiles(a, tm) * a.cache.heads; }
// Rows of a tile: 16 or 32 for a run of queries that fits, else 128, or 64 (the kernel for
// many queries).  64 rows leave no wave idle where a run has no more, but two waves then do
// what four do for the values: of 256 values, where registers leave a SIMD one wave, it is
// faster everywhere (36 rows of 16 sequences of 16384 keys: 201 us, 318 with 128 rows; 64 of
// 2048: 104 and 166; one of 65536: 64 and 97), else where the keys give four workgroups a
// compute unit (of 128 values: 96 and 118, 56 and 61; one sequence, 512 workgroups: 43 and 40;
// of 64: 72 and 96, 52 and 50, 37 and 33).
constexpr int64_t FILL_64 = 1024;
int64_t rows_of(const KvAttention& a) {
  const int64_t rows = a.max_queries < 65536 ? a.max_queries * group_of(a) : 65536;
  if (rows <= 32) return rows <= 16 ? 16 : 32;
  if (rows > 64) return 128;
  const int64_t most = keys_of(a) / LEAST_KEYS;
  return a.cache.head_dim == 256 || blocks_of(a, 64) * (most < MOST_PARTS ? most : MOST_PARTS) >= FILL_64 ? 64 : 128;
}

// Of a tile's keys: the parts that give every compute unit a workgroup (of the kernel for
// many queries as many as it holds), and the places that the table's width may want for them,
// as far as their sums and the grid have room.  How many a tile really has is settled on the
// device (part_steps).  One token of a sequence of 131071 keys, 8 heads: 30 us with 32 parts,
// 29 with 64, 46 with 16; of 2048 keys: 11.4 with 4, 14.0 with 1; 64 sequences of up to 8192:
// 66 us with 1 part, 70 with 2 and with 4; 500 queries over 49152 keys: 379 with 4, 447 with 3,
// 384 with 8.
struct Parts {
  int64_t fill, places;
};
Parts parts_of(const KvAttention& a) {
  const int64_t tm = rows_of(a), blocks = blocks_of(a, tm), keys = keys_of(a), rows = a.tokens * a.heads;
  const int64_t wanted = tm < 64 ? 256 : tm == 64 && a.cache.head_dim < 256 ? FILL_64 : 512;
  const auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
  const int64_t most = least(keys / LEAST_KEYS, MOST_PARTS);
  Parts p{least(wanted / (blocks > 0 ? blocks : 1), most), least((keys + MOST_KEYS - 1) / MOST_KEYS, most)};
  p.fill = p.fill < 1 ? 1 : p.fill;
  if (blocks > 0) p.places = least(p.places, MOST_BLOCKS / blocks);
  p.places = p.fill > p.places ? p.fill : p.places;
  if (rows > 0) p.places = least(p.places, (MOST_BYTES / rows / 4 - 1) / (a.cache.head_dim + 2));
  const int64_t tiles = kv_tiles(a, tm) * a.cache.heads;
  if (tiles > 0) p.places = least(p.places, kMaxWorkItems / (64 * WAVES) / tiles);
  p.places = p.places < 1 ? 1 : p.places;
  return p;
}

template <int D>
hipError_t launch_all(const KvAttention& a, const Args& g, hipStream_t stream) {
  const int64_t tm = rows_of(a);
  const dim3 grid((unsigned)g.tiles * (unsigned)g.parts * (unsigned)a.cache.heads);
  hipError_t e = hipSuccess;
  if (tm >= 64) {
    e = launch_kv_attention_tile(a.cache, g, tm, grid, stream);
  } else {
    if (tm == 16) hipLaunchKernelGGL((kv_attention_rows_kernel<D, 1>), grid, dim3(64 * WAVES), 0, stream, g);
    else hipLaunchKernelGGL((kv_attention_rows_kernel<D, 2>), grid, dim3(64 * WAVES), 0, stream, g);
    e = hipGetLastError();
  }
  if (e == hipSuccess && g.parts > 1) {
    // four waves a row where one would go through the parts in more than two rounds; the rows
    // that MOST_BYTES has room for fit a grid in either form
    const int64_t rows = a.tokens * a.heads;
    if (g.parts <= 8) hipLaunchKernelGGL((kv_join_kernel<D, 1>), dim3((unsigned)((rows + WAVES - 1) / WAVES)), dim3(64 * WAVES), 0, stream, g);
    else hipLaunchKernelGGL((kv_join_kernel<D, WAVES>), dim3((unsigned)rows), dim3(64 * WAVES), 0, stream, g);
    e = hipGetLastError();
  }
  return e;
}

kv::Args kv_args(const KvAttention& a, Parts parts) {
  kv::Args g{};
  g.q = a.q;
  g.q_token = a.q_token;
  g.q_head = a.q_head;
  g.cache = a.cache.data;
  g.record = a.cache.record();
  g.page_stride = (uint32_t)(a.cache.record() * a.cache.heads);
  g.table = a.table;
  g.ld_table = a.ld_table;
  g.lengths = a.lengths;
  g.offsets = a.offsets;
  g.out = a.out;
  g.lse = a.lse;
  if (parts.places > 1) {
    g.sums = a.workspace;
    g.used = reinterpret_cast<int32_t*>(a.workspace + parts.places * a.tokens * a.heads * (a.cache.head_dim + 2));
  }
  g.tokens = (int32_t)a.tokens;
  g.heads = a.heads;
  g.kv_heads = a.cache.heads;
  g.group = (int32_t)group_of(a);
  g.sequences = (int32_t)a.sequences;
  g.pages = (int32_t)a.cache.pages;
  g.page_shift = a.cache.page_shift;
  g.keys_most = (int32_t)(a.table_width * a.cache.page_size);
  g.window = (int32_t)a.window;
  g.tiles = (int32_t)kv_tiles(a, rows_of(a));
  g.likely = (int32_t)likely_tiles(a, rows_of(a));
  g.parts = (int32_t)parts.places;
  g.fill = (int32_t)parts.fill;
  g.scale2 = a.scale * kLog2e;
  return g;
}

}  // namespace

size_t kv_attention_workspace(const KvAttention& a) {
  const size_t parts = (size_t)parts_of(a).places, rows = (size_t)a.tokens * (size_t)a.heads;
  return parts > 1 ? rows * (parts * (size_t)(a.cache.head_dim + 2) + 1) * 4 : 0;
}

bool kv_attention_grid_fits(const KvAttention& a) {
  return grid_fits(kv_tiles(a, rows_of(a)), a.cache.heads, 64 * WAVES);
}

hipError_t launch_kv_attention(const KvAttention& a, hipStream_t stream) {
  const Args g = kv_args(a, parts_of(a));
  if (a.cache.head_dim == 64) return launch_all<64>(a, g, stream);
  if (a.cache.head_dim == 128) return launch_all<128>(a, g, stream);
  return launch_all<256>(a, g, stream);
}

}  // namespace mx
