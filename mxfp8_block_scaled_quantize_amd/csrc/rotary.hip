// Rotary positions: the pairs of a head's first 2 F dimensions turned by angles
// that grow with the position.
//
// A thread takes one token's V neighbouring pairs (or V pairs of dimensions that
// stay), makes their sines and cosines once and turns those of several heads of q
// and k.  Its loads and stores are two runs of 16 bytes, and neighbouring threads' runs
// stand next to each other: in the two halves of the turned dimensions, interleaved or
// not (40 heads of 128, fp32, 4096 tokens, interleaved: 32.0 us, with the second run
// behind the first 40.6), and of those that stay.  The angle in turns is position *
// turns[f], reduced to [-1/2, 1/2] in 64 bits (the product is exact to 2^-53 of itself:
// 4e-8 turns for a position of 2^31 at 1/(2 pi) turns each), so that far positions cost
// no accuracy; the rest is fp32.
//
// Bound by HBM: every element is read and written once, 168 MB (8192 tokens, 40 heads of
// 128, BF16) in 32 to 36 us, 4.7 to 5.2 TB/s, a large copy's rate.  Few tokens: latency, 4 us.
#include "kv.h"
#include "launch.h"
#include "mx_device.h"

namespace mx {

namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }
template <>
__device__ __forceinline__ float to_f32(__bf16 v) { return (float)v; }

template <typename T, int V>
struct alignas(sizeof(T) * V) Run {
  T v[V];
};

struct Rotary {
  RotaryRows q, k;
  int64_t tokens;
  int32_t head_dim, pairs, heads, heads_each, parts, turning;   // parts of a token: `turning` of them turn
  int32_t width;   // elements of a run: 16 bytes, or one
  const int32_t* positions;
  const double* turns;
  float magnitude;
};

template <typename T, int V, bool INTERLEAVED, bool INVERSE>
__global__ __launch_bounds__(256) void rotary_kernel(Rotary r) {
  const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const uint32_t part = (uint32_t)(x % r.parts);
  const int64_t y = x / r.parts;
  const int groups = (r.heads + r.heads_each - 1) / r.heads_each;
  const int64_t token = y / groups;
  if (token >= r.tokens) return;
  const int h0 = (int)(y % groups) * r.heads_each, h1 = h0 + r.heads_each < r.heads ? h0 + r.heads_each : r.heads;
  const bool turn = part < (uint32_t)r.turning;
  // the two runs of V dimensions that this thread takes, neighbouring threads' ones next to
  // each other (of those that stay: the second may be behind the end)
  constexpr bool EACH = INTERLEAVED && V > 1;   // either run is V / 2 pairs
  const int other = r.parts - r.turning;
  int64_t a, b;
  float c[V], s[V];
  if (turn) {
    a = INTERLEAVED && !EACH ? 2 * (int)part : (int)part * V;
    b = EACH ? a + r.pairs : INTERLEAVED ? a + 1 : a + r.pairs;
    const double position = (double)r.positions[token];
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int f = EACH ? (int)(i < V / 2 ? a : b) / 2 + i % (V > 1 ? V / 2 : 1) : (int)part * V + i;
      const double t = position * r.turns[f];
      float sn, cs;
      sincospif(2.0f * (float)(t - rint(t)), &sn, &cs);
      c[i] = cs * r.magnitude;
      s[i] = INVERSE ? -(sn * r.magnitude) : sn * r.magnitude;
    }
  } else {
    a = 2 * (int64_t)r.pairs + (int64_t)(part - r.turning) * V;
    b = a + (int64_t)other * V;
  }
  const bool second = b < r.head_dim;
  for (int h = h0; h < h1; h++) {
    const bool is_q = h < r.q.heads;
    const RotaryRows& rows = is_q ? r.q : r.k;
    const int64_t head = is_q ? h : h - r.q.heads;
    const T* in = static_cast<const T*>(rows.in) + token * rows.token + head * rows.head;
    T* out = static_cast<T*>(rows.out) + (token * rows.heads + head) * r.head_dim;
    Run<T, V> u = *reinterpret_cast<const Run<T, V>*>(in + a), w = u;
    if (second) w = *reinterpret_cast<const Run<T, V>*>(in + b);
    if (turn) {
      if constexpr (EACH) {
#pragma unroll
        for (int i = 0; i < V; i++) {
          Run<T, V>& x = i < V / 2 ? u : w;
          const int j = 2 * i % V;
          const float p = to_f32(x.v[j]), q = to_f32(x.v[j + 1]);
          x.v[j] = (T)(p * c[i] - q * s[i]);
          x.v[j + 1] = (T)(p * s[i] + q * c[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; i++) {
          const float p = to_f32(u.v[i]), q = to_f32(w.v[i]);
          u.v[i] = (T)(p * c[i] - q * s[i]);
          w.v[i] = (T)(p * s[i] + q * c[i]);
        }
      }
    }
    *reinterpret_cast<Run<T, V>*>(out + a) = u;
    if (second) *reinterpret_cast<Run<T, V>*>(out + b) = w;
  }
}

// Runs of v elements start on multiples of v everywhere: 16-byte accesses.
bool wide(const RotaryRows& x, int64_t v) {
  return x.heads == 0 || ((reinterpret_cast<uintptr_t>(x.in) | reinterpret_cast<uintptr_t>(x.out)) % 16 == 0 && x.token % v == 0 &&
                          x.head % v == 0);
}

int64_t groups_of(const Rotary& r) { return (r.heads + r.heads_each - 1) / r.heads_each; }

// How a call is cut into threads.
Rotary plan_of(const RotaryCall& c) {
  Rotary r{c.q, c.k, c.tokens, (int32_t)c.head_dim, (int32_t)c.pairs, (int32_t)(c.q.heads + c.k.heads), 8, 0, 0, 1, c.positions, c.turns, c.magnitude};
  const int32_t v = c.dtype == 0 ? 4 : 8;
  if (c.pairs % v == 0 && c.head_dim % v == 0 && wide(c.q, v) && wide(c.k, v)) r.width = v;
  r.turning = r.pairs / r.width;
  const int64_t rest = r.head_dim - 2 * (int64_t)r.pairs;
  r.parts = (int)(r.turning + (rest + 2 * r.width - 1) / (2 * r.width));
  // heads of a thread: up to 8, fewer where that would leave less than 8 waves a compute unit
  // (2^17 tokens and more never do)
  const int64_t tokens = r.tokens < (1 << 17) ? r.tokens : 1 << 17;
  while (r.heads_each > 1 && tokens * r.parts * groups_of(r) < 256 * 8 * 64) r.heads_each >>= 1;
  return r;
}

template <typename T, int V>
hipError_t launch(const Rotary& r, bool interleaved, bool inverse, hipStream_t stream) {
  const dim3 grid((unsigned)((r.tokens * r.parts * groups_of(r) + 255) / 256));
#define MX_ROT(IL, INV) hipLaunchKernelGGL((rotary_kernel<T, V, IL, INV>), grid, dim3(256), 0, stream, r)
  if (interleaved) { if (inverse) MX_ROT(true, true); else MX_ROT(true, false); }
  else { if (inverse) MX_ROT(false, true); else MX_ROT(false, false); }
#undef MX_ROT
  return hipGetLastError();
}

template <typename T>
hipError_t launch_type(const Rotary& r, bool interleaved, bool inverse, hipStream_t stream) {
  return r.width > 1 ? launch<T, 16 / sizeof(T)>(r, interleaved, inverse, stream) : launch<T, 1>(r, interleaved, inverse, stream);
}

}  // namespace

bool rotary_grid_fits(const RotaryCall& c) {
  const Rotary r = plan_of(c);
  return grid_fits(c.tokens, (int64_t)r.parts * groups_of(r), 1) && c.tokens * r.parts * groups_of(r) <= kMaxWorkItems - 255;
}

hipError_t launch_rotary(const RotaryCall& c, hipStream_t stream) {
  const Rotary r = plan_of(c);
  if (c.dtype == 0) return launch_type<float>(r, c.interleaved, c.inverse, stream);
  if (c.dtype == 1) return launch_type<__bf16>(r, c.interleaved, c.inverse, stream);
  return launch_type<_Float16>(r, c.interleaved, c.inverse, stream);
}

}  // namespace mx
