// Block tables and slots of new tokens, and the pages given back.
//
// Both are prefix sums over the requests followed by lists (of rows, of pages)
// whose entries look up their request.  A workgroup makes all the sums itself,
// 1024 requests at a time, and its share of the lists: the requests' numbers are
// a few KB that every L2 holds, and no workgroup has to wait for another, so a
// step is one launch.  Sums saturate at 2^31 - 1 (saturating addition of numbers
// that are not negative is associative), which no valid size reaches.
//
// Bound by latency: one decoding step of 64 requests takes 4.6 us (two sums of 1024 numbers
// with their barriers, two binary searches, a store; an empty launch is 2), 509 requests with
// 592000 new tokens 8.6, of which 4.7 MB of lists are 1.  Pages are given back by one
// workgroup, 256 entries a round (a load, a search, a sum): 64 requests of 4 pages 3.0 us, of
// 512 pages 117.
#include "kv.h"
#include "launch.h"
#include "wave_scan.h"

namespace mx {

namespace {

constexpr int THREADS = 256, EACH = 4, CHUNK = THREADS * EACH;
constexpr int FULL = 0x7FFFFFFF;

__device__ __forceinline__ int sat_add(int a, int b) {
  const unsigned s = (unsigned)a + (unsigned)b;
  return s > (unsigned)FULL ? FULL : (int)s;
}

// Sum of the values of all threads before this one, `carry` first; the sum of
// all of them goes to *total.  `waves` is four ints of LDS.
__device__ __forceinline__ int sum_before(int v, int carry, int* waves, int* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int incl = scan64(v, [](int a, int b) { return sat_add(a, b); });
  const int up = __shfl_up(incl, 1, 64);
  if (lane == 63) waves[w] = incl;
  __syncthreads();
  int before = carry, all = carry;
#pragma unroll
  for (int i = 0; i < THREADS / 64; i++) {
    if (i < w) before = sat_add(before, waves[i]);
    all = sat_add(all, waves[i]);
  }
  __syncthreads();   // `waves` can be used again
  *total = all;
  return sat_add(before, lane ? up : 0);
}

// Last entry of an ascending list of CHUNK that is at most x (the first one is).
__device__ __forceinline__ int last_at_most(const int* list, int x) {
  int at = 0;
#pragma unroll
  for (int step = CHUNK / 2; step; step >>= 1)
    if (list[at + step] <= x) at += step;
  return at;
}

__device__ __forceinline__ int pages_of(int tokens, int shift) { return (int)(((unsigned)tokens + (1u << shift) - 1) >> shift); }

// A row is written by the workgroup blockIdx.x of its range [row0, row1), a new page
// by that of its range [page0, page1) of the order in which pages are taken.
__global__ __launch_bounds__(THREADS) void kv_extend_kernel(int32_t* __restrict__ table, int64_t ld, int64_t width,
                                                            const int32_t* __restrict__ lengths,
                                                            const int32_t* __restrict__ counts, int requests,
                                                            const int32_t* __restrict__ free,
                                                            const int32_t* __restrict__ free_count, int pages, int shift,
                                                            int tokens, int rows_each, int pages_each,
                                                            int32_t* __restrict__ offsets, int32_t* __restrict__ lengths_out,
                                                            int32_t* __restrict__ slots, int32_t* __restrict__ positions,
                                                            int32_t* __restrict__ free_count_out) {
  __shared__ int starts[CHUNK], befores[CHUNK], pasts[CHUNK];
  __shared__ int waves[4];
  const int tid = threadIdx.x;
  const int64_t row0 = (int64_t)blockIdx.x * rows_each, row1 = row0 + rows_each < tokens ? row0 + rows_each : tokens;
  const int64_t page0 = (int64_t)blockIdx.x * pages_each, page1 = page0 + pages_each;
  int count = free_count[0];
  count = count < 0 ? 0 : count > pages ? pages : count;
  int rows = 0, taken = 0, spent = 0;   // of the requests so far; spent: the pages that were really taken
  for (int b0 = 0, chunk = 0; b0 < requests; b0 += CHUNK, chunk++) {
    int past[EACH], fresh[EACH], mine = 0;
#pragma unroll
    for (int i = 0; i < EACH; i++) {
      const int b = b0 + tid * EACH + i;
      past[i] = b < requests ? lengths[b] : 0;
      fresh[i] = b < requests ? counts[b] : 0;
      past[i] = past[i] < 0 ? 0 : past[i];
      fresh[i] = fresh[i] < 0 ? 0 : fresh[i];
      mine = sat_add(mine, fresh[i]);
    }
    const int rows_before = rows, taken_before = taken;
    int start = sum_before(mine, rows, waves, &rows);
    int first[EACH], need[EACH], wanted = 0;
    bool fits[EACH];
#pragma unroll
    for (int i = 0; i < EACH; i++) {
      first[i] = start;
      start = sat_add(start, fresh[i]);
      const int total = sat_add(past[i], fresh[i]);
      fits[i] = start <= tokens && total < FULL && pages_of(total, shift) <= width;
      need[i] = fits[i] ? pages_of(total, shift) - pages_of(past[i], shift) : 0;
      wanted = sat_add(wanted, need[i]);
    }
    int before = sum_before(wanted, taken, waves, &taken);
    const bool owner = (int)(blockIdx.x) == chunk % (int)gridDim.x;
#pragma unroll
    for (int i = 0; i < EACH; i++) {
      const int at = tid * EACH + i, b = b0 + at;
      const int end = sat_add(before, need[i]);
      const bool granted = fits[i] && (need[i] == 0 || end <= count);
      if (granted && need[i]) spent = end > spent ? end : spent;
      starts[at] = first[i] < tokens ? first[i] : tokens;
      befores[at] = before;
      pasts[at] = granted ? past[i] : ~past[i];   // the sign: nothing for this one
      if (owner && b < requests) {
        offsets[b] = first[i] < tokens ? first[i] : tokens;
        lengths_out[b] = granted ? past[i] + fresh[i] : past[i];
      }
      before = end;
    }
    __syncthreads();
    const int64_t r0 = row0 > rows_before ? row0 : rows_before, r1 = row1 < rows ? row1 : rows;
    for (int64_t r = r0 + tid; r < r1; r += THREADS) {
      const int at = last_at_most(starts, (int)r);
      const int p = pasts[at];
      const int position = sat_add(p < 0 ? ~p : p, (int)r - starts[at]);
      int64_t slot = -1;
      if (p >= 0) {
        const int held = pages_of(p, shift), j = position >> shift;
        const int page = j < held ? table[(int64_t)(b0 + at) * ld + j] : free[count - 1 - (befores[at] + j - held)];
        if (page >= 0 && page < pages) slot = ((int64_t)page << shift) + (position & ((1 << shift) - 1));
      }
      slots[r] = (int32_t)slot;
      positions[r] = position;
    }
    const int64_t p0 = page0 > taken_before ? page0 : taken_before;
    int64_t p1 = page1 < taken ? page1 : taken;
    if (p1 > count) p1 = count;
    for (int64_t x = p0 + tid; x < p1; x += THREADS) {
      const int at = last_at_most(befores, (int)x);
      const int p = pasts[at];
      if (p >= 0) table[(int64_t)(b0 + at) * ld + pages_of(p, shift) + ((int)x - befores[at])] = free[count - 1 - x];
    }
    __syncthreads();
  }
  const int64_t r0 = row0 > rows ? row0 : rows;
  for (int64_t r = r0 + tid; r < row1; r += THREADS) {
    slots[r] = -1;
    positions[r] = 0;
  }
  if (blockIdx.x == 0) {
    spent = __builtin_amdgcn_readlane(scan64(spent, [](int a, int b) { return a > b ? a : b; }), 63);
    if ((tid & 63) == 0) waves[tid >> 6] = spent;
    __syncthreads();
    if (tid == 0) {
      for (int i = 1; i < THREADS / 64; i++) spent = waves[i] > spent ? waves[i] : spent;
      offsets[requests] = rows < tokens ? rows : tokens;
      free_count_out[0] = count - spent;
    }
  }
}

__global__ __launch_bounds__(THREADS) void kv_release_kernel(int32_t* __restrict__ table, int64_t ld, int64_t width,
                                                             const int32_t* __restrict__ lengths,
                                                             const uint8_t* __restrict__ finished, int requests,
                                                             int32_t* __restrict__ free,
                                                             const int32_t* __restrict__ free_count, int pages, int shift,
                                                             int32_t* __restrict__ lengths_out,
                                                             int32_t* __restrict__ free_count_out) {
  // One workgroup: how many of a request's entries are page numbers decides where
  // the next ones go, so the entries are looked at in order.
  __shared__ int befores[CHUNK];
  __shared__ int waves[4];
  const int tid = threadIdx.x;
  int count = free_count[0];
  count = count < 0 ? 0 : count > pages ? pages : count;
  for (int b0 = 0; b0 < requests; b0 += CHUNK) {
    int mine = 0, held[EACH];
#pragma unroll
    for (int i = 0; i < EACH; i++) {
      const int b = b0 + tid * EACH + i;
      int length = b < requests ? lengths[b] : 0;
      length = length < 0 ? 0 : length;
      const bool ends = b < requests && finished[b] != 0;
      const int n = pages_of(length, shift);
      held[i] = ends ? (n < width ? n : (int)width) : 0;
      mine = sat_add(mine, held[i]);
      if (b < requests) lengths_out[b] = ends ? 0 : length;
    }
    int entries;
    int before = sum_before(mine, 0, waves, &entries);
#pragma unroll
    for (int i = 0; i < EACH; i++) {
      befores[tid * EACH + i] = before;
      before = sat_add(before, held[i]);
    }
    __syncthreads();
    for (int64_t x0 = 0; x0 < entries; x0 += THREADS) {
      const int64_t x = x0 + tid;
      int page = -1;
      if (x < entries) {
        const int at = last_at_most(befores, (int)x);
        int32_t* entry = table + (int64_t)(b0 + at) * ld + ((int)x - befores[at]);
        page = *entry;
        *entry = -1;
      }
      const bool valid = page >= 0 && page < pages;
      int next;
      const int place = sum_before(valid ? 1 : 0, count, waves, &next);
      if (valid && place < pages) free[place] = page;
      count = next < pages ? next : pages;
    }
    __syncthreads();
  }
  if (tid == 0) free_count_out[0] = count;
}

}  // namespace

hipError_t launch_kv_extend(int32_t* table, int64_t ld, int64_t width, const int32_t* lengths, const int32_t* counts,
                            int64_t requests, const int32_t* free, const int32_t* free_count, int64_t pages, int page_shift,
                            int64_t tokens, int32_t* offsets, int32_t* lengths_out, int32_t* slots, int32_t* positions,
                            int32_t* free_count_out, hipStream_t stream) {
  // rows of a workgroup: 1024, more where that would be over 1024 workgroups
  int64_t blocks = (tokens + 1023) / 1024;
  blocks = blocks < 1 ? 1 : blocks > 1024 ? 1024 : blocks;
  const int64_t rows_each = (tokens + blocks - 1) / blocks;
  // a request takes at most one page more than its rows fill
  const int64_t most = (tokens >> page_shift) + requests;
  const int64_t pages_each = ((most < pages ? most : pages) + blocks - 1) / blocks;
  hipLaunchKernelGGL(kv_extend_kernel, dim3((unsigned)blocks), dim3(THREADS), 0, stream, table, ld, width, lengths, counts,
                     (int)requests, free, free_count, (int)pages, page_shift, (int)tokens, (int)rows_each, (int)pages_each,
                     offsets, lengths_out, slots, positions, free_count_out);
  return hipGetLastError();
}

hipError_t launch_kv_release(int32_t* table, int64_t ld, int64_t width, const int32_t* lengths, const uint8_t* finished,
                             int64_t requests, int32_t* free, const int32_t* free_count, int64_t pages, int page_shift,
                             int32_t* lengths_out, int32_t* free_count_out, hipStream_t stream) {
  hipLaunchKernelGGL(kv_release_kernel, dim3(1), dim3(THREADS), 0, stream, table, ld, width, lengths, finished, (int)requests,
                     free, free_count, (int)pages, page_shift, lengths_out, free_count_out);
  return hipGetLastError();
}

}  // namespace mx
