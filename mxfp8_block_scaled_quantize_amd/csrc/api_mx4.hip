// C ABI of the MXFP4 and mixture-of-experts operators: host-side validation,
// then one launch sequence on the caller's stream.  See include/mxfp4.h and
// include/moe.h for the contracts.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "../../include/mxfp4.h"
#include "launch.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 40;
constexpr int64_t kMaxK = int64_t(1) << 22;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

mxfp8_status hip_status(hipError_t e) {
  if (e == hipSuccess) return MXFP8_OK;
  mx::note_hip_error(e);
  return MXFP8_ERR_HIP;
}

// rows * cols with both below 2^40: whether the product stays below 2^40
bool product_ok(int64_t a, int64_t b) { return a <= kMaxDim && b <= kMaxDim && (a == 0 || b <= kMaxDim / a); }

mxfp8_status gemm4(const uint8_t* a, const uint32_t* ap, const uint8_t* b, const uint32_t* bp, const int32_t* offsets,
                   int32_t G, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K, uint32_t flags, void* stream) {
  if (flags != 0 && flags != MXFP4_GEMM_ACCUMULATE && flags != MXFP4_GEMM_SWIGLU) return MXFP8_ERR_FLAGS;
  if (M < 0 || N < 0 || K < 0 || N % 32 || K % 128 || ldc < N) return MXFP8_ERR_SHAPE;
  if (!product_ok(M, ldc) || !product_ok(N, K) || K > kMaxK || N > (int64_t(1) << 30) || M > 0x7FFFFFFF) return MXFP8_ERR_LIMIT;
  if (M == 0 || N == 0) return MXFP8_OK;
  if (!c || (K > 0 && (!a || !ap || !b || !bp)) || (G > 0 && !offsets)) return MXFP8_ERR_NULL;
  if (!aligned(c, 16) || ldc % 8 || (G > 0 && !aligned(offsets, 4))) return MXFP8_ERR_MISALIGNED;
  if (K > 0 && (!aligned(a, 16) || !aligned(b, 16) || !aligned(ap, 4) || !aligned(bp, 4))) return MXFP8_ERR_MISALIGNED;
  mx::Mx4Gemm g{a, ap, b, bp, static_cast<uint16_t*>(c), ldc, M, N, K, G > 0 ? offsets : nullptr, G,
                flags == MXFP4_GEMM_ACCUMULATE ? 1 : flags == MXFP4_GEMM_SWIGLU ? 2 : 0};
  if (!mx::mx4_gemm_grid_fits(g)) return MXFP8_ERR_LIMIT;
  return hip_status(mx::launch_mx4_gemm(g, static_cast<hipStream_t>(stream)));
}

int element_size(int32_t dtype) { return dtype == MOE_FP32 ? 4 : 2; }
bool dtype_ok(int32_t dtype) { return dtype == MOE_FP32 || dtype == MOE_BF16 || dtype == MOE_FP16; }

mxfp8_status check_route(const void* logits, int32_t dtype, int64_t tokens, int64_t experts, int64_t ld, int32_t top_k,
                         uint32_t flags) {
  if (!dtype_ok(dtype) || (flags & ~(MOE_ROUTE_SIGMOID | MOE_ROUTE_RENORMALIZE))) return MXFP8_ERR_FLAGS;
  if (tokens < 0 || experts < 1 || experts > MOE_MAX_EXPERTS || ld < experts) return MXFP8_ERR_SHAPE;
  if (top_k < 1 || top_k > experts || top_k > MOE_MAX_TOP_K) return MXFP8_ERR_SHAPE;
  if (!product_ok(tokens, ld) || !mx::moe_route_grid_fits(tokens)) return MXFP8_ERR_LIMIT;
  if (tokens > 0 && !logits) return MXFP8_ERR_NULL;
  if (tokens > 0 && !aligned(logits, element_size(dtype))) return MXFP8_ERR_MISALIGNED;
  return MXFP8_OK;
}

mxfp8_status check_combine(const void* y, int32_t dtype, int64_t rows, int64_t ld_y, const int32_t* position,
                           const float* weights, int64_t tokens, int64_t top_k, int64_t hidden) {
  if (!dtype_ok(dtype)) return MXFP8_ERR_FLAGS;
  if (rows < 0 || tokens < 0 || hidden < 0 || top_k < 1 || ld_y < hidden) return MXFP8_ERR_SHAPE;
  if (!product_ok(rows, ld_y) || !product_ok(tokens, hidden) || top_k > (int64_t(1) << 20) || !product_ok(tokens, top_k) ||
      rows > 0x7FFFFFFF)
    return MXFP8_ERR_LIMIT;
  if (tokens > 0 && hidden > 0) {
    if ((rows > 0 && !y) || !position || !weights) return MXFP8_ERR_NULL;
    if (!aligned(y, element_size(dtype)) || !aligned(position, 4) || !aligned(weights, 4)) return MXFP8_ERR_MISALIGNED;
  }
  return MXFP8_OK;
}

}  // namespace

extern "C" {

mxfp8_status mxfp4_quantize(const void* x, int64_t x_rows, int64_t rows, int64_t cols, int64_t ld_x, const int32_t* index,
                            uint32_t flags, uint8_t* q_row, void* s_row, uint8_t* q_colT, void* s_colT, void* stream) {
  const bool row = flags & MXFP4_ROWWISE, col = flags & MXFP4_COLWISE, packed = flags & MXFP4_PACKED_SCALES;
  if ((flags & ~(MXFP4_ROWWISE | MXFP4_COLWISE | MXFP4_PACKED_SCALES)) || !(row || col)) return MXFP8_ERR_FLAGS;
  if (index && col) return MXFP8_ERR_FLAGS;
  if (rows < 0 || cols < 0 || x_rows < 0 || ld_x < cols || cols % 32 || (col && rows % 32)) return MXFP8_ERR_SHAPE;
  if (packed && ((row && cols % 128) || (col && rows % 128))) return MXFP8_ERR_SHAPE;
  if (!index && x_rows != rows) return MXFP8_ERR_SHAPE;
  if (!product_ok(x_rows, ld_x) || !product_ok(rows, cols) || !mx::mx4_quantize_grid_fits(rows, cols)) return MXFP8_ERR_LIMIT;
  if (rows == 0 || cols == 0) return MXFP8_OK;
  if ((x_rows > 0 && !x) || (row && (!q_row || !s_row)) || (col && (!q_colT || !s_colT))) return MXFP8_ERR_NULL;
  if (!aligned(x, 16) || ld_x % 8 || (row && !aligned(q_row, 16)) || (col && !aligned(q_colT, 16)) || (index && !aligned(index, 4)))
    return MXFP8_ERR_MISALIGNED;
  if (packed && ((row && !aligned(s_row, 4)) || (col && !aligned(s_colT, 4)))) return MXFP8_ERR_MISALIGNED;
  return hip_status(mx::launch_mx4_quantize(static_cast<const uint16_t*>(x), x_rows, rows, cols, ld_x, index, row, col, packed,
                                            q_row, s_row, q_colT, s_colT, static_cast<hipStream_t>(stream)));
}

mxfp8_status mxfp4_dequantize(const uint8_t* q, const void* s, int64_t rows, int64_t cols, void* out, int64_t ld_out,
                              uint32_t flags, void* stream) {
  const bool packed = flags & MXFP4_PACKED_SCALES;
  if (flags & ~MXFP4_PACKED_SCALES) return MXFP8_ERR_FLAGS;
  if (rows < 0 || cols < 0 || cols % (packed ? 128 : 32) || ld_out < cols) return MXFP8_ERR_SHAPE;
  if (!product_ok(rows, ld_out) || !mx::mx4_quantize_grid_fits(rows, cols)) return MXFP8_ERR_LIMIT;
  if (rows == 0 || cols == 0) return MXFP8_OK;
  if (!q || !s || !out) return MXFP8_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || ld_out % 8 || (packed && !aligned(s, 4))) return MXFP8_ERR_MISALIGNED;
  return hip_status(mx::launch_mx4_dequantize(q, s, rows, cols, packed, static_cast<uint16_t*>(out), ld_out,
                                              static_cast<hipStream_t>(stream)));
}

mxfp8_status mxfp4_gemm(const uint8_t* a, const uint32_t* a_packed, const uint8_t* b, const uint32_t* b_packed, void* c,
                        int64_t ldc, int64_t M, int64_t N, int64_t K, uint32_t flags, void* stream) {
  return gemm4(a, a_packed, b, b_packed, nullptr, 0, c, ldc, M, N, K, flags, stream);
}

mxfp8_status mxfp4_grouped_gemm(const uint8_t* a, const uint32_t* a_packed, const uint8_t* b, const uint32_t* b_packed,
                                const int32_t* offsets, int32_t G, void* c, int64_t ldc, int64_t M_total, int64_t N, int64_t K,
                                uint32_t flags, void* stream) {
  if (G < 1 || G > 65535) return MXFP8_ERR_SHAPE;
  return gemm4(a, a_packed, b, b_packed, offsets, G, c, ldc, M_total, N, K, flags, stream);
}

mxfp8_status moe_route(const void* logits, int32_t dtype, int64_t tokens, int64_t experts, int64_t ld, const float* bias,
                       int32_t top_k, int32_t groups, int32_t top_groups, int32_t group_top, uint32_t flags, float* weights,
                       int32_t* ids, void* stream) {
  const mxfp8_status st = check_route(logits, dtype, tokens, experts, ld, top_k, flags);
  if (st != MXFP8_OK) return st;
  if (groups < 1 || groups > 64 || groups > experts || experts % groups || top_groups < 1 || top_groups > groups)
    return MXFP8_ERR_SHAPE;
  if (top_k > top_groups * (experts / groups) || (groups > 1 && group_top != 1 && group_top != 2)) return MXFP8_ERR_SHAPE;
  if (tokens == 0) return MXFP8_OK;
  if (!weights || !ids) return MXFP8_ERR_NULL;
  if (!aligned(weights, 4) || !aligned(ids, 4) || !aligned(bias, 4)) return MXFP8_ERR_MISALIGNED;
  return hip_status(mx::launch_moe_route(logits, dtype, tokens, experts, ld, bias, top_k, groups, top_groups, group_top,
                                         flags & MOE_ROUTE_SIGMOID, flags & MOE_ROUTE_RENORMALIZE, weights, ids,
                                         static_cast<hipStream_t>(stream)));
}

mxfp8_status moe_route_backward(const void* logits, int32_t dtype, int64_t tokens, int64_t experts, int64_t ld,
                                const int32_t* ids, const float* dweights, int32_t top_k, uint32_t flags, void* dlogits,
                                void* stream) {
  const mxfp8_status st = check_route(logits, dtype, tokens, experts, ld, top_k, flags);
  if (st != MXFP8_OK) return st;
  if (tokens == 0) return MXFP8_OK;
  if (!ids || !dweights || !dlogits) return MXFP8_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(dweights, 4) || !aligned(dlogits, element_size(dtype))) return MXFP8_ERR_MISALIGNED;
  return hip_status(mx::launch_moe_route_backward(logits, dtype, tokens, experts, ld, ids, dweights, top_k,
                                                  flags & MOE_ROUTE_SIGMOID, flags & MOE_ROUTE_RENORMALIZE, dlogits,
                                                  static_cast<hipStream_t>(stream)));
}

size_t moe_dispatch_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k) {
  if (tokens <= 0 || experts < 1 || experts > MOE_MAX_EXPERTS || top_k < 1 || tokens > 0x7FFFFFFF / top_k) return 0;
  return mx::moe_dispatch_workspace(tokens * top_k, experts);
}

mxfp8_status moe_dispatch(const int32_t* ids, int64_t tokens, int64_t experts, int64_t top_k, int32_t* offsets, int32_t* token,
                          int32_t* position, void* workspace, size_t workspace_bytes, void* stream) {
  if (tokens < 0 || experts < 1 || experts > MOE_MAX_EXPERTS || top_k < 1) return MXFP8_ERR_SHAPE;
  if (top_k > 0x7FFFFFFF || tokens > 0x7FFFFFFF / top_k) return MXFP8_ERR_LIMIT;
  if (!offsets || (tokens > 0 && (!ids || !token || !position))) return MXFP8_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(token, 4) || !aligned(position, 4)) return MXFP8_ERR_MISALIGNED;
  const size_t need = moe_dispatch_workspace_bytes(tokens, experts, top_k);
  if (need && (!workspace || workspace_bytes < need)) return MXFP8_ERR_WORKSPACE;
  if (need && !aligned(workspace, 4)) return MXFP8_ERR_MISALIGNED;
  return hip_status(mx::launch_moe_dispatch(ids, tokens * top_k, experts, (int32_t)top_k, offsets, token, position,
                                            static_cast<int32_t*>(workspace), static_cast<hipStream_t>(stream)));
}

mxfp8_status moe_combine(const void* y, int32_t dtype, int64_t rows, int64_t ld_y, const int32_t* position,
                         const float* weights, int64_t tokens, int64_t top_k, int64_t hidden, void* out, void* stream) {
  const mxfp8_status st = check_combine(y, dtype, rows, ld_y, position, weights, tokens, top_k, hidden);
  if (st != MXFP8_OK) return st;
  if (tokens == 0 || hidden == 0) return MXFP8_OK;
  if (!out) return MXFP8_ERR_NULL;
  if (!aligned(out, element_size(dtype))) return MXFP8_ERR_MISALIGNED;
  if (!mx::moe_combine_grid_fits(y, dtype, ld_y, tokens, hidden, out)) return MXFP8_ERR_LIMIT;
  return hip_status(mx::launch_moe_combine(y, dtype, rows, ld_y, position, weights, tokens, (int)top_k, hidden, out,
                                           static_cast<hipStream_t>(stream)));
}

mxfp8_status moe_combine_backward(const void* y, int32_t dtype, int64_t rows, int64_t ld_y, const int32_t* position,
                                  const float* weights, int64_t tokens, int64_t top_k, int64_t hidden, const void* dout,
                                  int64_t ld_dout, void* dy, float* dweights, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  const mxfp8_status st = check_combine(y, dtype, rows, ld_y, position, weights, tokens, top_k, hidden);
  if (st != MXFP8_OK) return st;
  if (ld_dout < hidden) return MXFP8_ERR_SHAPE;
  if (!product_ok(tokens, ld_dout) || !mx::moe_combine_backward_grid_fits(tokens, top_k, rows)) return MXFP8_ERR_LIMIT;
  if (!dy && !dweights) return MXFP8_OK;
  // nothing to read: the weights' gradients are zeros, which a hidden size of 0 alone gives
  if (tokens > 0 && (!dout && hidden > 0)) return MXFP8_ERR_NULL;
  if (tokens > 0 && (!position || !weights)) return MXFP8_ERR_NULL;
  if (!aligned(dout, element_size(dtype)) || !aligned(dy, element_size(dtype)) || !aligned(dweights, 4))
    return MXFP8_ERR_MISALIGNED;
  if (dy && rows > 0) {
    if (!workspace || workspace_bytes < (size_t)rows * 4u) return MXFP8_ERR_WORKSPACE;
    if (!aligned(workspace, 4)) return MXFP8_ERR_MISALIGNED;
  }
  return hip_status(mx::launch_moe_combine_backward(y, dtype, rows, ld_y, position, weights, tokens, (int)top_k, hidden, dout,
                                                    ld_dout, rows > 0 ? dy : nullptr, dweights,
                                                    static_cast<int32_t*>(workspace), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
