// Tensor-level entry points of the MXFP4, mixture-of-experts, key-value cache and
// rotary operators: the extension module _mx_torch.  Each function checks its tensors, allocates the
// outputs and makes one call of the C ABI on the current stream of the
// tensors' device.  It is C++ because the smallest calls take less time on the
// GPU than argument handling and allocations take in Python (one decoding step's
// combine: 9.3 us a call with Python and ctypes, 3.8 us from here, 3.0 of them
// the launch), and a backward node in C++ needs neither the interpreter nor its
// lock (routing with its gradient: 85 -> 48 us a step, of which 42 are PyTorch's
// engine's own).
#include <Python.h>

#include <array>
#include <unordered_set>
#include <vector>

#include <ATen/hip/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <c10/hip/HIPGraphsC10Utils.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/custom_function.h>
#include <torch/csrc/autograd/functions/accumulate_grad.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/graph_task.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kvcache.h"
#include "../../include/moe.h"
#include "../../include/mxfp4.h"
#include "../../include/rotary.h"

namespace {

using at::Tensor;
using torch::autograd::AutogradContext;
using torch::autograd::Variable;
using torch::autograd::variable_list;

// An argument error: a Python exception of this type.
struct ArgError {
  PyObject* type;
  std::string text;
};
// A status of the C ABI other than MXFP8_OK; the text is what the backward of
// a node shows, the entry points raise the package's MXFP8Error.
struct StatusError : std::runtime_error {
  StatusError(int s, const char* w)
      : std::runtime_error(std::string(w) + ": " + mxfp8_status_string((mxfp8_status)s)), status(s), where(w) {}
  int status;
  const char* where;
};

[[noreturn]] void refuse(std::string text, PyObject* type = PyExc_ValueError) { throw ArgError{type, std::move(text)}; }

void check(mxfp8_status s, const char* where) {
  if (s != MXFP8_OK) throw StatusError(s, where);
}

PyObject* raise_status(const StatusError& e) {
  static PyObject* type = nullptr;   // with the interpreter's lock held
  if (!type) {
    PyObject* m = PyImport_ImportModule("mxfp8_block_scaled_quantize_amd");
    if (!m) return nullptr;
    type = PyObject_GetAttrString(m, "MXFP8Error");
    Py_DECREF(m);
    if (!type) return nullptr;
  }
  PyObject* args = Py_BuildValue("(is)", e.status, e.where);
  if (args) {
    PyErr_SetObject(type, args);
    Py_DECREF(args);
  }
  return nullptr;
}

// Every entry point's body: C++ exceptions become Python's.
template <typename F>
PyObject* guarded(F body) {
  HANDLE_TH_ERRORS
  try {
    return body();
  } catch (const ArgError& e) {
    PyErr_SetString(e.type, e.text.c_str());
    return nullptr;
  } catch (const StatusError& e) {
    return raise_status(e);
  }
  END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ arguments
void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse("wrong number of arguments", PyExc_TypeError);
}
const Tensor* tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a torch tensor", PyExc_TypeError);
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a torch tensor", PyExc_TypeError);
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer", PyExc_TypeError);
  }
  return v;
}
int32_t small_integer(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " is out of range");
  return (int32_t)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();   // the object's own error is set
  return v == 1;
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); i++) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}
void on_gpu(const Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA (HIP) tensor, got " + t.device().str());
}
// A dense tensor of this type and shape on this device.
void need(const Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, c10::Device device) {
  on_gpu(t, name);
  if (t.scalar_type() != type) refuse(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  if (t.sizes() != shape) refuse(std::string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
  if (t.device() != device) refuse(std::string(name) + " is on " + t.device().str() + ", expected " + device.str());
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
}

// The operators have no forward-mode derivative: a dual tensor's tangent must not
// get lost (inside a custom function's forward it is the function's affair).
void no_tangent(const Tensor* t, const char* name) {
  if (t && c10::AutogradState::get_tls_state().get_fw_grad_mode() && t->_fw_grad(0).defined())
    refuse(std::string(name) + " carries a forward-mode tangent, which this operator does not propagate",
           PyExc_NotImplementedError);
}

// ------------------------------------------------------------------- the call
// From the caching allocator of the current stream, without a round through the
// dispatcher (0.4 us each).
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, c10::Device device) {
  return at::detail::empty_cuda(shape, type, device, std::nullopt);
}
// Several outputs of one call in one allocation, each from a multiple of 256
// bytes on: an allocation and its release take 0.35 us of a call's 4 to 5.
class Block {
 public:
  explicit Block(c10::Device device) : device_(device) {}
  size_t add(at::IntArrayRef shape, at::ScalarType type) {   // before make()
    const size_t at = bytes_;
    bytes_ += (c10::multiply_integers(shape) * c10::elementSize(type) + 255) / 256 * 256;
    return at;
  }
  void make() { storage_ = fresh({(int64_t)bytes_}, at::kByte, device_).storage(); }
  Tensor get(size_t at, at::IntArrayRef shape, at::ScalarType type) const {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(storage_), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                        c10::scalarTypeToTypeMeta(type));
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    t.unsafeGetTensorImpl()->set_storage_offset((int64_t)(at / c10::elementSize(type)));
    return t;
  }

 private:
  c10::Device device_;
  size_t bytes_ = 0;
  c10::Storage storage_;
};
void* stream_of(c10::Device d) { return c10::hip::getCurrentHIPStream(d.index()).stream(); }
// Stride between the rows of a matrix with unit column stride; of one row it
// says nothing.  Rows that overlap (expanded ones) are refused by the C ABI.
int64_t ld(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }
// Whether the columns of a matrix follow each other (of one column the stride
// says nothing).
bool unit_columns(const Tensor& t) { return t.size(1) <= 1 || t.stride(1) == 1; }
PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* pair(Tensor a, Tensor b) {
  PyObject* r = PyTuple_New(2);
  if (r) {
    PyTuple_SET_ITEM(r, 0, wrap(std::move(a)));
    PyTuple_SET_ITEM(r, 1, wrap(std::move(b)));
  }
  return r;
}

// ---------------------------------------------------------------------- MXFP4
void put(PyObject* dict, const char* key, const Tensor& t) {
  PyObject* o = wrap(t);
  if (!o || PyDict_SetItemString(dict, key, o)) {
    Py_XDECREF(o);
    throw python_error();
  }
  Py_DECREF(o);
}

// quantize(x, rowwise, colwise, packed, index)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 5);
    if (!THPVariable_Check(a[0])) refuse("x must be a BF16 [rows, cols] tensor with unit column stride");
    const Tensor& x = THPVariable_Unpack(a[0]);
    const bool row = truth(a[1]), col = truth(a[2]), packed = truth(a[3]);
    const Tensor* index = tensor_or_none(a[4], "index");
    if (x.scalar_type() != at::kBFloat16 || x.dim() != 2 || x.stride(1) != 1)
      refuse("x must be a BF16 [rows, cols] tensor with unit column stride");
    on_gpu(x, "x");
    const int64_t X = x.size(0), C = x.size(1);
    int64_t R = X;
    const c10::Device dev = x.device();
    if (index) {
      if (col) refuse("index goes with the rowwise copy alone");
      R = index->numel();
      need(*index, "index", at::kInt, {R}, dev);
    }
    c10::DeviceGuard guard(dev);
    at::AutoDispatchBelowADInplaceOrView below;
    Tensor q, s, qT, sT;
    // a copy's codes and scales in one allocation
    auto copy = [&](int64_t rows, int64_t cols, Tensor* codes, Tensor* scales) {
      const std::array<int64_t, 2> qs{rows, cols / 2}, ss = packed ? std::array<int64_t, 2>{cols / 128, rows} : std::array<int64_t, 2>{rows, cols / 32};
      const at::ScalarType type = packed ? at::kInt : at::kByte;
      Block both(dev);
      const size_t at_q = both.add(qs, at::kByte), at_s = both.add(ss, type);
      both.make();
      *codes = both.get(at_q, qs, at::kByte);
      *scales = both.get(at_s, ss, type);
    };
    if (row) copy(R, C, &q, &s);
    if (col) copy(C, R, &qT, &sT);
    const uint32_t flags = (row ? MXFP4_ROWWISE : 0) | (col ? MXFP4_COLWISE : 0) | (packed ? MXFP4_PACKED_SCALES : 0);
    check(mxfp4_quantize(x.data_ptr(), X, R, C, ld(x), index ? index->const_data_ptr<int32_t>() : nullptr, flags,
                         row ? q.data_ptr<uint8_t>() : nullptr, row ? s.data_ptr() : nullptr,
                         col ? qT.data_ptr<uint8_t>() : nullptr, col ? sT.data_ptr() : nullptr, stream_of(dev)),
          "mxfp4_quantize");
    PyObject* d = PyDict_New();
    if (!d) return nullptr;
    try {
      if (row) {
        put(d, "q_row", q);
        put(d, packed ? "p_row" : "s_row", s);
      }
      if (col) {
        put(d, "q_colT", qT);
        put(d, packed ? "p_colT" : "s_colT", sT);
      }
    } catch (...) {
      Py_DECREF(d);
      throw;
    }
    return d;
  });
}

// The BF16 [rows, cols] output of a call: `out`, or a fresh tensor.
Tensor output(const Tensor* out, int64_t rows, int64_t cols, c10::Device dev, const char* text) {
  if (!out) return fresh({rows, cols}, at::kBFloat16, dev);
  if (out->scalar_type() != at::kBFloat16 || out->sizes() != at::IntArrayRef{rows, cols} || out->stride(1) != 1 ||
      out->device() != dev)
    refuse(text);
  if (out->requires_grad() && at::GradMode::is_enabled())
    refuse("out requires a gradient, which this operator does not have: pass it with gradients disabled");
  no_tangent(out, "out");
  return *out;
}
// The kernel has written a caller's tensor behind autograd's back: what was saved
// of it for a backward pass is stale.
void written(const Tensor* out) {
  if (out && !out->is_inference()) torch::autograd::impl::bump_version(*out);
}

// dequantize(q, scales, out)
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 3);
    if (!THPVariable_Check(a[0]) || !THPVariable_Check(a[1]) || THPVariable_Unpack(a[0]).dim() != 2)
      refuse("q must be a 2-D tensor of MXFP4 codes, scales a tensor");
    const Tensor &q = THPVariable_Unpack(a[0]), &s = THPVariable_Unpack(a[1]);
    const Tensor* out = tensor_or_none(a[2], "out");
    const int64_t R = q.size(0), K = 2 * q.size(1);
    const c10::Device dev = q.device();
    need(q, "q", at::kByte, {R, K / 2}, dev);
    const bool packed = s.scalar_type() == at::kInt;
    if (packed) need(s, "scales", at::kInt, {K / 128, R}, dev);
    else need(s, "scales", at::kByte, {R, K / 32}, dev);
    c10::DeviceGuard guard(dev);
    at::AutoDispatchBelowADInplaceOrView below;
    Tensor o = output(out, R, K, dev, "out must be a BF16 [R, K] tensor with unit column stride on q's device");
    check(mxfp4_dequantize(q.const_data_ptr<uint8_t>(), s.const_data_ptr(), R, K, o.data_ptr(), ld(o),
                           packed ? MXFP4_PACKED_SCALES : 0, stream_of(dev)),
          "mxfp4_dequantize");
    written(out);
    return wrap(o);
  });
}

// gemm(a, a_packed, b, b_packed, out, accumulate, swiglu)
// grouped_gemm(a, a_packed, b, b_packed, offsets, out, accumulate, swiglu)
template <bool GROUPED>
PyObject* product(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, GROUPED ? 8 : 7);
    const char* shapes = GROUPED ? "a must be 2-D [M, K / 2] and b 3-D [G, N, K / 2] tensors of MXFP4 codes"
                                 : "a and b must be 2-D tensors of MXFP4 codes";
    if (!THPVariable_Check(v[0]) || !THPVariable_Check(v[2])) refuse(shapes);
    const Tensor &a = THPVariable_Unpack(v[0]), &b = THPVariable_Unpack(v[2]);
    const Tensor &ap = tensor(v[1], "a_packed"), &bp = tensor(v[3], "b_packed");
    const Tensor* offsets = GROUPED ? &tensor(v[4], "offsets") : nullptr;
    PyObject* const* opt = v + (GROUPED ? 5 : 4);
    const Tensor* out = tensor_or_none(opt[0], "out");
    const bool accumulate = truth(opt[1]), swiglu = truth(opt[2]);
    if (a.dim() != 2 || b.dim() != (GROUPED ? 3 : 2)) refuse(shapes);
    const int64_t M = a.size(0), K = 2 * a.size(1), G = GROUPED ? b.size(0) : 1, rows = b.size(GROUPED ? 1 : 0);
    if (swiglu && rows % 2)
      refuse(GROUPED ? "swiglu=True needs experts with an even number of rows (gate rows, then up rows)"
                     : "swiglu=True needs b with an even number of rows (gate rows, then up rows)");
    if (accumulate && swiglu) refuse("accumulate and swiglu exclude each other");
    if (accumulate && !out) refuse("accumulate=True needs out");
    const int64_t N = swiglu ? rows / 2 : rows;
    const c10::Device dev = a.device();
    need(a, "a", at::kByte, {M, K / 2}, dev);
    if (GROUPED) need(b, "b", at::kByte, {G, rows, K / 2}, dev);
    else need(b, "b", at::kByte, {rows, K / 2}, dev);
    need(ap, "a_packed", at::kInt, {K / 128, M}, dev);
    need(bp, "b_packed", at::kInt, {K / 128, G * rows}, dev);
    if (GROUPED) {
      if (G > INT32_MAX) refuse("too many groups");
      need(*offsets, "offsets", at::kInt, {G + 1}, dev);
    }
    c10::DeviceGuard guard(dev);
    at::AutoDispatchBelowADInplaceOrView below;
    Tensor c = output(out, M, N, dev, "out must be a BF16 [M, N] tensor with unit column stride on the operands' device");
    const uint32_t flags = accumulate ? MXFP4_GEMM_ACCUMULATE : swiglu ? MXFP4_GEMM_SWIGLU : 0;
    const uint8_t *pa = a.const_data_ptr<uint8_t>(), *pb = b.const_data_ptr<uint8_t>();
    const auto *sa = static_cast<const uint32_t*>(ap.const_data_ptr()), *sb = static_cast<const uint32_t*>(bp.const_data_ptr());
    if (GROUPED)
      check(mxfp4_grouped_gemm(pa, sa, pb, sb, offsets->const_data_ptr<int32_t>(), (int32_t)G, c.data_ptr(), ld(c), M, N, K,
                               flags, stream_of(dev)),
            "mxfp4_grouped_gemm");
    else
      check(mxfp4_gemm(pa, sa, pb, sb, c.data_ptr(), ld(c), M, N, K, flags, stream_of(dev)), "mxfp4_gemm");
    written(out);
    return wrap(c);
  });
}

// --------------------------------------------------------- mixture of experts
int32_t moe_dtype(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return MOE_FP32;
    case at::kBFloat16: return MOE_BF16;
    case at::kHalf: return MOE_FP16;
    default: return -1;
  }
}

// Outputs of a backward node: differentiating them again is an error.
variable_list once_only(variable_list grads) {
  if (!at::GradMode::is_enabled()) return grads;
  auto node = std::make_shared<torch::autograd::DelayedError>(
      "this operator is differentiable once", (int)grads.size());
  variable_list in;
  for (auto& g : grads) in.push_back(g.defined() ? g.detach().requires_grad_(true) : g);
  return (*node)(std::move(in));
}

struct RoutePlan {
  int32_t top_k, groups, top_groups, group_top;
  uint32_t flags;
};

std::pair<Tensor, Tensor> route_forward(const Tensor& logits, const Tensor* bias, const RoutePlan& p) {
  c10::DeviceGuard guard(logits.device());
  at::AutoDispatchBelowADInplaceOrView below;
  const int64_t T = logits.size(0), E = logits.size(1);
  Block both(logits.device());
  const std::array<int64_t, 2> shape{T, p.top_k};
  const size_t at_w = both.add(shape, at::kFloat), at_ids = both.add(shape, at::kInt);
  both.make();
  Tensor w = both.get(at_w, shape, at::kFloat), ids = both.get(at_ids, shape, at::kInt);
  check(moe_route(logits.const_data_ptr(), moe_dtype(logits), T, E, ld(logits), bias ? bias->const_data_ptr<float>() : nullptr,
                  p.top_k, p.groups, p.top_groups, p.group_top, p.flags, w.data_ptr<float>(), ids.data_ptr<int32_t>(),
                  stream_of(logits.device())),
        "moe_route");
  return {w, ids};
}

struct Route : torch::autograd::Function<Route> {
  static variable_list forward(AutogradContext* ctx, const Variable& logits, const std::optional<Tensor>& bias, int64_t top_k,
                               int64_t groups, int64_t top_groups, int64_t group_top, int64_t flags) {
    const RoutePlan p{(int32_t)top_k, (int32_t)groups, (int32_t)top_groups, (int32_t)group_top, (uint32_t)flags};
    auto [w, ids] = route_forward(logits, bias ? &*bias : nullptr, p);
    ctx->save_for_backward({logits, ids});
    ctx->saved_data["flags"] = flags;
    ctx->mark_non_differentiable({ids});
    ctx->set_materialize_grads(false);
    return {w, ids};
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    variable_list out(7);
    if (!grads[0].defined()) return out;
    const auto saved = ctx->get_saved_variables();
    const Tensor &logits = saved[0], &ids = saved[1];
    const int64_t T = logits.size(0), E = logits.size(1);
    c10::DeviceGuard guard(logits.device());
    {
      at::AutoDispatchBelowADInplaceOrView below;
      const Tensor dw = grads[0].to(at::kFloat).contiguous();
      Tensor d = fresh({T, E}, logits.scalar_type(), logits.device());
      check(moe_route_backward(logits.const_data_ptr(), moe_dtype(logits), T, E, ld(logits), ids.const_data_ptr<int32_t>(),
                               dw.const_data_ptr<float>(), (int32_t)ids.size(1), (uint32_t)ctx->saved_data["flags"].toInt(),
                               d.data_ptr(), stream_of(logits.device())),
            "moe_route_backward");
      out[0] = d;
    }
    return once_only(std::move(out));
  }
};

// route(logits, top_k, flags, bias, groups, top_groups, group_top)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 7);
    if (!THPVariable_Check(a[0]) || moe_dtype(THPVariable_Unpack(a[0])) < 0 || THPVariable_Unpack(a[0]).dim() != 2)
      refuse("logits must be a [tokens, experts] tensor of float32, bfloat16 or float16");
    const Tensor& logits = THPVariable_Unpack(a[0]);
    on_gpu(logits, "logits");
    if (!unit_columns(logits)) refuse("logits must have unit stride along the experts");
    const RoutePlan p{small_integer(a[1], "top_k"), small_integer(a[4], "groups"), small_integer(a[5], "top_groups"),
                      small_integer(a[6], "group_top"), (uint32_t)integer(a[2], "flags")};
    if (p.top_k < 1) refuse("top_k must be at least 1");
    const Tensor* bias = tensor_or_none(a[3], "bias");
    if (bias) need(*bias, "bias", at::kFloat, {logits.size(1)}, logits.device());
    no_tangent(&logits, "logits");
    no_tangent(bias, "bias");
    if (logits.requires_grad() && at::GradMode::is_enabled()) {
      auto r = Route::apply(logits, bias ? std::optional<Tensor>(*bias) : std::nullopt, p.top_k, p.groups, p.top_groups,
                            p.group_top, (int64_t)p.flags);
      return pair(r[0], r[1]);
    }
    auto [w, ids] = route_forward(logits, bias, p);
    return pair(w, ids);
  });
}

// dispatch(ids, experts)
PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 2);
    if (!THPVariable_Check(a[0]) || THPVariable_Unpack(a[0]).dim() != 2) refuse("ids must be an int32 [tokens, top_k] tensor");
    const Tensor& ids = THPVariable_Unpack(a[0]);
    const int64_t T = ids.size(0), K = ids.size(1), E = integer(a[1], "experts");
    const c10::Device dev = ids.device();
    need(ids, "ids", at::kInt, {T, K}, dev);
    if (E < 1 || E > MOE_MAX_EXPERTS) refuse("experts must be 1 .. " + std::to_string(MOE_MAX_EXPERTS));
    c10::DeviceGuard guard(dev);
    at::AutoDispatchBelowADInplaceOrView below;
    Block all(dev);
    const size_t at_o = all.add({E + 1}, at::kInt), at_t = all.add({T * K}, at::kInt), at_p = all.add({T, K}, at::kInt);
    all.make();
    Tensor offsets = all.get(at_o, {E + 1}, at::kInt), token = all.get(at_t, {T * K}, at::kInt),
           position = all.get(at_p, {T, K}, at::kInt);
    const size_t bytes = moe_dispatch_workspace_bytes(T, E, K);
    Tensor work;
    if (bytes) work = fresh({(int64_t)(bytes / 4)}, at::kInt, dev);
    check(moe_dispatch(ids.const_data_ptr<int32_t>(), T, E, K, offsets.data_ptr<int32_t>(), token.data_ptr<int32_t>(),
                       position.data_ptr<int32_t>(), bytes ? work.data_ptr() : nullptr, bytes, stream_of(dev)),
          "moe_dispatch");
    PyObject* r = PyTuple_New(3);
    if (r) {
      PyTuple_SET_ITEM(r, 0, wrap(offsets));
      PyTuple_SET_ITEM(r, 1, wrap(token));
      PyTuple_SET_ITEM(r, 2, wrap(position));
    }
    return r;
  });
}

Tensor combine_forward(const Tensor& y, const Tensor& position, const Tensor& w) {
  c10::DeviceGuard guard(y.device());
  at::AutoDispatchBelowADInplaceOrView below;
  const int64_t T = position.size(0), K = position.size(1), H = y.size(1);
  Tensor out = fresh({T, H}, y.scalar_type(), y.device());
  check(moe_combine(y.const_data_ptr(), moe_dtype(y), y.size(0), ld(y), position.const_data_ptr<int32_t>(),
                    w.const_data_ptr<float>(), T, K, H, out.data_ptr(), stream_of(y.device())),
        "moe_combine");
  return out;
}

struct Combine : torch::autograd::Function<Combine> {
  static Variable forward(AutogradContext* ctx, const Variable& y, const Variable& position, const Variable& w) {
    ctx->save_for_backward({y, position, w});
    return combine_forward(y, position, w);
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const auto saved = ctx->get_saved_variables();
    const Tensor &y = saved[0], &position = saved[1], &w = saved[2];
    const int64_t rows = y.size(0), T = position.size(0), K = position.size(1), H = y.size(1);
    const c10::Device dev = y.device();
    c10::DeviceGuard guard(dev);
    variable_list out(3);
    {
      at::AutoDispatchBelowADInplaceOrView below;
      Tensor d = grads[0];
      if (d.stride(1) != 1 || d.stride(0) < H) d = d.contiguous();   // expanded or transposed gradients
      Tensor dy, dw, work;
      if (ctx->needs_input_grad(0)) {
        dy = fresh({rows, H}, y.scalar_type(), dev);
        work = fresh({rows}, at::kInt, dev);
      }
      if (ctx->needs_input_grad(2)) dw = fresh({T, K}, at::kFloat, dev);
      check(moe_combine_backward(y.const_data_ptr(), moe_dtype(y), rows, ld(y), position.const_data_ptr<int32_t>(),
                                 w.const_data_ptr<float>(), T, K, H, d.const_data_ptr(), ld(d),
                                 dy.defined() ? dy.data_ptr() : nullptr, dw.defined() ? dw.data_ptr<float>() : nullptr,
                                 work.defined() ? work.data_ptr() : nullptr, work.defined() ? 4 * (size_t)rows : 0,
                                 stream_of(dev)),
            "moe_combine_backward");
      out[0] = dy;
      out[2] = dw;
    }
    return once_only(std::move(out));
  }
};

// combine(y, position, weights)
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 3);
    const char* text = "y must be a [rows, hidden] tensor of float32, bfloat16 or float16 with unit column stride";
    if (!THPVariable_Check(a[0])) refuse(text);
    const Tensor& y = THPVariable_Unpack(a[0]);
    if (moe_dtype(y) < 0 || y.dim() != 2 || !unit_columns(y)) refuse(text);
    on_gpu(y, "y");
    if (!THPVariable_Check(a[1]) || THPVariable_Unpack(a[1]).dim() != 2)
      refuse("position must be an int32 [tokens, top_k] tensor");
    const Tensor &position = THPVariable_Unpack(a[1]), &w = tensor(a[2], "weights");
    need(position, "position", at::kInt, position.sizes(), y.device());
    need(w, "weights", at::kFloat, position.sizes(), y.device());
    no_tangent(&y, "y");
    no_tangent(&w, "weights");
    if (at::GradMode::is_enabled() && (y.requires_grad() || w.requires_grad())) return wrap(Combine::apply(y, position, w));
    return wrap(combine_forward(y, position, w));
  });
}

// ------------------------------------------------------------ key-value cache
// The caller's cache: its sizes follow from its shape and the head size.
struct CacheShape {
  int64_t pages, kv_heads;
  int32_t page_size, head_dim;
};
CacheShape cache_shape(const Tensor& c, int64_t head_dim) {
  if (c.scalar_type() != at::kByte || c.dim() != 3) refuse("cache must be a uint8 [pages, kv_heads, bytes] tensor");
  need(c, "cache", at::kByte, c.sizes(), c.device());
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) refuse("head_dim must be 64, 128 or 256, got " + std::to_string(head_dim));
  const int64_t token = head_dim + head_dim / 16;
  const int64_t page = c.size(2) / token;
  if (c.size(2) % token || page < 16 || page > 256 || (page & (page - 1)))
    refuse("a cache of heads of " + std::to_string(head_dim) + " has 16, 32, 64, 128 or 256 times " + std::to_string(token) +
           " bytes to a page and head, got " + std::to_string(c.size(2)));
  if (c.size(0) < 1 || c.size(1) < 1) refuse("cache has no page or no head");
  if (c.size(1) > INT32_MAX) refuse("too many heads");
  return {c.size(0), c.size(1), (int32_t)page, (int32_t)head_dim};
}
// Whether the values of a head follow each other (of one value, or none, the stride says nothing).
bool unit_heads(const Tensor& t) { return t.size(2) <= 1 || t.numel() == 0 || t.stride(2) == 1; }
// A BF16 [tokens, heads, head_dim] tensor with unit stride along the head.
const Tensor& rows3(PyObject* o, const char* name) {
  const std::string text = std::string(name) + " must be a BF16 [tokens, heads, head_dim] tensor with unit stride along the head";
  if (!THPVariable_Check(o)) refuse(text, PyExc_TypeError);
  const Tensor& t = THPVariable_Unpack(o);
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || !unit_heads(t)) refuse(text);
  on_gpu(t, name);
  return t;
}
// Strides of a dimension of size 1 say nothing.
int64_t stride_of(const Tensor& t, int d) { return t.size(d) > 1 && t.numel() ? t.stride(d) : 0; }
void no_gradient(const Tensor& t, const char* name) {
  if (t.requires_grad() && at::GradMode::is_enabled())
    refuse(std::string(name) + " requires a gradient, which this operator does not have: call it with gradients disabled");
  no_tangent(&t, name);
}
// The caller's block table [rows, width].
const Tensor& block_table(PyObject* o, int64_t rows, c10::Device dev) {
  const Tensor& t = tensor(o, "table");
  if (t.dim() != 2) refuse("table must be an int32 [requests, pages] tensor");
  on_gpu(t, "table");
  if (t.scalar_type() != at::kInt || !(t.numel() == 0 || unit_columns(t))) refuse("table must be int32 with unit stride along a request's pages");
  if (t.size(0) != rows) refuse("table has " + std::to_string(t.size(0)) + " requests, lengths " + std::to_string(rows));
  if (t.device() != dev) refuse("table is on " + t.device().str() + ", expected " + dev.str());
  return t;
}
int64_t length_of(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name);
  if (t.dim() != 1) refuse(std::string(name) + " must have one dimension");
  return t.size(0);
}

// extend(table, lengths, counts, free, free_count, tokens, page_size)
PyObject* kv_extend_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 7);
    const int64_t B = length_of(a[1], "lengths"), pages = length_of(a[3], "free"), T = integer(a[5], "tokens");
    const Tensor &lengths = tensor(a[1], "lengths"), &counts = tensor(a[2], "counts"), &free = tensor(a[3], "free"),
                 &free_count = tensor(a[4], "free_count");
    const c10::Device dev = lengths.device();
    need(lengths, "lengths", at::kInt, {B}, dev);
    need(counts, "counts", at::kInt, {B}, dev);
    need(free, "free", at::kInt, {pages}, dev);
    need(free_count, "free_count", at::kInt, {1}, dev);
    const Tensor& table = block_table(a[0], B, dev);
    const int32_t page = small_integer(a[6], "page_size");
    if (T < 0 || T >= INT32_MAX) refuse("tokens is out of range");
    c10::DeviceGuard guard(dev);
    at::AutoDispatchBelowADInplaceOrView below;
    Block all(dev);
    const std::array<int64_t, 5> size{B + 1, B, T, T, 1};
    std::array<size_t, 5> at_;
    for (int i = 0; i < 5; i++) at_[i] = all.add({size[i]}, at::kInt);
    all.make();
    std::array<Tensor, 5> o;
    for (int i = 0; i < 5; i++) o[i] = all.get(at_[i], {size[i]}, at::kInt);
    check(kv_extend(table.data_ptr<int32_t>(), ld(table), table.size(1), lengths.const_data_ptr<int32_t>(),
                    counts.const_data_ptr<int32_t>(), B, free.const_data_ptr<int32_t>(), free_count.const_data_ptr<int32_t>(),
                    pages, page, T, o[0].data_ptr<int32_t>(), o[1].data_ptr<int32_t>(), o[2].data_ptr<int32_t>(),
                    o[3].data_ptr<int32_t>(), o[4].data_ptr<int32_t>(), stream_of(dev)),
          "kv_extend");
    written(&table);
    PyObject* r = PyTuple_New(5);
    if (r)
      for (int i = 0; i < 5; i++) PyTuple_SET_ITEM(r, i, wrap(o[i]));
    return r;
  });
}

// release(table, lengths, finished, free, free_count, page_size)
PyObject* kv_release_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 6);
    const int64_t B = length_of(a[1], "lengths"), pages = length_of(a[3], "free");
    const Tensor &lengths = tensor(a[1], "lengths"), &finished = tensor(a[2], "finished"), &free = tensor(a[3], "free"),
                 &free_count = tensor(a[4], "free_count");
    const c10::Device dev = lengths.device();
    need(lengths, "lengths", at::kInt, {B}, dev);
    need(finished, "finished", at::kBool, {B}, dev);
    need(free, "free", at::kInt, {pages}, dev);
    need(free_count, "free_count", at::kInt, {1}, dev);
    const Tensor& table = block_table(a[0], B, dev);
    const int32_t page = small_integer(a[5], "page_size");
    c10::DeviceGuard guard(dev);
    at::AutoDispatchBelowADInplaceOrView below;
    Block all(dev);
    const size_t at_l = all.add({B}, at::kInt), at_c = all.add({1}, at::kInt);
    all.make();
    Tensor l = all.get(at_l, {B}, at::kInt), c = all.get(at_c, {1}, at::kInt);
    check(kv_release(table.data_ptr<int32_t>(), ld(table), table.size(1), lengths.const_data_ptr<int32_t>(),
                     static_cast<const uint8_t*>(finished.const_data_ptr()), B, free.data_ptr<int32_t>(),
                     free_count.const_data_ptr<int32_t>(), pages, page, l.data_ptr<int32_t>(), c.data_ptr<int32_t>(),
                     stream_of(dev)),
          "kv_release");
    written(&table);
    written(&free);
    return pair(l, c);
  });
}

// append(cache, k, v, slots)
PyObject* kv_append_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 4);
    const Tensor &cache = tensor(a[0], "cache"), &k = rows3(a[1], "k"), &v = rows3(a[2], "v"), &slots = tensor(a[3], "slots");
    const CacheShape s = cache_shape(cache, k.size(2));
    const c10::Device dev = cache.device();
    const int64_t T = k.size(0);
    if (k.size(1) != s.kv_heads) refuse("k has " + std::to_string(k.size(1)) + " heads, the cache " + std::to_string(s.kv_heads));
    if (v.sizes() != k.sizes()) refuse("v must have k's shape " + shape_text(k.sizes()) + ", got " + shape_text(v.sizes()));
    for (const Tensor* t : {&k, &v})
      if (t->device() != dev) refuse("k and v are on " + t->device().str() + ", expected " + dev.str());
    need(slots, "slots", at::kInt, {T}, dev);
    no_gradient(k, "k");
    no_gradient(v, "v");
    c10::DeviceGuard guard(dev);
    at::AutoDispatchBelowADInplaceOrView below;
    check(kv_append(cache.data_ptr<uint8_t>(), s.pages, s.page_size, (int32_t)s.kv_heads, s.head_dim, k.const_data_ptr(),
                    stride_of(k, 0), stride_of(k, 1), v.const_data_ptr(), stride_of(v, 0), stride_of(v, 1),
                    slots.const_data_ptr<int32_t>(), T, stream_of(dev)),
          "kv_append");
    written(&cache);
    Py_RETURN_NONE;
  });
}

// read(cache, slots, head_dim)
PyObject* kv_read_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 3);
    const Tensor &cache = tensor(a[0], "cache"), &slots = tensor(a[1], "slots");
    const CacheShape s = cache_shape(cache, integer(a[2], "head_dim"));
    const c10::Device dev = cache.device();
    const int64_t T = length_of(a[1], "slots");
    need(slots, "slots", at::kInt, {T}, dev);
    c10::DeviceGuard guard(dev);
    at::AutoDispatchBelowADInplaceOrView below;
    const std::array<int64_t, 3> shape{T, s.kv_heads, s.head_dim};
    Block both(dev);
    const size_t at_k = both.add(shape, at::kBFloat16), at_v = both.add(shape, at::kBFloat16);
    both.make();
    Tensor k = both.get(at_k, shape, at::kBFloat16), v = both.get(at_v, shape, at::kBFloat16);
    check(kv_read(cache.const_data_ptr<uint8_t>(), s.pages, s.page_size, (int32_t)s.kv_heads, s.head_dim,
                  slots.const_data_ptr<int32_t>(), T, k.data_ptr(), v.data_ptr(), stream_of(dev)),
          "kv_read");
    return pair(k, v);
  });
}

// attention(q, cache, table, lengths, offsets, scale, window, max_queries, lse, out)
PyObject* kv_attention_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 10);
    const Tensor &q = rows3(a[0], "q"), &cache = tensor(a[1], "cache"), &lengths = tensor(a[3], "lengths");
    const CacheShape s = cache_shape(cache, q.size(2));
    const c10::Device dev = q.device();
    if (cache.device() != dev) refuse("cache is on " + cache.device().str() + ", expected " + dev.str());
    const int64_t T = q.size(0), H = q.size(1), B = length_of(a[3], "lengths");
    if (H < 1 || H % s.kv_heads || H > INT32_MAX)
      refuse("q has " + std::to_string(H) + " heads, the cache " + std::to_string(s.kv_heads) + ", which must divide them");
    need(lengths, "lengths", at::kInt, {B}, dev);
    const Tensor& table = block_table(a[2], B, dev);
    const Tensor* offsets = tensor_or_none(a[4], "offsets");
    if (offsets) need(*offsets, "offsets", at::kInt, {B + 1}, dev);
    else if (T != B) refuse("without offsets every sequence has one query: q has " + std::to_string(T) + ", lengths " + std::to_string(B));
    double scale = 1.0 / std::sqrt((double)s.head_dim);
    if (a[5] != Py_None) {
      scale = PyFloat_AsDouble(a[5]);
      if (scale == -1.0 && PyErr_Occurred()) throw python_error();
    }
    if (!((float)scale > 0.0f) || !std::isfinite((float)scale)) refuse("scale must be a positive finite number");
    const int64_t window = integer(a[6], "window");
    if (window < 0) refuse("window must not be negative (0: none)");
    int64_t most = T > 1 ? T : 1;
    if (a[7] != Py_None) {
      most = integer(a[7], "max_queries");
      if (most < 1) refuse("max_queries must be at least 1");
    }
    const bool with_lse = truth(a[8]);
    const Tensor* out = tensor_or_none(a[9], "out");
    no_gradient(q, "q");
    const std::array<int64_t, 3> shape{T, H, s.head_dim};
    if (out) {
      need(*out, "out", at::kBFloat16, shape, dev);
      no_gradient(*out, "out");
    }
    c10::DeviceGuard guard(dev);
    at::AutoDispatchBelowADInplaceOrView below;
    const size_t bytes = kv_attention_workspace_bytes(T, (int32_t)H, (int32_t)s.kv_heads, s.head_dim, B, table.size(1), s.page_size,
                                                      offsets != nullptr, most, window);
    Tensor work, o = out ? *out : fresh(shape, at::kBFloat16, dev), lse;
    if (bytes) work = fresh({(int64_t)bytes}, at::kByte, dev);
    if (with_lse) lse = fresh({T, H}, at::kFloat, dev);
    check(kv_attention(q.const_data_ptr(), stride_of(q, 0), stride_of(q, 1), T, (int32_t)H, cache.const_data_ptr<uint8_t>(), s.pages,
                       s.page_size, (int32_t)s.kv_heads, s.head_dim, table.const_data_ptr<int32_t>(), ld(table), table.size(1),
                       lengths.const_data_ptr<int32_t>(), offsets ? offsets->const_data_ptr<int32_t>() : nullptr, B, most,
                       (float)scale, window, o.data_ptr(), with_lse ? lse.data_ptr<float>() : nullptr,
                       bytes ? work.data_ptr() : nullptr, bytes, stream_of(dev)),
          "kv_attention");
    written(out);
    return with_lse ? pair(o, lse) : wrap(o);
  });
}

// --------------------------------------------------------------------- rotary
int32_t rotary_dtype(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return ROTARY_FP32;
    case at::kBFloat16: return ROTARY_BF16;
    case at::kHalf: return ROTARY_FP16;
    default: return -1;
  }
}
struct Turn {
  Tensor positions, turns;
  double magnitude;
  uint32_t flags;
};
// q and k (which may be undefined) turned: fresh tensors.
std::pair<Tensor, Tensor> rotate_both(const Tensor& q, const Tensor& k, const Turn& t) {
  const Tensor& some = q.defined() ? q : k;
  c10::DeviceGuard guard(some.device());
  at::AutoDispatchBelowADInplaceOrView below;
  Block both(some.device());
  const size_t at_q = q.defined() ? both.add(q.sizes(), q.scalar_type()) : 0;
  const size_t at_k = k.defined() ? both.add(k.sizes(), k.scalar_type()) : 0;
  both.make();
  Tensor qo, ko;
  if (q.defined()) qo = both.get(at_q, q.sizes(), q.scalar_type());
  if (k.defined()) ko = both.get(at_k, k.sizes(), k.scalar_type());
  check(rotary_rotate(q.defined() ? q.const_data_ptr() : nullptr, q.defined() ? stride_of(q, 0) : 0, q.defined() ? stride_of(q, 1) : 0,
                      q.defined() ? q.size(1) : 0, k.defined() ? k.const_data_ptr() : nullptr, k.defined() ? stride_of(k, 0) : 0,
                      k.defined() ? stride_of(k, 1) : 0, k.defined() ? k.size(1) : 0, rotary_dtype(some), some.size(0), some.size(2),
                      t.turns.numel(), t.positions.const_data_ptr<int32_t>(), t.turns.const_data_ptr<double>(), (float)t.magnitude,
                      t.flags, qo.defined() ? qo.data_ptr() : nullptr, ko.defined() ? ko.data_ptr() : nullptr,
                      stream_of(some.device())),
        "rotary_rotate");
  return {qo, ko};
}

// A leaf's accumulator keeps the stream on which it was made for as long as some graph
// holds it.  If that is not the stream of a backward pass that is being captured, the
// engine makes the two wait for each other once the pass is through, which a capture
// does not allow: the process ends.  So a pass that leads from this operator to such a
// leaf, directly or through other operators, is refused before.
void refuse_capture(c10::Device dev) {
  if (c10::hip::currentStreamCaptureStatusMayInitCtx() == c10::hip::CaptureStatus::None) return;
  using torch::autograd::Node;
  const auto here = torch::autograd::get_current_node();
  if (!here) return;
  const auto* const run = torch::autograd::get_current_graph_task_exec_info();   // empty: every node
  const c10::StreamId now = c10::hip::getCurrentHIPStream(dev.index()).id();
  std::unordered_set<const Node*> seen;
  std::vector<Node*> open{here.get()};
  while (!open.empty()) {
    Node* const n = open.back();
    open.pop_back();
    for (const auto& e : n->next_edges()) {
      Node* const next = e.function.get();
      if (!next || !seen.insert(next).second) continue;
      if (run && !run->empty()) {
        const auto info = run->find(next);
        if (info == run->end() || !info->second.should_execute()) continue;
      }
      open.push_back(next);
      if (!dynamic_cast<torch::autograd::AccumulateGrad*>(next)) continue;
      const auto stream = next->stream();
      if (stream && stream->device_index() == dev.index() && stream->id() != now)   // (a HIP stream's device has another type)
        throw std::runtime_error("rotate: its gradient cannot be captured while a graph of q or k, or of what they were made of, lives "
                                 "that was made on another stream: let go of that graph, or capture on its stream");
    }
  }
}

struct Rotate : torch::autograd::Function<Rotate> {
  static variable_list forward(AutogradContext* ctx, const Variable& q, const std::optional<Tensor>& k, const Tensor& positions,
                               const Tensor& turns, double magnitude, int64_t flags) {
    ctx->save_for_backward({positions, turns});
    ctx->saved_data["magnitude"] = magnitude;
    ctx->saved_data["flags"] = flags;
    ctx->set_materialize_grads(false);
    auto [qo, ko] = rotate_both(q, k ? *k : Tensor(), {positions, turns, magnitude, (uint32_t)flags});
    if (!k) return {qo};
    return {qo, ko};
  }
  static variable_list backward(AutogradContext* ctx, variable_list grads) {
    const auto saved = ctx->get_saved_variables();
    variable_list out(6);
    refuse_capture(saved[0].device());
    auto usable = [&](size_t i) {
      if (i >= grads.size() || !grads[i].defined() || !ctx->needs_input_grad(i)) return Tensor();
      at::AutoDispatchBelowADInplaceOrView below;
      return unit_heads(grads[i]) ? grads[i].detach() : grads[i].contiguous();
    };
    const Tensor dq = usable(0), dk = usable(1);
    if (dq.defined() || dk.defined()) {
      auto [q, k] = rotate_both(dq, dk, {saved[0], saved[1], ctx->saved_data["magnitude"].toDouble(),
                                         (uint32_t)(ctx->saved_data["flags"].toInt() ^ ROTARY_INVERSE)});
      out[0] = q;
      out[1] = k;
    }
    return once_only(std::move(out));
  }
};

// rotate(q, k, positions, turns, interleaved, magnitude)
PyObject* rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    count(n, 6);
    const char* text = "q must be a [tokens, heads, head_dim] tensor of float32, bfloat16 or float16 with unit stride along the head";
    if (!THPVariable_Check(a[0])) refuse(text, PyExc_TypeError);
    const Tensor& q = THPVariable_Unpack(a[0]);
    const Tensor* k = tensor_or_none(a[1], "k");
    if (rotary_dtype(q) < 0 || q.dim() != 3 || !unit_heads(q)) refuse(text);
    on_gpu(q, "q");
    const c10::Device dev = q.device();
    if (k) {
      if (k->scalar_type() != q.scalar_type() || k->dim() != 3 || k->size(0) != q.size(0) || k->size(2) != q.size(2) ||
          !unit_heads(*k))
        refuse("k must be [tokens, heads, head_dim] with q's type, tokens and head_dim and unit stride along the head");
      if (k->device() != dev) refuse("k is on " + k->device().str() + ", expected " + dev.str());
    }
    const Tensor &positions = tensor(a[2], "positions"), &turns = tensor(a[3], "turns");
    need(positions, "positions", at::kInt, {q.size(0)}, dev);
    need(turns, "turns", at::kDouble, {length_of(a[3], "turns")}, dev);
    if (2 * turns.numel() > q.size(2)) refuse("turns has more pairs than a head has dimensions");
    const bool interleaved = truth(a[4]);
    const double magnitude = PyFloat_AsDouble(a[5]);
    if (magnitude == -1.0 && PyErr_Occurred()) throw python_error();
    no_tangent(&q, "q");
    no_tangent(k, "k");
    no_gradient(turns, "turns");
    const int64_t flags = interleaved ? ROTARY_INTERLEAVED : 0;
    if (at::GradMode::is_enabled() && (q.requires_grad() || (k && k->requires_grad()))) {
      auto r = Rotate::apply(q, k ? std::optional<Tensor>(*k) : std::nullopt, positions, turns, magnitude, flags);
      return k ? pair(r[0], r[1]) : wrap(r[0]);
    }
    auto [qo, ko] = rotate_both(q, k ? *k : Tensor(), {positions, turns, magnitude, (uint32_t)flags});
    return k ? pair(qo, ko) : wrap(qo);
  });
}

#define MX_FN(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f))
PyMethodDef methods[] = {{"quantize", MX_FN(quantize), METH_FASTCALL, nullptr},
                         {"dequantize", MX_FN(dequantize), METH_FASTCALL, nullptr},
                         {"gemm", MX_FN(product<false>), METH_FASTCALL, nullptr},
                         {"grouped_gemm", MX_FN(product<true>), METH_FASTCALL, nullptr},
                         {"route", MX_FN(route), METH_FASTCALL, nullptr},
                         {"dispatch", MX_FN(dispatch), METH_FASTCALL, nullptr},
                         {"combine", MX_FN(combine), METH_FASTCALL, nullptr},
                         {"extend", MX_FN(kv_extend_), METH_FASTCALL, nullptr},
                         {"release", MX_FN(kv_release_), METH_FASTCALL, nullptr},
                         {"append", MX_FN(kv_append_), METH_FASTCALL, nullptr},
                         {"read", MX_FN(kv_read_), METH_FASTCALL, nullptr},
                         {"attention", MX_FN(kv_attention_), METH_FASTCALL, nullptr},
                         {"rotate", MX_FN(rotate), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mx_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mx_torch() { return PyModule_Create(&module); }
