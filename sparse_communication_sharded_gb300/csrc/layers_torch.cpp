// layers_torch.cpp -- the training-layer operators for torch tensors: checks of
// types, shapes and layouts, outputs and workspaces from torch's allocator, the
// current stream, and one call of the C ABI (include/scape_layers.h) each.
//
// Native because a call's host side is longer than the kernels of a small
// layer: the same checks and marshalling through ctypes took 17 to 20 us a call
// on the GPU host's Arm cores, against 4 us for a one-token norm kernel.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>
#include <vector>

#include "scape_layers.h"

namespace {

using at::Tensor;

struct ValueError : std::exception {
  std::string what_;
  explicit ValueError(std::string s) : what_(std::move(s)) {}
  const char* what() const noexcept override { return what_.c_str(); }
};
struct LibraryError : std::exception {
  int code;
  explicit LibraryError(int c) : code(c) {}
};

void library(int rc) {
  if (rc != SCAPE_OK) throw LibraryError(rc);
}

constexpr int64_t kBlock = SCAPE_PACK_BLOCK;
enum Types { kBf16 = 1, kF32 = 2, kE4m3 = 4 };

int type_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return kBf16;
    case at::kFloat: return kF32;
    case at::kFloat8_e4m3fn: return kE4m3;
    default: return 0;
  }
}
int dtype_of(const Tensor& t) { return t.scalar_type() == at::kBFloat16 ? SCAPE_BF16 : SCAPE_F32; }

std::string names(int types) {
  std::string s;
  if (types & kBf16) s += " bfloat16";
  if (types & kF32) s += " float32";
  if (types & kE4m3) s += " float8_e4m3fn";
  return s;
}

// A tensor argument.  These operators record nothing for autograd: where it would
// look for a graph, a result without one would train less than the caller thinks.
const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw ValueError(std::string(name) + " must be a tensor");
  const Tensor& t = THPVariable_Unpack(o);
  if (t.requires_grad() && at::GradMode::is_enabled())
    throw ValueError(std::string(name) +
                     " requires grad, and layer operators are not recorded by autograd: call them "
                     "under torch.no_grad() (or in an autograd.Function), or detach it");
  return t;
}
// A tensor that the call has written in place, for autograd's check that saved
// values are as they were.
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// A tensor seen as the rows of its last dimension.
struct Rows {
  void* p;
  int64_t rows, cols, ld;
};

void same_shape(const Tensor& t, at::IntArrayRef lead, int64_t cols, const char* name) {
  const auto s = t.sizes();
  if (s.size() != lead.size() + 1 || s.back() != cols || s.slice(0, lead.size()) != lead)
    throw ValueError(std::string(name) + " has another shape than the call's other tensors say");
}

Rows rows_of(const Tensor& t, int types, const char* name) {
  if (!t.is_cuda()) throw ValueError(std::string(name) + " must be a CUDA tensor");
  if (!(type_of(t) & types))
    throw ValueError(std::string(name) + " must be of type" + names(types));
  const int64_t nd = t.dim();
  if (nd == 0) throw ValueError(std::string(name) + " has no dimension");
  const auto size = t.sizes(), stride = t.strides();
  Rows r;
  r.p = t.data_ptr();
  r.cols = size[nd - 1];
  if (r.cols > 1 && stride[nd - 1] != 1)
    throw ValueError(std::string(name) + " must have unit stride in its last dimension");
  r.rows = 1;
  r.ld = -1;
  for (int64_t d = nd - 2; d >= 0; --d) {
    if (size[d] == 0) r.rows = 0;
    if (size[d] <= 1 || r.rows == 0) continue;
    if (r.ld < 0)
      r.ld = stride[d];
    else if (stride[d] != r.ld * r.rows)
      throw ValueError(std::string(name) + ": leading dimensions do not collapse to one row stride");
    r.rows *= size[d];
  }
  if (r.rows <= 1 || r.cols == 0) r.ld = std::max(r.ld, r.cols);
  if (r.ld < r.cols) throw ValueError(std::string(name) + " has overlapping rows");
  return r;
}

void on_device(const Tensor& t, const Tensor& like, const char* name) {
  if (t.device() != like.device())
    throw ValueError(std::string(name) + " is on another device");
}

// A matrix argument that must agree with the call's leading shape and width.
Rows like(const Tensor& t, int types, at::IntArrayRef lead, int64_t cols, const Tensor& ref,
          const char* name) {
  same_shape(t, lead, cols, name);
  on_device(t, ref, name);
  return rows_of(t, types, name);
}

void* vector(const Tensor& t, int types, int64_t n, const Tensor& ref, const char* name) {
  on_device(t, ref, name);
  if (!(type_of(t) & types))
    throw ValueError(std::string(name) + " must be of type" + names(types));
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    throw ValueError(std::string(name) + " must be a contiguous vector of " + std::to_string(n) +
                     " elements");
  return t.data_ptr();
}

struct Packed {
  Rows q;
  uint8_t* scale;
};
Packed packed(PyObject* o, at::IntArrayRef lead, int64_t cols, const Tensor* ref, const char* name) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2)
    throw ValueError(std::string(name) + " must be a Packed8");
  const Tensor& q = tensor(PyTuple_GET_ITEM(o, 0), name);
  const Tensor& s = tensor(PyTuple_GET_ITEM(o, 1), name);
  Packed p;
  if (ref) {
    p.q = like(q, kE4m3, lead, cols, *ref, name);
  } else {
    p.q = rows_of(q, kE4m3, name);
  }
  const auto qs = q.sizes(), ss = s.sizes();
  const size_t n = qs.size();
  if (s.scalar_type() != at::kByte || s.device() != q.device() || !s.is_contiguous() ||
      ss.size() != n || ss.slice(0, n - 1) != qs.slice(0, n - 1) ||
      ss.back() != (p.q.cols + kBlock - 1) / kBlock)
    throw ValueError(std::string(name) +
                     ".scale must be contiguous uint8, one byte for 32 columns of a row");
  p.scale = s.data_ptr<uint8_t>();
  return p;
}

Tensor empty(at::IntArrayRef lead, int64_t cols, at::ScalarType type, const Tensor& ref) {
  c10::SmallVector<int64_t, 8> s(lead.begin(), lead.end());
  s.push_back(cols);
  return at::detail::empty_cuda(s, type, ref.device(), std::nullopt);
}
Tensor bytes(size_t n, const Tensor& ref) {
  return at::detail::empty_cuda({(int64_t)n}, at::kByte, ref.device(), std::nullopt);
}

// An output that the caller may have given.
struct Out {
  Tensor t;
  Rows r;
  bool is_given = false;
  // the call has filled it
  PyObject* done() {
    if (is_given) written(t);
    return THPVariable_Wrap(std::move(t));
  }
};
Out output(PyObject* o, at::IntArrayRef lead, int64_t cols, at::ScalarType type, const Tensor& ref,
           const char* name) {
  Out out;
  if (o == Py_None) {
    out.t = empty(lead, cols, type, ref);
    out.r.p = out.t.data_ptr();
    out.r.ld = cols;
  } else {
    out.t = tensor(o, name);
    out.is_given = true;
    if (out.t.scalar_type() != type) throw ValueError(std::string(name) + " has the wrong type");
    out.r = like(out.t, kBf16 | kF32, lead, cols, ref, name);
  }
  return out;
}

struct Packing {
  Tensor q, scale;
  uint8_t* qp = nullptr;
  uint8_t* sp = nullptr;
};
Packing new_packed(at::IntArrayRef lead, int64_t cols, const Tensor& ref) {
  Packing p;
  p.q = empty(lead, cols, at::kFloat8_e4m3fn, ref);
  p.scale = empty(lead, (cols + kBlock - 1) / kBlock, at::kByte, ref);
  p.qp = static_cast<uint8_t*>(p.q.data_ptr());
  p.sp = p.scale.data_ptr<uint8_t>();
  return p;
}

at::IntArrayRef lead_of(const Tensor& t) { return t.sizes().slice(0, t.dim() - 1); }

void* stream_of(const Tensor& t) {
  return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
}

int integer(PyObject* o) { return (int)PyLong_AsLong(o); }

// ------------------------------------------------------------------ operators
// Each takes its Python arguments by position (layers.py has the names and
// defaults) and returns a new reference.
using Args = PyObject* const*;

PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* tuple(std::initializer_list<PyObject*> v) {
  PyObject* t = PyTuple_New((Py_ssize_t)v.size());
  Py_ssize_t i = 0;
  for (PyObject* o : v) PyTuple_SET_ITEM(t, i++, o);
  return t;
}
PyObject* none() { return Py_NewRef(Py_None); }
bool given(PyObject* o) { return o != Py_None; }

// (x) -> (q, scale)
PyObject* do_pack8(Args a) {
  const Tensor& x = tensor(a[0], "x");
  const Rows r = rows_of(x, kBf16 | kF32, "x");
  c10::cuda::CUDAGuard guard(x.device());
  Packing p = new_packed(lead_of(x), r.cols, x);
  library(scape_layer_pack8(r.p, r.ld, dtype_of(x), r.rows, r.cols, p.qp, r.cols, p.sp, stream_of(x)));
  return tuple({wrap(p.q), wrap(p.scale)});
}

// (packed, is_bf16, activation, out) -> y
PyObject* do_unpack8(Args a) {
  const Packed p = packed(a[0], {}, 0, nullptr, "p");
  const Tensor& q = THPVariable_Unpack(PyTuple_GET_ITEM(a[0], 0));
  const at::ScalarType type = integer(a[1]) ? at::kBFloat16 : at::kFloat;
  c10::cuda::CUDAGuard guard(q.device());
  Out out = output(a[3], lead_of(q), p.q.cols, type, q, "out");
  library(scape_layer_unpack8(static_cast<uint8_t*>(p.q.p), p.q.ld, p.scale, p.q.rows, p.q.cols,
                              integer(a[2]), out.r.p, out.r.ld, dtype_of(out.t), stream_of(q)));
  return out.done();
}

// (dy, packed, activation, out) -> dz
PyObject* do_activation_grad(Args a) {
  const Tensor& dy = tensor(a[0], "dy");
  const Rows r = rows_of(dy, kBf16 | kF32, "dy");
  const Packed p = packed(a[1], lead_of(dy), r.cols, &dy, "pre");
  c10::cuda::CUDAGuard guard(dy.device());
  Out out = output(a[3], lead_of(dy), r.cols, dy.scalar_type(), dy, "out");
  library(scape_layer_act_grad(r.p, r.ld, static_cast<uint8_t*>(p.q.p), p.q.ld, p.scale, r.rows,
                               r.cols, integer(a[2]), out.r.p, out.r.ld, dtype_of(dy), stream_of(dy)));
  return out.done();
}

// (x, weight, residual, eps, pack) -> (y, h, rstd, q, scale), h None without a residual
PyObject* do_add_rmsnorm(Args a) {
  const Tensor& x = tensor(a[0], "x");
  const Rows r = rows_of(x, kBf16 | kF32, "x");
  const auto lead = lead_of(x);
  const Tensor& w = tensor(a[1], "weight");
  const void* wp = vector(w, kBf16 | kF32, r.cols, x, "weight");
  Rows res = {nullptr, 0, 0, r.cols};
  if (given(a[2])) res = like(tensor(a[2], "residual"), type_of(x), lead, r.cols, x, "residual");
  const double eps = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) return nullptr;
  c10::cuda::CUDAGuard guard(x.device());
  Tensor y = empty(lead, r.cols, x.scalar_type(), x), h;
  if (given(a[2])) h = empty(lead, r.cols, x.scalar_type(), x);
  Tensor rstd = at::detail::empty_cuda(lead, at::kFloat, x.device(), std::nullopt);
  Packing p;
  if (integer(a[4])) p = new_packed(lead, r.cols, x);
  library(scape_layer_add_rmsnorm(r.p, r.ld, res.p, res.ld, wp, dtype_of(w), r.rows, r.cols,
                                  (float)eps, dtype_of(x), y.data_ptr(), r.cols,
                                  h.defined() ? h.data_ptr() : nullptr, r.cols,
                                  rstd.data_ptr<float>(), p.qp, r.cols, p.sp, stream_of(x)));
  return tuple({wrap(y), h.defined() ? wrap(h) : none(), wrap(rstd),
                p.qp || p.q.defined() ? wrap(p.q) : none(),
                p.q.defined() ? wrap(p.scale) : none()});
}

// (dy, h, weight, rstd, dh, dweight, out) -> dx
PyObject* do_add_rmsnorm_backward(Args a) {
  const Tensor& dy = tensor(a[0], "dy");
  const Rows r = rows_of(dy, kBf16 | kF32, "dy");
  const auto lead = lead_of(dy);
  const Rows h = like(tensor(a[1], "h"), type_of(dy), lead, r.cols, dy, "h");
  const Tensor& w = tensor(a[2], "weight");
  const void* wp = vector(w, kBf16 | kF32, r.cols, dy, "weight");
  const Tensor& rstd = tensor(a[3], "rstd");
  if (rstd.scalar_type() != at::kFloat || rstd.device() != dy.device() || rstd.numel() != r.rows ||
      !rstd.is_contiguous())
    throw ValueError("rstd must be contiguous float32, one a row");
  Rows dh = {nullptr, 0, 0, r.cols};
  if (given(a[4])) dh = like(tensor(a[4], "dh"), type_of(dy), lead, r.cols, dy, "dh");
  c10::cuda::CUDAGuard guard(dy.device());
  Out out = output(a[6], lead, r.cols, dy.scalar_type(), dy, "out");
  void* dw = nullptr;
  int dwt = SCAPE_F32;
  size_t n = 0;
  Tensor ws;
  if (given(a[5])) {
    const Tensor& t = tensor(a[5], "dweight");
    dw = vector(t, kBf16 | kF32, r.cols, dy, "dweight");
    dwt = dtype_of(t);
    library(scape_layer_add_rmsnorm_bwd_workspace(r.rows, r.cols, &n));
    if (n) ws = bytes(n, dy);
  }
  library(scape_layer_add_rmsnorm_bwd(r.p, r.ld, h.p, h.ld, wp, dtype_of(w), rstd.data_ptr<float>(),
                                      dh.p, dh.ld, r.rows, r.cols, dtype_of(dy), out.r.p, out.r.ld,
                                      dw, dwt, n ? ws.data_ptr() : nullptr, n, stream_of(dy)));
  if (dw) written(tensor(a[5], "dweight"));
  return out.done();
}

Rows weight_of(const Tensor& w, const Tensor& ref) {
  if (w.dim() != 2) throw ValueError("weight must be a matrix");
  on_device(w, ref, "weight");
  return rows_of(w, kBf16, "weight");
}

// (x, weight, bias, residual, activation, keep_pre, out) -> y or (y, q, scale)
PyObject* do_linear(Args a) {
  const Tensor& x = tensor(a[0], "x");
  const Rows r = rows_of(x, kBf16, "x");
  const auto lead = lead_of(x);
  const Rows w = weight_of(tensor(a[1], "weight"), x);
  if (w.cols != r.cols) throw ValueError("weight and x differ in their columns");
  const int64_t n = w.rows;
  const void* bias = given(a[2]) ? vector(tensor(a[2], "bias"), kBf16, n, x, "bias") : nullptr;
  Rows res = {nullptr, 0, 0, n};
  if (given(a[3])) res = like(tensor(a[3], "residual"), kBf16, lead, n, x, "residual");
  c10::cuda::CUDAGuard guard(x.device());
  Out out = output(a[6], lead, n, at::kBFloat16, x, "out");
  Packing p;
  const bool keep = integer(a[5]) != 0;
  if (keep) p = new_packed(lead, n, x);
  size_t bytes_needed = 0;
  library(scape_layer_linear_workspace(r.p, r.ld, w.p, w.ld, r.rows, r.cols, n, &bytes_needed));
  Tensor ws;
  if (bytes_needed) ws = bytes(bytes_needed, x);
  library(scape_layer_linear(r.p, r.ld, w.p, w.ld, bias, res.p, res.ld, r.rows, r.cols, n,
                             integer(a[4]), out.r.p, out.r.ld, p.qp, n, p.sp,
                             bytes_needed ? ws.data_ptr() : nullptr, bytes_needed, stream_of(x)));
  if (!keep) return out.done();
  return tuple({out.done(), wrap(p.q), wrap(p.scale)});
}

// (dy, weight, packed or None, activation, out) -> dx
PyObject* do_linear_backward_input(Args a) {
  const Tensor& dy = tensor(a[0], "dy");
  const Rows r = rows_of(dy, kBf16, "dy");
  const auto lead = lead_of(dy);
  const Rows w = weight_of(tensor(a[1], "weight"), dy);
  if (w.rows != r.cols) throw ValueError("weight's rows are not dy's columns");
  const int64_t k = w.cols;
  Packed p = {{nullptr, 0, 0, k}, nullptr};
  if (given(a[2])) p = packed(a[2], lead, k, &dy, "pre");
  c10::cuda::CUDAGuard guard(dy.device());
  Out out = output(a[4], lead, k, at::kBFloat16, dy, "out");
  size_t n = 0;
  library(scape_layer_linear_bwd_input_workspace(r.p, r.ld, w.p, w.ld, r.rows, k, r.cols, &n));
  Tensor ws;
  if (n) ws = bytes(n, dy);
  library(scape_layer_linear_bwd_input(r.p, r.ld, w.p, w.ld, static_cast<uint8_t*>(p.q.p), p.q.ld,
                                       p.scale, integer(a[3]), r.rows, k, r.cols, out.r.p, out.r.ld,
                                       n ? ws.data_ptr() : nullptr, n, stream_of(dy)));
  return out.done();
}

// (dy, x or packed, activation, dweight or None, dbias or None, new one is float32) -> dweight
PyObject* do_linear_backward_weight(Args a) {
  const Tensor& dy = tensor(a[0], "dy");
  const Rows r = rows_of(dy, kBf16, "dy");
  const auto lead = lead_of(dy);
  Rows x = {nullptr, 0, 0, 0};
  Packed p = {{nullptr, 0, 0, 0}, nullptr};
  int64_t k;
  if (THPVariable_Check(a[1])) {
    const Tensor& t = tensor(a[1], "x");
    k = t.dim() ? t.size(-1) : 0;
    x = like(t, kBf16, lead, k, dy, "x");
    p.q.ld = k;
  } else {
    if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 2)
      throw ValueError("x must be a tensor or a Packed8");
    const Tensor& t = tensor(PyTuple_GET_ITEM(a[1], 0), "x.q");
    k = t.dim() ? t.size(-1) : 0;
    p = packed(a[1], lead, k, &dy, "x");
    x.ld = k;
  }
  const int64_t n = r.cols;
  c10::cuda::CUDAGuard guard(dy.device());
  Tensor dw;
  Rows wr;
  if (given(a[3])) {
    dw = tensor(a[3], "dweight");
    if (dw.dim() != 2 || dw.size(0) != n || dw.size(1) != k)
      throw ValueError("dweight has another shape than dy and x say");
    on_device(dw, dy, "dweight");
    wr = rows_of(dw, kBf16 | kF32, "dweight");
  } else {
    dw = empty({n}, k, integer(a[5]) ? at::kFloat : at::kBFloat16, dy);
    wr = {dw.data_ptr(), n, k, k};
  }
  void* db = given(a[4]) ? vector(tensor(a[4], "dbias"), type_of(dw), n, dy, "dbias") : nullptr;
  size_t need = 0;
  library(scape_layer_linear_bwd_weight_workspace(r.p, r.ld, x.p, x.ld, r.rows, k, n, &need));
  Tensor ws;
  if (need) ws = bytes(need, dy);
  library(scape_layer_linear_bwd_weight(r.p, r.ld, x.p, x.ld, static_cast<uint8_t*>(p.q.p), p.q.ld,
                                        p.scale, integer(a[2]), r.rows, k, n, wr.p, wr.ld, db,
                                        dtype_of(dw), need ? ws.data_ptr() : nullptr, need,
                                        stream_of(dy)));
  if (given(a[3])) written(dw);
  if (db) written(tensor(a[4], "dbias"));
  return wrap(dw);
}

// ------------------------------------------------------------------ tokens
// Tokens or targets: contiguous, int64 or int32.
struct Ids {
  const void* p;
  int bytes;
};
Ids ids_of(const Tensor& t, at::IntArrayRef shape, const Tensor& ref, const char* name) {
  on_device(t, ref, name);
  if (t.scalar_type() != at::kLong && t.scalar_type() != at::kInt)
    throw ValueError(std::string(name) + " must be of type int64 or int32");
  if (t.sizes() != shape) throw ValueError(std::string(name) + " has another shape than the call's other tensors say");
  if (!t.is_contiguous()) throw ValueError(std::string(name) + " must be contiguous");
  return {t.data_ptr(), t.scalar_type() == at::kLong ? 8 : 4};
}
// One float32 a row.
float* floats_of(const Tensor& t, at::IntArrayRef shape, const Tensor& ref, const char* name) {
  on_device(t, ref, name);
  if (t.scalar_type() != at::kFloat || t.sizes() != shape || !t.is_contiguous())
    throw ValueError(std::string(name) + " must be contiguous float32, one a row");
  return t.data_ptr<float>();
}
// A contiguous part of an allocation, from its at-th element on.  (An allocation is a
// microsecond, and several a quarter of what a call for one row takes.)
Tensor part_of(const Tensor& all, int64_t at, at::IntArrayRef sizes) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
  t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  return t;
}
Tensor row_floats(at::IntArrayRef lead, const Tensor& ref) {
  return at::detail::empty_cuda(lead, at::kFloat, ref.device(), std::nullopt);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw ValueError("scale, weight, max_norm and eps must be numbers");
  }
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw ValueError("entropy, lse_rest and accumulate must be true or false");
  }
  return v != 0;
}

Rows table_of(const Tensor& t, const char* name) {
  if (t.dim() != 2) throw ValueError(std::string(name) + " must be a matrix");
  if (t.size(0) == 0) throw ValueError(std::string(name) + " has no rows");
  return rows_of(t, kBf16 | kF32, name);
}

// (tokens, weight, scale, 0 or 1: bfloat16 or 2: float32, out) -> y
PyObject* do_embedding(Args a) {
  const Tensor& tokens = tensor(a[0], "tokens");
  const Tensor& w = tensor(a[1], "weight");
  const Rows t = table_of(w, "weight");
  const Ids ids = ids_of(tokens, tokens.sizes(), w, "tokens");
  const double scale = number(a[2]);
  const int kind = integer(a[3]);
  c10::cuda::CUDAGuard guard(w.device());
  at::ScalarType type = kind == 0 ? w.scalar_type() : kind == 1 ? at::kBFloat16 : at::kFloat;
  if (kind == 0 && given(a[4])) {
    const Tensor& o = tensor(a[4], "out");
    if (type_of(o) & (kBf16 | kF32)) type = o.scalar_type();
  }
  Out out = output(a[4], tokens.sizes(), t.cols, type, w, "out");
  library(scape_layer_embedding(ids.p, ids.bytes, tokens.numel(), t.p, t.ld, dtype_of(w), t.rows, t.cols,
                                (float)scale, out.r.p, out.r.ld, dtype_of(out.t), stream_of(w)));
  return out.done();
}

// (dy, tokens, dweight, scale, accumulate) -> dweight
PyObject* do_embedding_backward(Args a) {
  const Tensor& dy = tensor(a[0], "dy");
  const Rows r = rows_of(dy, kBf16 | kF32, "dy");
  const Ids ids = ids_of(tensor(a[1], "tokens"), lead_of(dy), dy, "tokens");
  const Tensor& dw = tensor(a[2], "dweight");
  on_device(dw, dy, "dweight");
  const Rows w = table_of(dw, "dweight");
  if (w.cols != r.cols) throw ValueError("dweight and dy differ in their columns");
  const double scale = number(a[3]);
  const bool accumulate = truth(a[4]);
  c10::cuda::CUDAGuard guard(dy.device());
  size_t n = 0;
  library(scape_layer_embedding_bwd_workspace(r.rows, w.rows, r.cols, &n));
  Tensor ws;
  if (n) ws = bytes(n, dy);
  library(scape_layer_embedding_bwd(r.p, r.ld, dtype_of(dy), ids.p, ids.bytes, r.rows, w.rows, r.cols, (float)scale,
                                    accumulate, w.p, w.ld, dtype_of(dw), n ? ws.data_ptr() : nullptr, n,
                                    stream_of(dy)));
  written(dw);
  return wrap(dw);
}

// (logits, targets, entropy, top, with lse_rest) -> (logprob, lse, entropy, top_logprob, top_token[, lse_rest])
PyObject* do_token_logprobs(Args a) {
  const Tensor& x = tensor(a[0], "logits");
  const Rows r = rows_of(x, kBf16 | kF32, "logits");
  const auto lead = lead_of(x);
  const Ids ids = ids_of(tensor(a[1], "targets"), lead, x, "targets");
  const bool entropy = truth(a[2]);
  const long top = PyLong_AsLong(a[3]);
  if (top == -1 && PyErr_Occurred()) return nullptr;
  if (top < 0 || top > SCAPE_TOP_MAX || top > r.cols)
    throw ValueError("top must be 0 to 32, and at most the logits' columns");
  const bool with_rest = truth(a[4]);
  c10::cuda::CUDAGuard guard(x.device());
  const int64_t each = (r.rows + 127) / 128 * 128, at_ent = 2 * each, at_rest = at_ent + (entropy ? each : 0),
                at_tops = at_rest + (with_rest ? each : 0);
  const Tensor all = row_floats({at_tops + r.rows * top}, x);
  Tensor lp = part_of(all, 0, lead), lse = part_of(all, each, lead), rest, ent, tops, token;
  if (entropy) ent = part_of(all, at_ent, lead);
  if (with_rest) rest = part_of(all, at_rest, lead);
  if (top) {
    c10::SmallVector<int64_t, 8> sizes(lead.begin(), lead.end());
    sizes.push_back(top);
    tops = part_of(all, at_tops, sizes);
    token = empty(lead, top, at::kLong, x);
  }
  library(scape_layer_token_logprobs_rest(
      r.p, r.ld, dtype_of(x), ids.p, ids.bytes, r.rows, r.cols, (int)top, lp.data_ptr<float>(), lse.data_ptr<float>(),
      with_rest ? rest.data_ptr<float>() : nullptr, entropy ? ent.data_ptr<float>() : nullptr,
      top ? tops.data_ptr<float>() : nullptr, top ? token.data_ptr<int64_t>() : nullptr, stream_of(x)));
  PyObject* const e = entropy ? wrap(ent) : none();
  PyObject* const l = top ? wrap(tops) : none();
  PyObject* const k = top ? wrap(token) : none();
  if (with_rest) return tuple({wrap(lp), wrap(lse), e, l, k, wrap(rest)});
  return tuple({wrap(lp), wrap(lse), e, l, k});
}

// (logits, targets, lse, dlogprob, entropy or None, dentropy or None, out, lse_rest or None) -> dlogits
PyObject* do_token_logprobs_backward(Args a) {
  const Tensor& x = tensor(a[0], "logits");
  const Rows r = rows_of(x, kBf16 | kF32, "logits");
  const auto lead = lead_of(x);
  const Ids ids = ids_of(tensor(a[1], "targets"), lead, x, "targets");
  const float* lse = floats_of(tensor(a[2], "lse"), lead, x, "lse");
  const float* dlp = floats_of(tensor(a[3], "dlogprob"), lead, x, "dlogprob");
  const float* ent = given(a[4]) ? floats_of(tensor(a[4], "entropy"), lead, x, "entropy") : nullptr;
  const float* dent = given(a[5]) ? floats_of(tensor(a[5], "dentropy"), lead, x, "dentropy") : nullptr;
  const float* rest = given(a[7]) ? floats_of(tensor(a[7], "lse_rest"), lead, x, "lse_rest") : nullptr;
  c10::cuda::CUDAGuard guard(x.device());
  Out out = output(a[6], lead, r.cols, x.scalar_type(), x, "out");
  library(scape_layer_token_logprobs_rest_bwd(r.p, r.ld, dtype_of(x), ids.p, ids.bytes, r.rows, r.cols, lse, rest, dlp,
                                              ent, dent, out.r.p, out.r.ld, stream_of(x)));
  return out.done();
}

// (logits, targets, weight or None, weight of every row, out) -> (loss, dlogits)
PyObject* do_token_loss(Args a) {
  const Tensor& x = tensor(a[0], "logits");
  const Rows r = rows_of(x, kBf16 | kF32, "logits");
  const auto lead = lead_of(x);
  const Ids ids = ids_of(tensor(a[1], "targets"), lead, x, "targets");
  const float* w = given(a[2]) ? floats_of(tensor(a[2], "weight"), lead, x, "weight") : nullptr;
  const double all = number(a[3]);
  c10::cuda::CUDAGuard guard(x.device());
  Out out = output(a[4], lead, r.cols, x.scalar_type(), x, "out");
  Tensor loss = row_floats(lead, x), ws;
  size_t n = 0;
  library(scape_layer_token_loss_workspace(r.p, r.ld, dtype_of(x), r.rows, r.cols, out.r.p, out.r.ld, &n));
  if (n) ws = bytes(n, x);
  library(scape_layer_token_loss(r.p, r.ld, dtype_of(x), ids.p, ids.bytes, r.rows, r.cols, w, (float)all,
                                 loss.data_ptr<float>(), out.r.p, out.r.ld, n ? ws.data_ptr() : nullptr, n,
                                 stream_of(x)));
  return tuple({wrap(loss), out.done()});
}

// ------------------------------------------------------------------ gradients
struct Set {
  std::vector<Tensor> t;
  std::vector<const void*> p;
  std::vector<int64_t> numel;
  std::vector<int> dtype;
};
Set set_of(PyObject* o, const char* name) {
  Set s;
  if (THPVariable_Check(o)) throw ValueError(std::string(name) + " must be a list or tuple of tensors");
  PyObject* seq = PySequence_Fast(o, "");
  if (!seq) {
    PyErr_Clear();
    throw ValueError(std::string(name) + " must be a list or tuple of tensors");
  }
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
  try {
    s.t.reserve(n), s.p.reserve(n), s.numel.reserve(n), s.dtype.reserve(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      const Tensor& t = tensor(PySequence_Fast_GET_ITEM(seq, i), name);
      if (!t.is_cuda()) throw ValueError(std::string(name) + " must be CUDA tensors");
      if (!(type_of(t) & (kBf16 | kF32)))
        throw ValueError(std::string(name) + " must be of type" + names(kBf16 | kF32));
      if (i && t.device() != s.t[0].device()) throw ValueError(std::string(name) + " are on several devices");
      if (!t.is_non_overlapping_and_dense())
        throw ValueError(std::string(name) + " holds a tensor whose elements do not lie together");
      s.t.push_back(t);
      s.p.push_back(t.data_ptr());
      s.numel.push_back(t.numel());
      s.dtype.push_back(dtype_of(t));
    }
  } catch (...) {
    Py_DECREF(seq);
    throw;
  }
  Py_DECREF(seq);
  if (n == 0) throw ValueError(std::string(name) + " has no tensor");
  if (n > 0x7FFFFFFF) throw ValueError(std::string(name) + " has too many tensors");
  return s;
}
// The norm and the workspace.  A kept norm keeps its allocation, so the workspace has
// one of its own, unless both fit in kTogether: two allocations take no less, as each is
// 512 bytes at least, and the second is a microsecond of the 6 that a small set takes.
struct NormSpace {
  static constexpr int64_t kTogether = 1024, kNormFloats = 64;
  Tensor norm, own;
  void* ws = nullptr;
  size_t n = 0;
  explicit NormSpace(const Set& s) {
    library(scape_layer_grad_norm_workspace((int)s.t.size(), s.numel.data(), &n));
    if (kNormFloats * 4 + (int64_t)n <= kTogether) {
      const Tensor all = row_floats({kNormFloats + (int64_t)(n / 4)}, s.t[0]);
      norm = part_of(all, 0, {});
      if (n) ws = all.data_ptr<float>() + kNormFloats;
    } else {
      norm = row_floats({}, s.t[0]);
      own = bytes(n, s.t[0]);
      ws = own.data_ptr();
    }
  }
};

// (grads) -> norm
PyObject* do_grad_norm(Args a) {
  const Set s = set_of(a[0], "grads");
  c10::cuda::CUDAGuard guard(s.t[0].device());
  const NormSpace to(s);
  library(scape_layer_grad_norm((int)s.t.size(), s.p.data(), s.numel.data(), s.dtype.data(), to.norm.data_ptr<float>(),
                                to.ws, to.n, stream_of(s.t[0])));
  return wrap(to.norm);
}

// (grads, max_norm, eps, out or None) -> norm
PyObject* do_clip_grad_norm(Args a) {
  const Set s = set_of(a[0], "grads");
  const double max_norm = number(a[1]), eps = number(a[2]);
  Set o;
  if (given(a[3])) {
    o = set_of(a[3], "out");
    if (o.t.size() != s.t.size()) throw ValueError("out has another number of tensors than grads");
    for (size_t i = 0; i < s.t.size(); ++i) {
      on_device(o.t[i], s.t[0], "out");
      if (o.t[i].sizes() != s.t[i].sizes()) throw ValueError("a tensor of out has another shape than grads'");
      if (o.t[i].strides() != s.t[i].strides() && !(o.t[i].is_contiguous() && s.t[i].is_contiguous()))
        throw ValueError("a tensor of out has its dimensions in another order than grads'");
    }
  }
  c10::cuda::CUDAGuard guard(s.t[0].device());
  const NormSpace to(s);
  const Set& into = given(a[3]) ? o : s;
  library(scape_layer_clip_grads((int)s.t.size(), s.p.data(), s.numel.data(), s.dtype.data(),
                                 const_cast<void* const*>(into.p.data()), into.dtype.data(), (float)max_norm,
                                 (float)eps, to.norm.data_ptr<float>(), to.ws, to.n, stream_of(s.t[0])));
  for (const Tensor& t : into.t) written(t);
  return wrap(to.norm);
}

// () -> int
PyObject* do_status(Args) {
  int v = 0, rc = 0;
  void* st = c10::cuda::getCurrentCUDAStream().stream();
  // the stream may have to wait for a host function that needs the interpreter
  Py_BEGIN_ALLOW_THREADS rc = scape_layer_status(&v, st);
  Py_END_ALLOW_THREADS
  library(rc);
  return PyLong_FromLong(v);
}

// ------------------------------------------------------------------ module
// Raises module.name(*args); takes the reference to args.
void raise(const char* module, const char* name, PyObject* args) {
  PyObject* m = PyImport_ImportModule(module);
  PyObject* c = m ? PyObject_GetAttrString(m, name) : nullptr;
  PyObject* x = c && args ? PyObject_CallObject(c, args) : nullptr;
  if (x) PyErr_SetObject(c, x);
  Py_XDECREF(x);
  Py_XDECREF(c);
  Py_XDECREF(m);
  Py_XDECREF(args);
}

template <PyObject* (*F)(Args), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    PyObject* r = F(args);
    if (r && PyErr_Occurred()) {
      Py_DECREF(r);
      return nullptr;
    }
    return r;
  } catch (const ValueError& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const LibraryError& e) {
    raise("sparse_communication_sharded_gb300._scape", "ScapeError",
          Py_BuildValue("(is)", e.code, scape_layer_last_error()));
  } catch (const c10::OutOfMemoryError& e) {
    raise("torch", "OutOfMemoryError", Py_BuildValue("(s)", e.what_without_backtrace()));
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define ENTRY(name, n) \
  {#name, (PyCFunction)(void (*)(void))entry<do_##name, n>, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {ENTRY(pack8, 1),
                          ENTRY(unpack8, 4),
                          ENTRY(activation_grad, 4),
                          ENTRY(add_rmsnorm, 5),
                          ENTRY(add_rmsnorm_backward, 7),
                          ENTRY(linear, 7),
                          ENTRY(linear_backward_input, 5),
                          ENTRY(linear_backward_weight, 6),
                          ENTRY(embedding, 5),
                          ENTRY(embedding_backward, 5),
                          ENTRY(token_logprobs, 5),
                          ENTRY(token_logprobs_backward, 8),
                          ENTRY(token_loss, 5),
                          ENTRY(grad_norm, 1),
                          ENTRY(clip_grad_norm, 4),
                          ENTRY(status, 0),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_layers_torch", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers_torch(void) { return PyModule_Create(&kModule); }
