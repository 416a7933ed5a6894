// binding.cpp -- CPython binding of the operators in include/gemm_ops.h: reads
// the tensors' type, device, shape and strides, allocates results and
// workspaces with torch's allocator and calls the C ABI, whose functions ops.py
// hands over once.  Calls for few tokens are bound by the host.  One of w4_linear
// takes 4.5 us (10 us through ctypes and the tensors' Python attributes, 7.4 us
// through those attributes from here), of gated_ffn 7.9 us (two launches; 12.9).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/AutogradState.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <utility>

#include "gemm_ops.h"

namespace {

// What ops.py hands over (setup).
PyObject* g_error;
decltype(&gemm_gated_ffn_workspace) g_ffn_space;
decltype(&gemm_gated_ffn) g_ffn;
decltype(&gemm_gated_ffn_backward_workspace) g_bwd_space;
decltype(&gemm_gated_ffn_backward) g_bwd;
decltype(&gemm_w4_workspace) g_w4_space;
decltype(&gemm_w4_linear) g_w4;
decltype(&gemm_w4_gated) g_w4g;
decltype(&gemm_layer_norm) g_ln;
decltype(&gemm_rms_norm) g_rms;
decltype(&gemm_norm_backward_workspace) g_norm_bwd_space;
decltype(&gemm_layer_norm_backward) g_ln_bwd;
decltype(&gemm_rms_norm_backward) g_rms_bwd;
decltype(&gemm_linear_cross_entropy_workspace) g_xent_space;
decltype(&gemm_linear_cross_entropy) g_xent;
decltype(&gemm_linear_cross_entropy_backward_workspace) g_xent_bwd_space;
decltype(&gemm_linear_cross_entropy_backward) g_xent_bwd;

PyObject* s_cuda_stream;

// An owned reference.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* o = nullptr) : p(o) {}
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
  ~Ref() { Py_XDECREF(p); }
  PyObject* release() {
    PyObject* r = p;
    p = nullptr;
    return r;
  }
};

bool to_i64(PyObject* o, int64_t* v) {  // takes a borrowed reference
  *v = PyLong_AsLongLong(o);
  return *v != -1 || !PyErr_Occurred();
}

// One 2-D operand.
struct Mat {
  void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
};

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return "float16";
    case at::kBFloat16: return "bfloat16";
    case at::kByte: return "uint8";
    case at::kFloat: return "float32";
    case at::kLong: return "int64";
    default: return c10::toString(t);
  }
}

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
  PyErr_Format(PyExc_TypeError, "%s must be a tensor, got %R", name, reinterpret_cast<PyObject*>(Py_TYPE(o)));
  return nullptr;
}

// The operators record no graph and carry no tangents on: a tensor that asks for
// either is refused, rather than its gradient lost in silence.
bool no_graph(const at::Tensor& t, const char* name) {
  const auto& mode = c10::AutogradState::get_tls_state();
  const char* asks = mode.get_grad_mode() && t.requires_grad()               ? "requires grad"
                     : mode.get_fw_grad_mode() && t._fw_grad(0).defined() ? "has a forward-mode tangent"
                                                                            : nullptr;
  if (!asks) return true;
  PyErr_Format(PyExc_RuntimeError,
               "%s %s, and this operator records no graph: call it under torch.no_grad() or on detached tensors "
               "(gradients are operators of their own: gated_ffn_backward computes gated_ffn's)",
               name, asks);
  return false;
}

// A tensor that has to have this type and be on this device; null, with an
// error set, for any other object.
const at::Tensor* operand(PyObject* o, const char* name, at::ScalarType dtype, int64_t index) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return nullptr;
  if (t->scalar_type() != dtype) {
    PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name, type_name(dtype), type_name(t->scalar_type()));
    return nullptr;
  }
  if (!no_graph(*t, name)) return nullptr;
  if (!t->is_cuda()) {
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
    return nullptr;
  }
  if (t->get_device() != index) {
    PyErr_Format(PyExc_ValueError, "%s is on cuda:%d, the handle on cuda:%lld", name,
                 static_cast<int>(t->get_device()), static_cast<long long>(index));
    return nullptr;
  }
  return t;
}

// Reads o, such a tensor of two dimensions, and its row distance; rows and cols,
// where not -1, are what it has to have.
bool read(PyObject* o, const char* name, at::ScalarType dtype, int64_t index, int64_t rows, int64_t cols,
          bool contiguous, Mat* m) {
  const at::Tensor* t = operand(o, name, dtype, index);
  if (!t) return false;
  if (t->dim() != 2) {
    PyErr_Format(PyExc_ValueError, "%s must be 2-D, got %lld dimensions", name, static_cast<long long>(t->dim()));
    return false;
  }
  m->rows = t->size(0);
  m->cols = t->size(1);
  if ((rows >= 0 && m->rows != rows) || (cols >= 0 && m->cols != cols)) {
    PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld], got [%lld, %lld]", name,
                 static_cast<long long>(rows >= 0 ? rows : m->rows), static_cast<long long>(cols >= 0 ? cols : m->cols),
                 static_cast<long long>(m->rows), static_cast<long long>(m->cols));
    return false;
  }
  m->ld = m->cols;
  if (!t->is_contiguous()) {
    if (contiguous) {
      PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
      return false;
    }
    const int64_t ld = t->stride(0);
    if ((m->cols > 1 && t->stride(1) != 1) || (m->rows > 1 && ld < m->cols)) {
      PyErr_Format(PyExc_ValueError, "%s's rows must be contiguous", name);
      return false;
    }
    // One row or none, or nothing in a row: the distance to the next is free.
    if (m->rows > 1 && m->cols > 0) m->ld = ld;
  }
  m->p = t->data_ptr();
  return true;
}

// x's type: one of the two 16-bit ones, or float32 where the operator takes it.
bool read_x(PyObject* x, int64_t index, at::ScalarType* dtype, gemm_dtype_t* code, Mat* m, bool f32 = false) {
  const at::Tensor* t = tensor(x, "x");
  if (!t) return false;
  *dtype = t->scalar_type();
  if (*dtype != at::kHalf && *dtype != at::kBFloat16 && !(f32 && *dtype == at::kFloat)) {
    PyErr_Format(PyExc_TypeError, "x must be %s, got %s", f32 ? "float16, bfloat16 or float32" : "float16 or bfloat16",
                 type_name(*dtype));
    return false;
  }
  *code = *dtype == at::kHalf ? GEMM_F16 : *dtype == at::kBFloat16 ? GEMM_BF16 : GEMM_F32;
  return read(x, "x", *dtype, index, -1, -1, false, m);
}

// A vector of n elements side by side, or, where the operator takes any, `stride` apart.
bool read_vector(PyObject* o, const char* name, at::ScalarType dtype, int64_t index, int64_t n, void** p,
                 int64_t* stride = nullptr) {
  const at::Tensor* t = operand(o, name, dtype, index);
  if (!t) return false;
  if (t->dim() != 1 || t->size(0) != n) {
    PyErr_Format(PyExc_ValueError, "%s must be 1-D of %lld elements", name, static_cast<long long>(n));
    return false;
  }
  if (stride) *stride = n > 1 ? t->stride(0) : 1;
  if (!stride && n > 1 && t->stride(0) != 1) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    return false;
  }
  *p = t->data_ptr();
  return true;
}

// A norm's weight, or None: of x's type or float32, which `dtype` becomes.
bool read_weight(PyObject* o, int64_t index, int64_t n, at::ScalarType* dtype, gemm_dtype_t* code, void** p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o, "weight");
  if (!t) return false;
  if (t->scalar_type() == at::kFloat) *dtype = at::kFloat, *code = GEMM_F32;
  return read_vector(o, "weight", *dtype, index, n, p);
}

at::TensorOptions on(int64_t index, at::ScalarType dtype) {
  return at::TensorOptions().dtype(dtype).device(at::kCUDA, static_cast<c10::DeviceIndex>(index));
}

// A new matrix.
PyObject* empty(int64_t rows, int64_t cols, at::ScalarType dtype, int64_t index, void** p) {
  at::Tensor t = at::empty({rows, cols}, on(index, dtype));
  *p = t.data_ptr();
  return THPVariable_Wrap(std::move(t));
}

PyObject* empty_vector(int64_t n, at::ScalarType dtype, int64_t index, void** p) {
  at::Tensor t = at::empty({n}, on(index, dtype));
  *p = t.data_ptr();
  return THPVariable_Wrap(std::move(t));
}

// A workspace, freed in stream order when it goes out of scope; none for 0 bytes.
struct Workspace {
  at::Tensor t;
  void* p = nullptr;
  Workspace(size_t bytes, int64_t index) {
    if (!bytes) return;
    t = at::empty({static_cast<int64_t>(bytes)}, on(index, at::kByte));
    p = t.data_ptr();
  }
};

// `out`, checked, or a new matrix.
PyObject* result(PyObject* out, int64_t rows, int64_t cols, at::ScalarType dtype, int64_t index, Mat* m) {
  if (out == Py_None) {
    m->rows = rows, m->cols = cols, m->ld = cols;
    return empty(rows, cols, dtype, index, &m->p);
  }
  if (!read(out, "out", dtype, index, rows, cols, false, m)) return nullptr;
  return Py_NewRef(out);
}

// A tensor given as `out` has been written: autograd then refuses to use a value
// saved before.  (Tensors made in inference mode have no version.)
void wrote(PyObject* out) {
  if (out == Py_None) return;
  const at::Tensor& t = THPVariable_Unpack(out);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// The stream of a call: the device's current one, an address, or a torch
// stream.  What the call allocates belongs to that stream: a workspace of the
// current stream could be handed out again there while another still uses it.
struct Stream {
  c10::cuda::OptionalCUDAStreamGuard guard;
  void* s = nullptr;

  bool open(PyObject* o, int64_t index) {
    const auto dev = static_cast<c10::DeviceIndex>(index);
    if (o == Py_None) {
      s = c10::cuda::getCurrentCUDAStream(dev).stream();
      return true;
    }
    int64_t v;
    if (PyLong_Check(o)) {
      if (!to_i64(o, &v)) return false;
    } else {
      Ref r(PyObject_GetAttr(o, s_cuda_stream));
      if (!r.p || !to_i64(r.p, &v)) return false;
    }
    if (v == 1) v = 0;  // the legacy default stream by its handle: torch knows it as 0
    s = reinterpret_cast<void*>(v);
    guard.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(s), dev));
    return true;
  }
};

bool act_of(PyObject* o, gemm_act_t* a) {
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "silu") == 0) return *a = GEMM_ACT_SILU, true;
    if (PyUnicode_CompareWithASCIIString(o, "gelu_tanh") == 0) return *a = GEMM_ACT_GELU_TANH, true;
    if (PyUnicode_CompareWithASCIIString(o, "relu") == 0) return *a = GEMM_ACT_RELU, true;
  }
  PyErr_Format(PyExc_ValueError, "act must be 'silu', 'gelu_tanh' or 'relu', got %R", o);
  return false;
}

bool failed(gemm_status_t st, const char* where) {
  if (st == GEMM_OK) return false;
  Ref e(PyObject_CallFunction(g_error, "is", static_cast<int>(st), where));
  if (e.p) PyErr_SetObject(g_error, e.p);
  return true;
}

// The first two arguments of every call: handle, device index.
struct Target {
  gemm_ops_t h;
  int64_t index;
};
bool target(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, Target* t) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
    return false;
  }
  int64_t h;
  if (!to_i64(a[0], &h) || !to_i64(a[1], &t->index)) return false;
  t->h = reinterpret_cast<gemm_ops_t>(h);
  return true;
}

// (handle, index, x, w_in, w_down, act, save, out, stream)
PyObject* py_ffn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Target t;
  Mat x, wi, wd, y;
  at::ScalarType dt;
  gemm_dtype_t code;
  gemm_act_t act;
  if (!target(a, n, 9, &t) || !act_of(a[5], &act) || !read_x(a[2], t.index, &dt, &code, &x) ||
      !read(a[4], "w_down", dt, t.index, x.cols, -1, false, &wd) ||
      !read(a[3], "w_in", dt, t.index, 2 * wd.cols, x.cols, false, &wi))
    return nullptr;
  const int64_t T = x.rows, D = x.cols, F = wd.cols;
  const int save = PyObject_IsTrue(a[6]);
  Stream stream;
  if (save < 0 || !stream.open(a[8], t.index)) return nullptr;
  Ref out(result(a[7], T, D, dt, t.index, &y));
  if (!out.p) return nullptr;
  void* gp = nullptr;
  Ref gu(save ? empty(T, 2 * F, dt, t.index, &gp) : nullptr);
  if (save && !gu.p) return nullptr;
  const size_t need = g_ffn_space(t.h, T, D, F);
  const Workspace ws(need, t.index);
  gemm_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_ffn(t.h, x.p, x.ld, wi.p, wi.ld, wd.p, wd.ld, y.p, y.ld, gp, ws.p, need, T, D, F, act, code, stream.s);
  Py_END_ALLOW_THREADS;
  if (failed(st, "gemm_gated_ffn")) return nullptr;
  wrote(a[7]);
  return save ? PyTuple_Pack(2, out.p, gu.p) : out.release();
  END_HANDLE_TH_ERRORS
}

// (handle, index, dy, x, w_in, w_down, gu, act, stream)
PyObject* py_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Target t;
  Mat dy, x, wi, wd, gu;
  at::ScalarType dt;
  gemm_dtype_t code;
  gemm_act_t act;
  if (!target(a, n, 9, &t) || !act_of(a[7], &act) || !read_x(a[3], t.index, &dt, &code, &x) ||
      !read(a[5], "w_down", dt, t.index, x.cols, -1, false, &wd) ||
      !read(a[4], "w_in", dt, t.index, 2 * wd.cols, x.cols, false, &wi) ||
      !read(a[2], "dy", dt, t.index, x.rows, x.cols, false, &dy) ||
      !read(a[6], "gu", dt, t.index, x.rows, 2 * wd.cols, true, &gu))
    return nullptr;
  const int64_t T = x.rows, D = x.cols, F = wd.cols;
  Stream stream;
  if (!stream.open(a[8], t.index)) return nullptr;
  void *dxp, *dip, *ddp;
  Ref dx(empty(T, D, dt, t.index, &dxp));
  if (!dx.p) return nullptr;
  Ref di(empty(2 * F, D, dt, t.index, &dip));
  if (!di.p) return nullptr;
  Ref dd(empty(D, F, dt, t.index, &ddp));
  if (!dd.p) return nullptr;
  const size_t need = g_bwd_space(t.h, T, D, F);
  const Workspace ws(need, t.index);
  gemm_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_bwd(t.h, dy.p, dy.ld, x.p, x.ld, wi.p, wi.ld, wd.p, wd.ld, gu.p, dxp, D, dip, ddp, ws.p, need, T, D, F, act,
             code, stream.s);
  Py_END_ALLOW_THREADS;
  if (failed(st, "gemm_gated_ffn_backward")) return nullptr;
  return PyTuple_Pack(3, dx.p, di.p, dd.p);
  END_HANDLE_TH_ERRORS
}

// (handle, index, x, codes, scales, zeros, act or None, out, stream);
// act: gated.
PyObject* py_w4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Target t;
  Mat x, codes, scales, zeros, y;
  at::ScalarType dt;
  gemm_dtype_t code;
  gemm_act_t act = GEMM_ACT_SILU;
  const bool gated = n > 6 && a[6] != Py_None;
  if (!target(a, n, 9, &t) || (gated && !act_of(a[6], &act)) || !read_x(a[2], t.index, &dt, &code, &x) ||
      !read(a[3], "codes", at::kByte, t.index, -1, -1, true, &codes) ||
      !read(a[4], "scales", dt, t.index, codes.rows, -1, true, &scales))
    return nullptr;
  const int64_t T = x.rows, K = x.cols, groups = scales.cols;
  if (codes.cols * 2 != K) {
    PyErr_Format(PyExc_ValueError, "codes must be [N, %lld] for x of %lld columns, got [%lld, %lld]", K / 2, K,
                 codes.rows, codes.cols);
    return nullptr;
  }
  if ((groups == 0) != (K == 0) || (K != 0 && K % groups != 0)) {
    PyErr_Format(PyExc_ValueError, "scales must be [%lld, K / group], got [%lld, %lld]", codes.rows, scales.rows,
                 groups);
    return nullptr;
  }
  if (a[5] != Py_None && !read(a[5], "zeros", at::kByte, t.index, codes.rows, groups, true, &zeros)) return nullptr;
  if (gated && codes.rows % 2 != 0) {
    PyErr_SetString(PyExc_ValueError, "gated weights have an even number of rows: gate rows, then up rows");
    return nullptr;
  }
  const int64_t N = gated ? codes.rows / 2 : codes.rows, group = groups ? K / groups : 32;
  Stream stream;
  if (!stream.open(a[8], t.index)) return nullptr;
  Ref out(result(a[7], T, N, dt, t.index, &y));
  if (!out.p) return nullptr;
  const size_t need = g_w4_space(t.h, T, N, K, gated);
  const Workspace ws(need, t.index);
  gemm_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = gated ? g_w4g(t.h, x.p, x.ld, codes.p, scales.p, zeros.p, y.p, y.ld, ws.p, need, T, N, K, group, act, code, stream.s)
             : g_w4(t.h, x.p, x.ld, codes.p, scales.p, zeros.p, y.p, y.ld, ws.p, need, T, N, K, group, code, stream.s);
  Py_END_ALLOW_THREADS;
  if (failed(st, gated ? "gemm_w4_gated" : "gemm_w4_linear")) return nullptr;
  wrote(a[7]);
  return out.release();
  END_HANDLE_TH_ERRORS
}

// (handle, index, x, weight, bias, eps, save, out, stream); kRms: without a bias.
template <bool kRms>
PyObject* py_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Target t;
  Mat x, y;
  at::ScalarType dt;
  gemm_dtype_t code;
  void *weight, *bias = nullptr;
  if (!target(a, n, 9, &t) || !read_x(a[2], t.index, &dt, &code, &x, true)) return nullptr;
  const int64_t T = x.rows, D = x.cols;
  at::ScalarType wdt = dt;
  gemm_dtype_t wcode = code;
  if (!read_weight(a[3], t.index, D, &wdt, &wcode, &weight)) return nullptr;
  if (!kRms && a[4] != Py_None) {
    if (!weight) {
      PyErr_SetString(PyExc_ValueError, "a bias needs a weight");
      return nullptr;
    }
    if (!read_vector(a[4], "bias", wdt, t.index, D, &bias)) return nullptr;
  }
  const double eps = PyFloat_AsDouble(a[5]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const int save = PyObject_IsTrue(a[6]);
  Stream stream;
  if (save < 0 || !stream.open(a[8], t.index)) return nullptr;
  Ref out(result(a[7], T, D, dt, t.index, &y));
  if (!out.p) return nullptr;
  void* sp = nullptr;
  Ref stats(save ? empty(T, kRms ? 1 : 2, at::kFloat, t.index, &sp) : nullptr);
  if (save && !stats.p) return nullptr;
  gemm_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  if constexpr (kRms)
    st = g_rms(t.h, x.p, x.ld, weight, y.p, y.ld, static_cast<float*>(sp), T, D, static_cast<float>(eps), code, wcode,
               stream.s);
  else
    st = g_ln(t.h, x.p, x.ld, weight, bias, y.p, y.ld, static_cast<float*>(sp), T, D, static_cast<float>(eps), code,
              wcode, stream.s);
  Py_END_ALLOW_THREADS;
  if (failed(st, kRms ? "gemm_rms_norm" : "gemm_layer_norm")) return nullptr;
  wrote(a[7]);
  return save ? PyTuple_Pack(2, out.p, stats.p) : out.release();
  END_HANDLE_TH_ERRORS
}

// (handle, index, dy, x, weight, stats, bias, stream); bias: whether its gradient
// is wanted.
template <bool kRms>
PyObject* py_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Target t;
  Mat dy, x, stats;
  at::ScalarType dt;
  gemm_dtype_t code;
  void* weight;
  if (!target(a, n, 8, &t) || !read_x(a[3], t.index, &dt, &code, &x, true)) return nullptr;
  const int64_t T = x.rows, D = x.cols;
  at::ScalarType wdt = dt;
  gemm_dtype_t wcode = code;
  if (!read_weight(a[4], t.index, D, &wdt, &wcode, &weight) || !read(a[2], "dy", dt, t.index, T, D, false, &dy) ||
      !read(a[5], "stats", at::kFloat, t.index, T, kRms ? 1 : 2, true, &stats))
    return nullptr;
  const int bias = kRms ? 0 : PyObject_IsTrue(a[6]);
  Stream stream;
  if (bias < 0 || !stream.open(a[7], t.index)) return nullptr;
  void *dxp, *dwp = nullptr, *dbp = nullptr;
  Ref dx(empty(T, D, dt, t.index, &dxp));
  if (!dx.p) return nullptr;
  Ref dw(weight ? empty_vector(D, wdt, t.index, &dwp) : Py_NewRef(Py_None));
  if (!dw.p) return nullptr;
  Ref db(bias ? empty_vector(D, wdt, t.index, &dbp) : Py_NewRef(Py_None));
  if (!db.p) return nullptr;
  const size_t need = g_norm_bwd_space(t.h, T, D);
  const Workspace ws(need, t.index);
  gemm_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  if constexpr (kRms)
    st = g_rms_bwd(t.h, dy.p, dy.ld, x.p, x.ld, weight, static_cast<const float*>(stats.p), dxp, D, dwp, ws.p, need, T, D,
                   code, wcode, stream.s);
  else
    st = g_ln_bwd(t.h, dy.p, dy.ld, x.p, x.ld, weight, static_cast<const float*>(stats.p), dxp, D, dwp, dbp, ws.p, need,
                  T, D, code, wcode, stream.s);
  Py_END_ALLOW_THREADS;
  if (failed(st, kRms ? "gemm_rms_norm_backward" : "gemm_layer_norm_backward")) return nullptr;
  if constexpr (kRms)
    return PyTuple_Pack(2, dx.p, dw.p);
  else
    return PyTuple_Pack(3, dx.p, dw.p, db.p);
  END_HANDLE_TH_ERRORS
}

// (handle, index, x, w, targets, ignore_index, save, out, stream)
PyObject* py_xent(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Target t;
  Mat x, w;
  at::ScalarType dt;
  gemm_dtype_t code;
  void *targets, *loss, *lse = nullptr;
  int64_t ignore;
  if (!target(a, n, 9, &t) || !read_x(a[2], t.index, &dt, &code, &x) ||
      !read(a[3], "w", dt, t.index, -1, x.cols, false, &w) ||
      !read_vector(a[4], "targets", at::kLong, t.index, x.rows, &targets) || !to_i64(a[5], &ignore))
    return nullptr;
  const int64_t T = x.rows, D = x.cols, V = w.rows;
  const int save = PyObject_IsTrue(a[6]);
  Stream stream;
  if (save < 0 || !stream.open(a[8], t.index)) return nullptr;
  const bool given = a[7] != Py_None;
  if (given && !read_vector(a[7], "out", at::kFloat, t.index, T, &loss)) return nullptr;
  Ref out(given ? Py_NewRef(a[7]) : empty_vector(T, at::kFloat, t.index, &loss));
  if (!out.p) return nullptr;
  Ref kept(save ? empty_vector(T, at::kFloat, t.index, &lse) : nullptr);
  if (save && !kept.p) return nullptr;
  const size_t need = g_xent_space(t.h, T, D, V);
  const Workspace ws(need, t.index);
  gemm_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_xent(t.h, x.p, x.ld, w.p, w.ld, static_cast<const int64_t*>(targets), static_cast<float*>(loss),
              static_cast<float*>(lse), ws.p, need, T, D, V, ignore, code, stream.s);
  Py_END_ALLOW_THREADS;
  if (failed(st, "gemm_linear_cross_entropy")) return nullptr;
  wrote(a[7]);
  return save ? PyTuple_Pack(2, out.p, kept.p) : out.release();
  END_HANDLE_TH_ERRORS
}

// (handle, index, dloss, x, w, targets, lse, ignore_index, dlse or None, stream)
PyObject* py_xent_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Target t;
  Mat x, w;
  at::ScalarType dt;
  gemm_dtype_t code;
  void *dloss, *dlse = nullptr, *targets, *lse;
  int64_t ignore, dloss_stride, dlse_stride = 0;
  if (!target(a, n, 10, &t) || !read_x(a[3], t.index, &dt, &code, &x) ||
      !read(a[4], "w", dt, t.index, -1, x.cols, false, &w) ||
      !read_vector(a[2], "dloss", at::kFloat, t.index, x.rows, &dloss, &dloss_stride) ||
      !read_vector(a[5], "targets", at::kLong, t.index, x.rows, &targets) ||
      !read_vector(a[6], "lse", at::kFloat, t.index, x.rows, &lse) || !to_i64(a[7], &ignore))
    return nullptr;
  if (a[8] != Py_None && !read_vector(a[8], "dlse", at::kFloat, t.index, x.rows, &dlse, &dlse_stride)) return nullptr;
  const int64_t T = x.rows, D = x.cols, V = w.rows;
  Stream stream;
  if (!stream.open(a[9], t.index)) return nullptr;
  void *dxp, *dwp;
  Ref dx(empty(T, D, dt, t.index, &dxp));
  if (!dx.p) return nullptr;
  Ref dw(empty(V, D, dt, t.index, &dwp));
  if (!dw.p) return nullptr;
  const size_t need = g_xent_bwd_space(t.h, T, D, V);
  const Workspace ws(need, t.index);
  gemm_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_xent_bwd(t.h, static_cast<const float*>(dloss), dloss_stride, static_cast<const float*>(dlse), dlse_stride, x.p,
                  x.ld, w.p, w.ld, static_cast<const int64_t*>(targets), static_cast<const float*>(lse), dxp, D, dwp, ws.p,
                  need, T, D, V, ignore, code, stream.s);
  Py_END_ALLOW_THREADS;
  if (failed(st, "gemm_linear_cross_entropy_backward")) return nullptr;
  return PyTuple_Pack(2, dx.p, dw.p);
  END_HANDLE_TH_ERRORS
}

// (tensor, name): refuses as no_graph does.
PyObject* py_no_graph(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2) return PyErr_Format(PyExc_TypeError, "%zd arguments, 2 expected", n);
  const char* name = PyUnicode_AsUTF8(a[1]);
  const at::Tensor* t = name ? tensor(a[0], name) : nullptr;
  if (!t || !no_graph(*t, name)) return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (tensor): it has been written.
PyObject* py_wrote(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 1) return PyErr_Format(PyExc_TypeError, "%zd arguments, 1 expected", n);
  if (!tensor(a[0], "out")) return nullptr;
  wrote(a[0]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// (GemmError, then the addresses of the C functions, in this order)
PyObject* py_setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const std::pair<void*, size_t> fns[] = {
      {&g_ffn_space, sizeof g_ffn_space}, {&g_ffn, sizeof g_ffn}, {&g_bwd_space, sizeof g_bwd_space},
      {&g_bwd, sizeof g_bwd}, {&g_w4_space, sizeof g_w4_space}, {&g_w4, sizeof g_w4}, {&g_w4g, sizeof g_w4g},
      {&g_ln, sizeof g_ln}, {&g_rms, sizeof g_rms}, {&g_norm_bwd_space, sizeof g_norm_bwd_space},
      {&g_ln_bwd, sizeof g_ln_bwd}, {&g_rms_bwd, sizeof g_rms_bwd},
      {&g_xent_space, sizeof g_xent_space}, {&g_xent, sizeof g_xent}, {&g_xent_bwd_space, sizeof g_xent_bwd_space},
      {&g_xent_bwd, sizeof g_xent_bwd}};
  constexpr Py_ssize_t want = 1 + sizeof fns / sizeof fns[0];
  if (n != want) return PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
  void* addr[want];
  for (Py_ssize_t i = 1; i < want; ++i) {
    addr[i] = PyLong_AsVoidPtr(a[i]);
    if (!addr[i] && PyErr_Occurred()) return nullptr;
  }
  for (Py_ssize_t i = 1; i < want; ++i) std::memcpy(fns[i - 1].first, &addr[i], fns[i - 1].second);
  Py_XSETREF(g_error, Py_NewRef(a[0]));
  Py_RETURN_NONE;
}

template <PyObject* (*kF)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kF));
}

PyMethodDef methods[] = {
    {"setup", fast<py_setup>(), METH_FASTCALL, nullptr},
    {"gated_ffn", fast<py_ffn>(), METH_FASTCALL, nullptr},
    {"gated_ffn_backward", fast<py_bwd>(), METH_FASTCALL, nullptr},
    {"w4", fast<py_w4>(), METH_FASTCALL, nullptr},
    {"layer_norm", fast<py_norm<false>>(), METH_FASTCALL, nullptr},
    {"rms_norm", fast<py_norm<true>>(), METH_FASTCALL, nullptr},
    {"layer_norm_backward", fast<py_norm_bwd<false>>(), METH_FASTCALL, nullptr},
    {"rms_norm_backward", fast<py_norm_bwd<true>>(), METH_FASTCALL, nullptr},
    {"linear_cross_entropy", fast<py_xent>(), METH_FASTCALL, nullptr},
    {"linear_cross_entropy_backward", fast<py_xent_bwd>(), METH_FASTCALL, nullptr},
    {"no_graph", fast<py_no_graph>(), METH_FASTCALL, nullptr},
    {"wrote", fast<py_wrote>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  if (!(s_cuda_stream = PyUnicode_InternFromString("cuda_stream"))) return nullptr;
  return PyModule_Create(&module);
}
