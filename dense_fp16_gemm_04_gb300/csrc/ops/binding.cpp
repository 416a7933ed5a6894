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
               "(gated_ffn_backward computes the gradients of gated_ffn)",
               name, asks);
  return false;
}

// Reads o, a tensor that has to have this type and be on this device, and its
// row distance; rows and cols, where not -1, are what it has to have.
bool read(PyObject* o, const char* name, at::ScalarType dtype, int64_t index, int64_t rows, int64_t cols,
          bool contiguous, Mat* m) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  if (t->scalar_type() != dtype) {
    PyErr_Format(PyExc_TypeError, "%s must be %s, got %s", name, type_name(dtype), type_name(t->scalar_type()));
    return false;
  }
  if (!no_graph(*t, name)) return false;
  if (!t->is_cuda()) {
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
    return false;
  }
  if (t->get_device() != index) {
    PyErr_Format(PyExc_ValueError, "%s is on cuda:%d, the handle on cuda:%lld", name,
                 static_cast<int>(t->get_device()), static_cast<long long>(index));
    return false;
  }
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

// x's type: one of the two 16-bit ones.
bool read_x(PyObject* x, int64_t index, at::ScalarType* dtype, gemm_dtype_t* code, Mat* m) {
  const at::Tensor* t = tensor(x, "x");
  if (!t) return false;
  *dtype = t->scalar_type();
  if (*dtype != at::kHalf && *dtype != at::kBFloat16) {
    PyErr_Format(PyExc_TypeError, "x must be float16 or bfloat16, got %s", type_name(*dtype));
    return false;
  }
  *code = *dtype == at::kHalf ? GEMM_F16 : GEMM_BF16;
  return read(x, "x", *dtype, index, -1, -1, false, m);
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

// (GemmError, then the addresses of the seven C functions)
PyObject* py_setup(PyObject*, PyObject* args) {
  unsigned long long f[7];
  PyObject* error;
  if (!PyArg_ParseTuple(args, "OKKKKKKK", &error, &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6])) return nullptr;
  Py_XSETREF(g_error, Py_NewRef(error));
  g_ffn_space = reinterpret_cast<decltype(g_ffn_space)>(f[0]);
  g_ffn = reinterpret_cast<decltype(g_ffn)>(f[1]);
  g_bwd_space = reinterpret_cast<decltype(g_bwd_space)>(f[2]);
  g_bwd = reinterpret_cast<decltype(g_bwd)>(f[3]);
  g_w4_space = reinterpret_cast<decltype(g_w4_space)>(f[4]);
  g_w4 = reinterpret_cast<decltype(g_w4)>(f[5]);
  g_w4g = reinterpret_cast<decltype(g_w4g)>(f[6]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", py_setup, METH_VARARGS, nullptr},
    {"gated_ffn", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_ffn)), METH_FASTCALL, nullptr},
    {"gated_ffn_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_bwd)), METH_FASTCALL, nullptr},
    {"w4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_w4)), METH_FASTCALL, nullptr},
    {"no_graph", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_no_graph)), METH_FASTCALL, nullptr},
    {"wrote", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_wrote)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  if (!(s_cuda_stream = PyUnicode_InternFromString("cuda_stream"))) return nullptr;
  return PyModule_Create(&module);
}
