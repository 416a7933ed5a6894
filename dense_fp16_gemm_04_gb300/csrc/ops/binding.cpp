// binding.cpp -- CPython binding of the operators in include/gemm_ops.h: reads
// the tensors' type, device, shape and strides, allocates results and
// workspaces with torch's allocator and calls the C ABI.  Small products are
// bound by the host: through ctypes and Python code the checks and the
// marshalling of one w4_linear call took 10 us, of which the library itself
// needs 2.4; through this binding it takes 7, of which 1.5 each allocate the
// result and a workspace.  It is built without torch's headers: a tensor is used through
// its Python attributes, and the library through addresses that ops.py hands
// over once.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cstdint>

#include "gemm_ops.h"

namespace {

// What ops.py hands over (setup).
PyObject *g_empty, *g_f16, *g_bf16, *g_u8, *g_raw_stream, *g_error;
decltype(&gemm_gated_ffn_workspace) g_ffn_space;
decltype(&gemm_gated_ffn) g_ffn;
decltype(&gemm_gated_ffn_backward_workspace) g_bwd_space;
decltype(&gemm_gated_ffn_backward) g_bwd;
decltype(&gemm_w4_workspace) g_w4_space;
decltype(&gemm_w4_linear) g_w4;
decltype(&gemm_w4_gated) g_w4g;

PyObject *s_dtype, *s_shape, *s_get_device, *s_is_contiguous, *s_stride, *s_data_ptr, *s_cuda_stream, *kw_empty;

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

PyObject* call0(PyObject* self, PyObject* name) {
  PyObject* args[1] = {self};
  return PyObject_VectorcallMethod(name, args, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, nullptr);
}

bool to_i64(PyObject* o, int64_t* v) {  // takes a borrowed reference
  *v = PyLong_AsLongLong(o);
  return *v != -1 || !PyErr_Occurred();
}

bool int_call(PyObject* self, PyObject* name, int64_t* v) {
  Ref r(call0(self, name));
  return r.p && to_i64(r.p, v);
}

bool pair(PyObject* tuple, int64_t* a, int64_t* b) {
  return to_i64(PyTuple_GET_ITEM(tuple, 0), a) && to_i64(PyTuple_GET_ITEM(tuple, 1), b);
}

// One 2-D operand.
struct Mat {
  void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
};

// Reads t, which has to have this type and be on this device, and its row
// distance; rows and cols, where not -1, are what it has to have.
bool read(PyObject* t, const char* name, PyObject* dtype, int64_t index, int64_t rows, int64_t cols,
          bool contiguous, Mat* m) {
  Ref dt(PyObject_GetAttr(t, s_dtype));
  if (!dt.p) return false;
  if (dt.p != dtype) {
    PyErr_Format(PyExc_TypeError, "%s must be %S, got %S", name, dtype, dt.p);
    return false;
  }
  int64_t dev;
  if (!int_call(t, s_get_device, &dev)) return false;
  if (dev != index) {
    if (dev < 0)
      PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
    else
      PyErr_Format(PyExc_ValueError, "%s is on cuda:%lld, the handle on cuda:%lld", name, dev, index);
    return false;
  }
  Ref shape(PyObject_GetAttr(t, s_shape));
  if (!shape.p) return false;
  if (!PyTuple_Check(shape.p) || PyTuple_GET_SIZE(shape.p) != 2) {
    PyErr_Format(PyExc_ValueError, "%s must be 2-D, got %S", name, shape.p);
    return false;
  }
  if (!pair(shape.p, &m->rows, &m->cols)) return false;
  if ((rows >= 0 && m->rows != rows) || (cols >= 0 && m->cols != cols)) {
    if (rows >= 0 && cols >= 0)
      PyErr_Format(PyExc_ValueError, "%s must be [%lld, %lld], got %S", name, rows, cols, shape.p);
    else
      PyErr_Format(PyExc_ValueError, "%s must have %lld %s, got %S", name, rows >= 0 ? rows : cols,
                   rows >= 0 ? "rows" : "columns", shape.p);
    return false;
  }
  Ref cont(call0(t, s_is_contiguous));
  if (!cont.p) return false;
  m->ld = m->cols;
  if (cont.p != Py_True) {
    if (contiguous) {
      PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
      return false;
    }
    Ref st(call0(t, s_stride));
    int64_t ld, inner;
    if (!st.p || !pair(st.p, &ld, &inner)) return false;
    if ((m->cols > 1 && inner != 1) || (m->rows > 1 && ld < m->cols)) {
      PyErr_Format(PyExc_ValueError, "%s's rows must be contiguous", name);
      return false;
    }
    // One row or none, or nothing in a row: the distance to the next is free.
    if (m->rows > 1 && m->cols > 0) m->ld = ld;
  }
  int64_t p;
  if (!int_call(t, s_data_ptr, &p)) return false;
  m->p = reinterpret_cast<void*>(p);
  return true;
}

// x's type: one of the two 16-bit ones.
bool read_x(PyObject* x, int64_t index, PyObject** dtype, gemm_dtype_t* code, Mat* m) {
  Ref dt(PyObject_GetAttr(x, s_dtype));
  if (!dt.p) return false;
  if (dt.p != g_f16 && dt.p != g_bf16) {
    PyErr_Format(PyExc_TypeError, "x must be float16 or bfloat16, got %S", dt.p);
    return false;
  }
  *dtype = dt.p == g_f16 ? g_f16 : g_bf16;
  *code = dt.p == g_f16 ? GEMM_F16 : GEMM_BF16;
  return read(x, "x", *dtype, index, -1, -1, false, m);
}

// A new tensor: a matrix, or (cols < 0) `rows` bytes.
PyObject* empty(int64_t rows, int64_t cols, PyObject* dtype, PyObject* device, void** p) {
  Ref size(cols < 0 ? Py_BuildValue("(L)", static_cast<long long>(rows))
                    : Py_BuildValue("(LL)", static_cast<long long>(rows), static_cast<long long>(cols)));
  if (!size.p) return nullptr;
  PyObject* args[3] = {size.p, dtype, device};
  Ref t(PyObject_Vectorcall(g_empty, args, 1, kw_empty));
  int64_t a;
  if (!t.p || !int_call(t.p, s_data_ptr, &a)) return nullptr;
  *p = reinterpret_cast<void*>(a);
  return t.release();
}

// `out`, checked, or a new matrix.
PyObject* result(PyObject* out, int64_t rows, int64_t cols, PyObject* dtype, int64_t index, PyObject* device,
                 Mat* m) {
  if (out == Py_None) {
    m->rows = rows, m->cols = cols, m->ld = cols;
    return empty(rows, cols, dtype, device, &m->p);
  }
  if (!read(out, "out", dtype, index, rows, cols, false, m)) return nullptr;
  return Py_NewRef(out);
}

// The current stream of the device, an address, or a torch stream.
bool stream_of(PyObject* o, PyObject* index, void** s) {
  int64_t v;
  if (o == Py_None) {
    Ref r(PyObject_CallOneArg(g_raw_stream, index));
    if (!r.p || !to_i64(r.p, &v)) return false;
  } else if (PyLong_Check(o)) {
    if (!to_i64(o, &v)) return false;
  } else {
    Ref r(PyObject_GetAttr(o, s_cuda_stream));
    if (!r.p || !to_i64(r.p, &v)) return false;
  }
  *s = reinterpret_cast<void*>(v);
  return true;
}

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

// The first three arguments of every call: handle, device index, torch device.
struct Target {
  gemm_ops_t h;
  int64_t index;
  PyObject* device;
};
bool target(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, Target* t) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
    return false;
  }
  int64_t h;
  if (!to_i64(a[0], &h) || !to_i64(a[1], &t->index)) return false;
  t->h = reinterpret_cast<gemm_ops_t>(h);
  t->device = a[2];
  return true;
}

// (handle, index, device, x, w_in, w_down, act, save, out, stream)
PyObject* py_ffn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Target t;
  Mat x, wi, wd, y;
  PyObject* dt;
  gemm_dtype_t code;
  gemm_act_t act;
  if (!target(a, n, 10, &t) || !act_of(a[6], &act) || !read_x(a[3], t.index, &dt, &code, &x) ||
      !read(a[5], "w_down", dt, t.index, x.cols, -1, false, &wd) ||
      !read(a[4], "w_in", dt, t.index, 2 * wd.cols, x.cols, false, &wi))
    return nullptr;
  const int64_t T = x.rows, D = x.cols, F = wd.cols;
  const int save = PyObject_IsTrue(a[7]);
  if (save < 0) return nullptr;
  Ref out(result(a[8], T, D, dt, t.index, t.device, &y));
  if (!out.p) return nullptr;
  void *gp = nullptr, *wp = nullptr, *s;
  Ref gu(save ? empty(T, 2 * F, dt, t.device, &gp) : nullptr);
  if (save && !gu.p) return nullptr;
  const size_t need = g_ffn_space(t.h, T, D, F);
  Ref ws(need ? empty(static_cast<int64_t>(need), -1, g_u8, t.device, &wp) : nullptr);
  if ((need && !ws.p) || !stream_of(a[9], a[1], &s)) return nullptr;
  gemm_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_ffn(t.h, x.p, x.ld, wi.p, wi.ld, wd.p, wd.ld, y.p, y.ld, gp, wp, need, T, D, F, act, code, s);
  Py_END_ALLOW_THREADS;
  if (failed(st, "gemm_gated_ffn")) return nullptr;
  return save ? PyTuple_Pack(2, out.p, gu.p) : out.release();
}

// (handle, index, device, dy, x, w_in, w_down, gu, act, stream)
PyObject* py_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Target t;
  Mat dy, x, wi, wd, gu;
  PyObject* dt;
  gemm_dtype_t code;
  gemm_act_t act;
  if (!target(a, n, 10, &t) || !act_of(a[8], &act) || !read_x(a[4], t.index, &dt, &code, &x) ||
      !read(a[6], "w_down", dt, t.index, x.cols, -1, false, &wd) ||
      !read(a[5], "w_in", dt, t.index, 2 * wd.cols, x.cols, false, &wi) ||
      !read(a[3], "dy", dt, t.index, x.rows, x.cols, false, &dy) ||
      !read(a[7], "gu", dt, t.index, x.rows, 2 * wd.cols, true, &gu))
    return nullptr;
  const int64_t T = x.rows, D = x.cols, F = wd.cols;
  void *dxp, *dip, *ddp, *wp = nullptr, *s;
  Ref dx(empty(T, D, dt, t.device, &dxp));
  if (!dx.p) return nullptr;
  Ref di(empty(2 * F, D, dt, t.device, &dip));
  if (!di.p) return nullptr;
  Ref dd(empty(D, F, dt, t.device, &ddp));
  if (!dd.p) return nullptr;
  const size_t need = g_bwd_space(t.h, T, D, F);
  Ref ws(need ? empty(static_cast<int64_t>(need), -1, g_u8, t.device, &wp) : nullptr);
  if ((need && !ws.p) || !stream_of(a[9], a[1], &s)) return nullptr;
  gemm_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = g_bwd(t.h, dy.p, dy.ld, x.p, x.ld, wi.p, wi.ld, wd.p, wd.ld, gu.p, dxp, D, dip, ddp, wp, need, T, D, F, act,
             code, s);
  Py_END_ALLOW_THREADS;
  if (failed(st, "gemm_gated_ffn_backward")) return nullptr;
  return PyTuple_Pack(3, dx.p, di.p, dd.p);
}

// (handle, index, device, x, codes, scales, zeros, act or None, out, stream);
// act: gated.
PyObject* py_w4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  Target t;
  Mat x, codes, scales, zeros, y;
  PyObject* dt;
  gemm_dtype_t code;
  gemm_act_t act = GEMM_ACT_SILU;
  const bool gated = n > 7 && a[7] != Py_None;
  if (!target(a, n, 10, &t) || (gated && !act_of(a[7], &act)) || !read_x(a[3], t.index, &dt, &code, &x) ||
      !read(a[4], "codes", g_u8, t.index, -1, -1, true, &codes) ||
      !read(a[5], "scales", dt, t.index, codes.rows, -1, true, &scales))
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
  if (a[6] != Py_None && !read(a[6], "zeros", g_u8, t.index, codes.rows, groups, true, &zeros)) return nullptr;
  if (gated && codes.rows % 2 != 0) {
    PyErr_SetString(PyExc_ValueError, "gated weights have an even number of rows: gate rows, then up rows");
    return nullptr;
  }
  const int64_t N = gated ? codes.rows / 2 : codes.rows, group = groups ? K / groups : 32;
  Ref out(result(a[8], T, N, dt, t.index, t.device, &y));
  if (!out.p) return nullptr;
  void *wp = nullptr, *s;
  const size_t need = g_w4_space(t.h, T, N, K, gated);
  Ref ws(need ? empty(static_cast<int64_t>(need), -1, g_u8, t.device, &wp) : nullptr);
  if ((need && !ws.p) || !stream_of(a[9], a[1], &s)) return nullptr;
  gemm_status_t st;
  Py_BEGIN_ALLOW_THREADS;
  st = gated ? g_w4g(t.h, x.p, x.ld, codes.p, scales.p, zeros.p, y.p, y.ld, wp, need, T, N, K, group, act, code, s)
             : g_w4(t.h, x.p, x.ld, codes.p, scales.p, zeros.p, y.p, y.ld, wp, need, T, N, K, group, code, s);
  Py_END_ALLOW_THREADS;
  if (failed(st, gated ? "gemm_w4_gated" : "gemm_w4_linear")) return nullptr;
  return out.release();
}

// (torch.empty, float16, bfloat16, uint8, raw stream of a device,
// GemmError, then the addresses of the seven C functions)
PyObject* py_setup(PyObject*, PyObject* args) {
  unsigned long long f[7];
  PyObject* o[6];
  if (!PyArg_ParseTuple(args, "OOOOOOKKKKKKK", &o[0], &o[1], &o[2], &o[3], &o[4], &o[5], &f[0], &f[1], &f[2],
                        &f[3], &f[4], &f[5], &f[6]))
    return nullptr;
  PyObject** to[6] = {&g_empty, &g_f16, &g_bf16, &g_u8, &g_raw_stream, &g_error};
  for (int i = 0; i < 6; ++i) Py_XSETREF(*to[i], Py_NewRef(o[i]));
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
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  struct {
    PyObject** to;
    const char* text;
  } const names[] = {{&s_dtype, "dtype"},   {&s_shape, "shape"},   {&s_get_device, "get_device"},
                     {&s_is_contiguous, "is_contiguous"}, {&s_stride, "stride"}, {&s_data_ptr, "data_ptr"},
                     {&s_cuda_stream, "cuda_stream"}};
  for (const auto& n : names)
    if (!(*n.to = PyUnicode_InternFromString(n.text))) return nullptr;
  kw_empty = Py_BuildValue("(ss)", "dtype", "device");
  if (!kw_empty) return nullptr;
  return PyModule_Create(&module);
}
