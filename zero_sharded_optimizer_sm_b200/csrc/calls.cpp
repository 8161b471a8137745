// The calls around a layer's products from Python, for their plain use: every
// tensor on the current device, the current stream, new results.  A small
// call's kernels take a few microseconds; checking the operands, taking memory
// and calling through ctypes took 9 to 16 on the host (norm of one token 13 us
// a call, 20 with its backward pass), and from here 3 to 7.
//
// Python's lock is let go of while memory is taken and kernels are launched, as
// ctypes does: a launch waits where the stream's queue is full, and what it waits
// for may be another Python thread's to enqueue.  The operands are their caller's
// meanwhile; nothing of Python is touched.
//
// A function returns None for whatever is not plain -- another stream or device,
// a wrong type or shape, an error of the library -- and the caller, which has
// every check and every message, goes the long way.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include "../../include/zero_sm.h"

namespace {

int code_of(at::ScalarType t) {
  return t == at::kBFloat16 ? ZERO_DTYPE_BF16 : t == at::kHalf ? ZERO_DTYPE_F16 : t == at::kFloat ? ZERO_DTYPE_F32 : -1;
}

// The current device and stream, asked for once a call.
struct Here {
  c10::DeviceIndex device = c10::cuda::current_device();
  void* stream = c10::cuda::getCurrentCUDAStream(device).stream();
  at::Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::detail::empty_cuda(size, type, at::Device(at::kCUDA, device), std::nullopt);
  }
};

const at::Tensor* tensor(PyObject* o, const Here& h) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.device().index() == h.device ? &t : nullptr;
}

// A dense matrix with contiguous rows.
struct Matrix {
  const at::Tensor* t = nullptr;
  void* at = nullptr;
  int code = -1;
  int64_t rows = 0, cols = 0, ld = 0;
  bool read(PyObject* o, const Here& h) {
    t = tensor(o, h);
    if (!t || t->dim() != 2 || (code = code_of(t->scalar_type())) < 0) return false;
    rows = t->size(0), cols = t->size(1);
    if (cols > 1 && t->stride(1) != 1) return false;
    ld = rows > 1 ? t->stride(0) : cols;
    at = t->data_ptr();
    return true;
  }
  // The same, of another's shape and type.
  bool like(PyObject* o, const Here& h, const Matrix& m) {
    return read(o, h) && rows == m.rows && cols == m.cols && code == m.code;
  }
};

struct Vector {
  void* at = nullptr;
  int code = -1;
  at::ScalarType type = at::kFloat;
  bool read(PyObject* o, const Here& h, int64_t n) {
    const at::Tensor* t = tensor(o, h);
    if (!t || t->dim() != 1 || t->size(0) != n || (n > 1 && t->stride(0) != 1)) return false;
    type = t->scalar_type(), code = code_of(type), at = t->data_ptr();
    return code >= 0;
  }
};

struct Tokens {
  void* at = nullptr;
  int size = 0;
  int64_t n = 0;
  bool read(PyObject* o, const Here& h) {
    const at::Tensor* t = tensor(o, h);
    if (!t || t->dim() != 1) return false;
    size = t->scalar_type() == at::kLong ? 8 : t->scalar_type() == at::kInt ? 4 : 0;
    n = t->size(0), at = t->data_ptr();
    return size && (n <= 1 || t->stride(0) == 1);
  }
};

// ------------------------------------------------------------- MX matrices --

// The package's classes, and the names of what they keep.
PyObject *g_mx4 = nullptr, *g_mx8 = nullptr;
PyObject *s_codes, *s_scales, *s_space, *s_rows, *s_cols, *s_device, *s_at, *s_struct, *g_no_args;

bool whole(PyObject* o, int64_t* v) {
  *v = o && PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
  return *v >= 0;
}
bool take(PyObject* o, PyObject* name, int64_t* v) {
  PyObject* a = PyObject_GetAttr(o, name);
  const bool ok = whole(a, v);
  Py_XDECREF(a);
  return ok;
}

// zero_mx4 and zero_mx8 have the same members.
template <class M>
bool read_mx(PyObject* o, PyObject* type, const Here& h, M* m) {
  if ((PyObject*)Py_TYPE(o) != type) return false;
  bool ok = take(o, s_rows, &m->rows) && take(o, s_cols, &m->cols);
  PyObject* d = ok ? PyObject_GetAttr(o, s_device) : nullptr;
  ok = d && THPDevice_Check(d) && ((THPDevice*)d)->device == at::Device(at::kCUDA, h.device);
  Py_XDECREF(d);
  PyObject* at = ok ? PyObject_GetAttr(o, s_at) : nullptr;
  int64_t v[4];
  ok = at && PyTuple_Check(at) && PyTuple_GET_SIZE(at) == 4;
  for (int i = 0; ok && i < 4; ++i) ok = whole(PyTuple_GET_ITEM(at, i), &v[i]);
  Py_XDECREF(at);
  if (ok) {
    m->codes = reinterpret_cast<void*>(v[0]), m->scales = reinterpret_cast<void*>(v[1]);
    m->code_pitch = v[2], m->scale_pitch = v[3];
  }
  PyErr_Clear();
  return ok;
}

bool put(PyObject* o, PyObject* name, PyObject* value) {  // takes the value's reference
  const bool ok = value && PyObject_SetAttr(o, name, value) == 0;
  Py_XDECREF(value);
  return ok;
}

// Memory of a new MX8 matrix, and the package's own object of it.
at::Tensor mx8_memory(int64_t rows, int64_t cols, const Here& h, zero_mx8* m) {
  const int64_t nb = (cols + 31) / 32, cp = 32 * nb, sp = (nb + 15) / 16 * 16;
  at::Tensor space = h.empty({rows * (cp + sp)}, at::kByte);
  uint8_t* at = static_cast<uint8_t*>(space.data_ptr());
  *m = {at, at + rows * cp, rows, cols, cp, sp};
  return space;
}
PyObject* mx8_object(at::Tensor&& space, const Here& h, const zero_mx8& m) {
  PyTypeObject* type = (PyTypeObject*)g_mx8;
  PyObject* o = type->tp_new(type, g_no_args, nullptr);
  if (!o) return nullptr;
  const bool ok = put(o, s_space, THPVariable_Wrap(std::move(space))) && put(o, s_codes, Py_NewRef(Py_None)) &&
                  put(o, s_scales, Py_NewRef(Py_None)) && put(o, s_struct, Py_NewRef(Py_None)) &&
                  put(o, s_rows, PyLong_FromLongLong(m.rows)) && put(o, s_cols, PyLong_FromLongLong(m.cols)) &&
                  put(o, s_device, THPDevice_New(at::Device(at::kCUDA, h.device))) &&
                  put(o, s_at, Py_BuildValue("(LLLL)", (long long)m.codes, (long long)m.scales, (long long)m.code_pitch,
                                            (long long)m.scale_pitch));
  if (!ok) Py_CLEAR(o);
  return o;
}

// ----------------------------------------------------------------- the calls --

// C++ exceptions (no memory, say) end as None too: the long way meets them again.
template <class F>
PyObject* plainly(F f) {
  PyObject* r = nullptr;
  try {
    r = f();
  } catch (...) {
    r = nullptr;
  }
  if (r) return r;
  PyErr_Clear();
  Py_RETURN_NONE;
}

// Python's lock let go of, until the end of the scope.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F>
zero_status unlocked(F f) {
  const Unlocked scope;
  return f();
}

PyObject* wrap(at::Tensor&& t) { return t.defined() ? THPVariable_Wrap(std::move(t)) : Py_NewRef(Py_None); }

// mx8_quantize(x)
PyObject* mx8_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plainly([&]() -> PyObject* {
    const Here here;
    Matrix x;
    zero_mx8 m;
    if (n != 1 || !x.read(a[0], here)) return nullptr;
    at::Tensor space;
    const zero_status st = unlocked([&] {
      space = mx8_memory(x.rows, x.cols, here, &m);
      return zero_mx8_quantize(x.at, x.code, x.rows, x.cols, x.ld, &m, here.stream);
    });
    return st == ZERO_OK ? mx8_object(std::move(space), here, m) : nullptr;
  });
}

// mx8_dequantize(m, dtype)
PyObject* mx8_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plainly([&]() -> PyObject* {
    const Here here;
    zero_mx8 m;
    if (n != 2 || !read_mx(a[0], g_mx8, here, &m) || !THPDtype_Check(a[1])) return nullptr;
    const at::ScalarType type = ((THPDtype*)a[1])->scalar_type;
    if (code_of(type) < 0) return nullptr;
    at::Tensor out;
    const zero_status st = unlocked([&] {
      out = here.empty({m.rows, m.cols}, type);
      return zero_mx8_dequantize(&m, out.data_ptr(), code_of(type), m.cols, here.stream);
    });
    return st == ZERO_OK ? wrap(std::move(out)) : nullptr;
  });
}

// rms_norm(x, weight, eps, residual or None, h, rstd): (y, h, rstd), None for those not wanted
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plainly([&]() -> PyObject* {
    const Here here;
    Matrix x, r;
    Vector w;
    if (n != 6 || !PyFloat_Check(a[2]) || !x.read(a[0], here) || !w.read(a[1], here, x.cols)) return nullptr;
    if (a[3] != Py_None && !r.like(a[3], here, x)) return nullptr;
    if (!PyBool_Check(a[4]) || !PyBool_Check(a[5])) return nullptr;
    const at::ScalarType type = x.t->scalar_type();
    const bool want_h = a[4] == Py_True, want_s = a[5] == Py_True;
    const double eps = PyFloat_AS_DOUBLE(a[2]);
    at::Tensor y, h, s;
    const zero_status st = unlocked([&] {
      y = here.empty({x.rows, x.cols}, type);
      if (want_h) h = here.empty({x.rows, x.cols}, type);
      if (want_s) s = here.empty({x.rows}, at::kFloat);
      return zero_rms_norm(x.at, r.at, x.code, x.rows, x.cols, x.ld, r.ld, w.at, w.code, eps, y.data_ptr(), x.cols,
                           want_h ? h.data_ptr() : nullptr, x.cols, nullptr, nullptr,
                           want_s ? static_cast<float*>(s.data_ptr()) : nullptr, here.stream);
    });
    if (st != ZERO_OK) return nullptr;
    return Py_BuildValue("(NNN)", wrap(std::move(y)), wrap(std::move(h)), wrap(std::move(s)));
  });
}

// rms_norm_backward(dy, h, weight, rstd, dh or None): (dx, dw)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plainly([&]() -> PyObject* {
    const Here here;
    Matrix dy, h, dh;
    Vector w, s;
    zero_mx8 m;
    if (n != 5 || !dy.read(a[0], here)) return nullptr;
    const bool kept = (PyObject*)Py_TYPE(a[1]) == g_mx8;
    if (kept ? !read_mx(a[1], g_mx8, here, &m) || m.rows != dy.rows || m.cols != dy.cols : !h.like(a[1], here, dy)) return nullptr;
    if (!w.read(a[2], here, dy.cols) || !s.read(a[3], here, dy.rows) || s.code != ZERO_DTYPE_F32) return nullptr;
    if (a[4] != Py_None && !dh.like(a[4], here, dy)) return nullptr;
    int64_t need = 0;
    if (zero_rms_norm_backward_workspace(dy.rows, dy.cols, &need) != ZERO_OK) return nullptr;
    const at::ScalarType type = dy.t->scalar_type();
    at::Tensor dx, dw;
    const zero_status st = unlocked([&] {
      dx = here.empty({dy.rows, dy.cols}, type), dw = here.empty({dy.cols}, w.type);
      at::Tensor space = here.empty({need}, at::kByte);
      return zero_rms_norm_backward(dy.at, dy.code, dy.rows, dy.cols, dy.ld, h.at, h.ld, kept ? &m : nullptr, w.at, w.code,
                                    static_cast<const float*>(s.at), dh.at, dh.ld, dx.data_ptr(), dy.cols, dw.data_ptr(),
                                    w.code, space.data_ptr(), need, here.stream);
    });
    if (st != ZERO_OK) return nullptr;
    return Py_BuildValue("(NN)", wrap(std::move(dx)), wrap(std::move(dw)));
  });
}

// embedding(tokens, table, scale, dtype or None)
PyObject* embedding(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plainly([&]() -> PyObject* {
    const Here here;
    Tokens t;
    Matrix table;
    zero_mx4 m;
    if (n != 4 || !t.read(a[0], here) || !PyFloat_Check(a[2])) return nullptr;
    const bool mx = (PyObject*)Py_TYPE(a[1]) == g_mx4;
    if (mx ? !read_mx(a[1], g_mx4, here, &m) : !table.read(a[1], here)) return nullptr;
    at::ScalarType type = mx ? at::kBFloat16 : table.t->scalar_type();
    if (a[3] != Py_None) {
      if (!THPDtype_Check(a[3])) return nullptr;
      type = ((THPDtype*)a[3])->scalar_type;
      if (code_of(type) < 0) return nullptr;
    }
    const int64_t vocab = mx ? m.rows : table.rows, cols = mx ? m.cols : table.cols;
    const double scale = PyFloat_AS_DOUBLE(a[2]);
    at::Tensor out;
    const zero_status st = unlocked([&] {
      out = here.empty({t.n, cols}, type);
      return zero_embedding(t.at, t.size, t.n, table.at, mx ? 0 : table.code, vocab, cols, table.ld, mx ? &m : nullptr, scale,
                            out.data_ptr(), code_of(type), cols, here.stream);
    });
    return st == ZERO_OK ? wrap(std::move(out)) : nullptr;
  });
}

// embedding_backward(dy, tokens, vocab, scale)
PyObject* embedding_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return plainly([&]() -> PyObject* {
    const Here here;
    Matrix dy;
    Tokens t;
    int64_t vocab, need = 0;
    if (n != 4 || !dy.read(a[0], here) || !t.read(a[1], here) || t.n != dy.rows || !whole(a[2], &vocab) || !PyFloat_Check(a[3]))
      return nullptr;
    if (zero_embedding_backward_workspace(t.n, vocab, dy.cols, &need) != ZERO_OK) return nullptr;
    const double scale = PyFloat_AS_DOUBLE(a[3]);
    const at::ScalarType type = dy.t->scalar_type();
    at::Tensor out;
    const zero_status st = unlocked([&] {
      out = here.empty({vocab, dy.cols}, type);
      at::Tensor space;
      if (need) space = here.empty({need}, at::kByte);  // (few tokens need none)
      return zero_embedding_backward(dy.at, dy.code, dy.rows, dy.cols, dy.ld, t.at, t.size, vocab, scale, out.data_ptr(),
                                     dy.code, dy.cols, 0, need ? space.data_ptr() : nullptr, need, here.stream);
    });
    return st == ZERO_OK ? wrap(std::move(out)) : nullptr;
  });
}

// bind(MX4, MX8): the package's classes
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2 || !PyType_Check(a[0]) || !PyType_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "two classes are needed");
    return nullptr;
  }
  Py_XSETREF(g_mx4, Py_NewRef(a[0]));
  Py_XSETREF(g_mx8, Py_NewRef(a[1]));
  Py_RETURN_NONE;
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(bind), CALL(mx8_quantize), CALL(mx8_dequantize), CALL(rms_norm), CALL(rms_norm_backward),
                         CALL(embedding), CALL(embedding_backward), {nullptr, nullptr, 0, nullptr}};
#undef CALL
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() {
  s_codes = PyUnicode_InternFromString("_codes"), s_scales = PyUnicode_InternFromString("_scales");
  s_space = PyUnicode_InternFromString("_space"), s_rows = PyUnicode_InternFromString("rows");
  s_cols = PyUnicode_InternFromString("cols"), s_device = PyUnicode_InternFromString("device");
  s_at = PyUnicode_InternFromString("_at"), s_struct = PyUnicode_InternFromString("_struct_");
  g_no_args = PyTuple_New(0);
  PyObject* m = PyModule_Create(&module);
  // (torch's C++ interface is its version's own)
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
