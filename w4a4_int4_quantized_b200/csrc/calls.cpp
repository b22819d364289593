// Argument marshalling of the calls whose kernels take a few microseconds (the
// norm, the gated activation and the int8 product): tensors in, one C ABI call
// out, as a CPython module.  What the interpreter needs for the same checks (a
// dozen attribute reads and a ctypes call of 15 arguments, 5 us) takes 0.3 us
// here.  Each function returns the library's status; shapes, element types,
// devices and strides that do not fit are refused with the same codes.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include "w4a4.h"

namespace {

decltype(&w8a8_add_rmsnorm_quantize) g_norm = nullptr;
decltype(&w8a8_silu_mul_quantize) g_silu = nullptr;
decltype(&w8a8_matmul) g_matmul = nullptr;

struct Mat {
  void* p = nullptr;
  int64_t ld = 0;
};

w4a4_dtype dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return W4A4_DTYPE_BF16;
    case at::kHalf: return W4A4_DTYPE_FP16;
    case at::kFloat: return W4A4_DTYPE_FP32;
    default: return static_cast<w4a4_dtype>(-1);   // refused by the library
  }
}

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool like(const at::Tensor& t, at::ScalarType type, int64_t dev) {
  return t.scalar_type() == type && t.is_cuda() && t.get_device() == dev;
}

// A matrix whose rows are contiguous.
int matrix(PyObject* o, int64_t rows, int64_t cols, at::ScalarType type, int64_t dev, Mat& m) {
  const at::Tensor* t = tensor(o);
  if (!t || !like(*t, type, dev)) return W4A4_ERR_INVALID_ARG;
  if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols || (t->stride(1) != 1 && cols != 1))
    return W4A4_ERR_UNSUPPORTED_SHAPE;
  m.p = t->data_ptr();
  m.ld = t->stride(0);
  return W4A4_OK;
}

int vector(PyObject* o, int64_t n, at::ScalarType type, int64_t dev, void** p) {
  const at::Tensor* t = tensor(o);
  if (!t || !like(*t, type, dev)) return W4A4_ERR_INVALID_ARG;
  if (t->dim() != 1 || t->size(0) != n || (t->stride(0) != 1 && n > 1)) return W4A4_ERR_UNSUPPORTED_SHAPE;
  *p = t->data_ptr();
  return W4A4_OK;
}

bool fits_int(int64_t v) { return v >= 0 && v <= 0x7FFFFFFF; }

// An int argument; what does not fit one is no shape that the library takes.
int integer(PyObject* o, int& v) {
  const long l = PyLong_AsLong(o);
  if (l == -1 && PyErr_Occurred()) return -1;
  if (!fits_int(l)) return W4A4_ERR_UNSUPPORTED_SHAPE;
  v = (int)l;
  return W4A4_OK;
}

// The interpreter lock let go for the library's call, as ctypes does: a launch waits
// where the stream's queue is full, and what it waits for may be a host function
// that needs the lock.
struct WithoutLock {
  PyThreadState* state = PyEval_SaveThread();
  ~WithoutLock() { PyEval_RestoreThread(state); }
};

// (X, gamma, eps, group, residual, H, Xq, x_scale, stream)
int norm(PyObject* const* a) {
  int group = 0, e;
  const double eps = PyFloat_AsDouble(a[2]);
  if ((eps == -1.0 && PyErr_Occurred()) || (e = integer(a[3], group)) < 0) return -1;
  if (e != 0) return e;
  const at::Tensor* X = tensor(a[0]);
  if (!X || X->dim() != 2 || !X->is_cuda()) return W4A4_ERR_INVALID_ARG;
  const int64_t M = X->size(0), K = X->size(1), dev = X->get_device();
  const at::ScalarType type = X->scalar_type();
  if (!fits_int(M) || !fits_int(K)) return W4A4_ERR_UNSUPPORTED_SHAPE;
  Mat x, r, h, q;
  void *g = nullptr, *s = nullptr;
  if ((e = matrix(a[0], M, K, type, dev, x)) != 0) return e;
  if (a[4] != Py_None && (e = matrix(a[4], M, K, type, dev, r)) != 0) return e;
  if (a[1] != Py_None && (e = vector(a[1], K, type, dev, &g)) != 0) return e;
  if (a[5] != Py_None && (e = matrix(a[5], M, K, type, dev, h)) != 0) return e;
  if ((e = matrix(a[6], M, K, at::kChar, dev, q)) != 0) return e;
  if ((e = vector(a[7], M, at::kFloat, dev, &s)) != 0) return e;
  const auto stream = static_cast<w4a4_stream_t>(PyLong_AsVoidPtr(a[8]));
  if (PyErr_Occurred()) return -1;
  const WithoutLock unlocked;
  return g_norm(x.p, x.ld, r.p, r.ld, g, (float)eps, (int)M, (int)K, group, dtype_of(*X), h.p, h.ld,
                static_cast<int8_t*>(q.p), q.ld, static_cast<float*>(s), stream);
}

// (gate, up, group, Xq, x_scale, stream)
int silu(PyObject* const* a) {
  int group = 0, e;
  if ((e = integer(a[2], group)) != 0) return e;
  const at::Tensor* G = tensor(a[0]);
  if (!G || G->dim() != 2 || !G->is_cuda()) return W4A4_ERR_INVALID_ARG;
  const int64_t M = G->size(0), K = G->size(1), dev = G->get_device();
  if (!fits_int(M) || !fits_int(K)) return W4A4_ERR_UNSUPPORTED_SHAPE;
  Mat g, u, q;
  void* s = nullptr;
  if ((e = matrix(a[0], M, K, G->scalar_type(), dev, g)) != 0) return e;
  if ((e = matrix(a[1], M, K, G->scalar_type(), dev, u)) != 0) return e;
  if ((e = matrix(a[3], M, K, at::kChar, dev, q)) != 0) return e;
  if ((e = vector(a[4], M, at::kFloat, dev, &s)) != 0) return e;
  const auto stream = static_cast<w4a4_stream_t>(PyLong_AsVoidPtr(a[5]));
  if (PyErr_Occurred()) return -1;
  const WithoutLock unlocked;
  return g_silu(g.p, g.ld, u.p, u.ld, (int)M, (int)K, group, dtype_of(*G), static_cast<int8_t*>(q.p), q.ld,
                static_cast<float*>(s), stream);
}

// (Xq, x_scale, Wq, w_scale, group, bias, Y, stream)
int matmul(PyObject* const* a) {
  int group = 0, e;
  if ((e = integer(a[4], group)) != 0) return e;
  const at::Tensor *X = tensor(a[0]), *W = tensor(a[2]), *Y = tensor(a[6]);
  if (!X || !W || !Y || X->dim() != 2 || W->dim() != 2 || !X->is_cuda()) return W4A4_ERR_INVALID_ARG;
  const int64_t M = X->size(0), K = X->size(1), N = W->size(0), dev = X->get_device();
  if (!fits_int(M) || !fits_int(K) || !fits_int(N)) return W4A4_ERR_UNSUPPORTED_SHAPE;
  const at::ScalarType type = Y->scalar_type();
  Mat x, w, y;
  void *sx = nullptr, *sw = nullptr, *b = nullptr;
  if ((e = matrix(a[0], M, K, at::kChar, dev, x)) != 0) return e;
  if ((e = matrix(a[2], N, K, at::kChar, dev, w)) != 0) return e;
  if ((e = vector(a[1], M, at::kFloat, dev, &sx)) != 0) return e;
  if ((e = vector(a[3], N, at::kFloat, dev, &sw)) != 0) return e;
  if (a[5] != Py_None && (e = vector(a[5], N, type, dev, &b)) != 0) return e;
  if ((e = matrix(a[6], M, N, type, dev, y)) != 0) return e;
  const auto stream = static_cast<w4a4_stream_t>(PyLong_AsVoidPtr(a[7]));
  if (PyErr_Occurred()) return -1;
  const WithoutLock unlocked;
  return g_matmul(static_cast<const int8_t*>(x.p), x.ld, static_cast<const float*>(sx),
                  static_cast<const int8_t*>(w.p), w.ld, static_cast<const float*>(sw), (int)M, (int)N, (int)K,
                  group, b, dtype_of(*Y), y.p, y.ld, stream);
}

template <int (*F)(PyObject* const*), Py_ssize_t ARGS>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != ARGS || !g_norm) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or the library is not bound");
    return nullptr;
  }
  try {
    const int status = F(args);
    return PyErr_Occurred() ? nullptr : PyLong_FromLong(status);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// The library's entry points, as addresses (it is loaded by the package).
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 3) {
    PyErr_SetString(PyExc_TypeError, "three addresses are wanted");
    return nullptr;
  }
  g_silu = reinterpret_cast<decltype(g_silu)>(PyLong_AsVoidPtr(args[1]));
  g_matmul = reinterpret_cast<decltype(g_matmul)>(PyLong_AsVoidPtr(args[2]));
  g_norm = reinterpret_cast<decltype(g_norm)>(PyLong_AsVoidPtr(args[0]));
  if (PyErr_Occurred()) return nullptr;
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {{"bind", FAST(bind), METH_FASTCALL, nullptr},
                         {"add_rmsnorm_quantize", FAST((call<norm, 9>)), METH_FASTCALL, nullptr},
                         {"silu_mul_quantize", FAST((call<silu, 6>)), METH_FASTCALL, nullptr},
                         {"matmul", FAST((call<matmul, 8>)), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
