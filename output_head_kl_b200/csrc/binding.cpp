// Argument marshalling of the latency-bound calls (RMS norm, linear layer) for the Python binding.
//
// A call on one token takes the GPU 2 to 10 us; checking its tensors and building its argument list in Python
// took 4 to 5 us on top of the launch.  These functions do both for the ordinary case: every tensor has the type,
// shape, layout and device that the call expects.  In any other case they return None, and the caller's
// Python path checks again, step by step, and raises with the reason.  The addresses of the C entry points are
// passed in, so that the same code serves every build of the library.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kdkl.h"

namespace {

using at::ScalarType;

using NormForward = decltype(&kdkl_rmsnorm_forward);
using NormBackward = decltype(&kdkl_rmsnorm_backward);
using LinearForward = decltype(&kdkl_linear_forward);
using LinearBackward = decltype(&kdkl_linear_backward);

constexpr unsigned kBf = 1, kF32 = 2, kF8 = 4;

unsigned type_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case ScalarType::BFloat16: return kBf;
    case ScalarType::Float: return kF32;
    case ScalarType::Float8_e4m3fn: return kF8;
    default: return 0;
  }
}

int32_t dtype_code(unsigned type) { return type == kF32 ? KDKL_F32 : (type == kF8 ? KDKL_E4M3 : KDKL_BF16); }

// The arguments of one call; `good` turns false at the first that the fast path does not take.
struct Args {
  PyObject* const* v;
  bool good = true;
  int dev = -1;

  const at::Tensor* tensor(int i) {   // null for None
    if (v[i] == Py_None) return nullptr;
    if (!THPVariable_Check(v[i])) {
      good = false;
      return nullptr;
    }
    return &THPVariable_Unpack(v[i]);
  }
  // The tensor that fixes the call's device: two dimensions, on the current device.
  const at::Tensor* lead(int i) {
    const at::Tensor* t = tensor(i);
    if (!t || t->dim() != 2 || !t->is_cuda()) {
      good = false;
      return nullptr;
    }
    dev = t->get_device();
    if (dev != c10::cuda::current_device()) good = false;
    return t;
  }
  bool dense(const at::Tensor& t, unsigned types) {
    if (!t.is_cuda() || t.get_device() != dev || !(type_of(t) & types) || !t.is_contiguous()) good = false;
    return good;
  }
  template <class T = void>
  T* matrix(int i, int64_t rows, int64_t cols, unsigned types) {
    const at::Tensor* t = tensor(i);
    if (!t || !good || !dense(*t, types)) return nullptr;
    if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols) {
      good = false;
      return nullptr;
    }
    return static_cast<T*>(t->data_ptr());
  }
  template <class T = void>
  T* vector(int i, int64_t n, unsigned types) {
    const at::Tensor* t = tensor(i);
    if (!t || !good || !dense(*t, types)) return nullptr;
    if (t->dim() != 1 || t->size(0) != n) {
      good = false;
      return nullptr;
    }
    return static_cast<T*>(t->data_ptr());
  }
  void* workspace(int i, size_t* bytes) {
    const at::Tensor* t = tensor(i);
    if (!t || !good || !t->is_cuda() || t->get_device() != dev || !t->is_contiguous()) {
      good = false;
      return nullptr;
    }
    *bytes = t->nbytes();
    return t->data_ptr();
  }
  int32_t integer(int i) {
    const long x = PyLong_Check(v[i]) ? PyLong_AsLong(v[i]) : 0;
    if (!PyLong_Check(v[i]) || x < INT32_MIN || x > INT32_MAX) good = false;
    return static_cast<int32_t>(x);
  }
  float real(int i) {
    if (!PyFloat_Check(v[i])) good = false;
    return good ? static_cast<float>(PyFloat_AS_DOUBLE(v[i])) : 0.f;
  }
  void* address(int i) {
    if (!PyLong_Check(v[i])) good = false;
    return good ? PyLong_AsVoidPtr(v[i]) : nullptr;
  }
  // a stream's handle (0 is the legacy default stream), or the current stream for None
  void* stream(int i) {
    if (v[i] == Py_None) return good ? static_cast<void*>(c10::cuda::getCurrentCUDAStream(dev).stream()) : nullptr;
    return address(i);
  }
};

template <class F>
PyObject* guarded(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, F&& call) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  long status = -1;
  try {
    Args a{args};
    status = call(a);
  } catch (...) {
    status = -1;   // the Python path meets the same error and reports it
  }
  if (PyErr_Occurred()) PyErr_Clear();
  if (status < 0) Py_RETURN_NONE;
  return PyLong_FromLong(status);
}

// The library is called without the interpreter's lock, as ctypes calls it: a launch may wait for the queue.
template <class F>
long unlocked(F&& f) {
  long st;
  Py_BEGIN_ALLOW_THREADS;
  st = static_cast<long>(f());
  Py_END_ALLOW_THREADS;
  return st;
}

// (address, x, gamma, y, residual, h, y_scale, eps, stream)
PyObject* rmsnorm_forward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 9, [](Args& a) -> long {
    const at::Tensor* x = a.lead(1);
    const at::Tensor *g = a.tensor(2), *y = a.tensor(3), *r = a.tensor(4), *h = a.tensor(5);
    if (!a.good || !g || !y) return -1;
    const int64_t N = x->size(0), d = x->size(1);
    if (d > INT32_MAX) return -1;
    const unsigned ht = r ? type_of(*r) : (h ? type_of(*h) : type_of(*x));
    const void* px = a.matrix(1, N, d, kBf | kF32);
    const void* pg = a.vector(2, d, kBf | kF32);
    void* py = a.matrix(3, N, d, kBf | kF8);
    const void* pr = a.matrix(4, N, d, kBf | kF32);
    void* ph = a.matrix(5, N, d, ht & (kBf | kF32));
    float* ps = a.vector<float>(6, N, kF32);
    const float eps = a.real(7);
    void* s = a.stream(8);
    const auto fn = reinterpret_cast<NormForward>(a.address(0));
    if (!a.good) return -1;
    const int32_t xt = dtype_code(type_of(*x)), hc = dtype_code(ht), gt = dtype_code(type_of(*g)),
                  yt = dtype_code(type_of(*y));
    return unlocked([&] { return fn(px, pr, pg, N, static_cast<int32_t>(d), eps, xt, hc, gt, yt, ph, py, ps, s); });
  });
}

// (address, dy, h, gamma, dx, dgamma, workspace, dh, eps, stream)
PyObject* rmsnorm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 10, [](Args& a) -> long {
    const at::Tensor* h = a.lead(2);
    const at::Tensor* g = a.tensor(3);
    if (!a.good || !g || !a.tensor(1) || !a.tensor(4) || !a.tensor(5)) return -1;
    const int64_t N = h->size(0), d = h->size(1);
    if (d > INT32_MAX) return -1;
    const unsigned ht = type_of(*h);
    const void* pdy = a.matrix(1, N, d, kBf);
    const void* ph = a.matrix(2, N, d, kBf | kF32);
    const void* pg = a.vector(3, d, kBf | kF32);
    void* pdx = a.matrix(4, N, d, ht);
    float* pdg = a.vector<float>(5, d, kF32);
    size_t wsb = 0;
    void* ws = a.workspace(6, &wsb);
    const void* pdh = a.matrix(7, N, d, ht);
    const float eps = a.real(8);
    void* s = a.stream(9);
    const auto fn = reinterpret_cast<NormBackward>(a.address(0));
    if (!a.good) return -1;
    const int32_t hc = dtype_code(ht), gt = dtype_code(type_of(*g));
    return unlocked(
        [&] { return fn(pdy, ph, pg, pdh, N, static_cast<int32_t>(d), eps, hc, gt, pdx, pdg, ws, wsb, s); });
  });
}

// (address, x, W, y, workspace, bias, residual, pre, activation, x_scale, w_scale, plan, stream)
PyObject* linear_forward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 13, [](Args& a) -> long {
    const at::Tensor* x = a.lead(1);
    const at::Tensor* W = a.tensor(2);
    if (!a.good || !W || W->dim() != 2 || !a.tensor(3)) return -1;
    const int64_t M = x->size(0), k = x->size(1), o = W->size(0);
    if (k > INT32_MAX || o > INT32_MAX) return -1;
    const unsigned xt = type_of(*x);
    kdkl_linear_options opt{};
    const void* px = a.matrix(1, M, k, kBf | kF8);
    const void* pW = a.matrix(2, o, k, xt);
    void* py = a.matrix(3, M, o, kBf);
    size_t wsb = 0;
    void* ws = a.workspace(4, &wsb);
    const void* pb = a.vector(5, o, kBf);
    const void* pr = a.matrix(6, M, o, kBf);
    void* pp = a.matrix(7, M, o, kBf);
    opt.operands = xt == kF8 ? KDKL_E4M3 : KDKL_BF16;
    opt.activation = a.integer(8);
    opt.x_scale = a.vector<float>(9, M, kF32);
    opt.w_scale = a.vector<float>(10, o, kF32);
    opt.plan = a.integer(11);
    void* s = a.stream(12);
    const auto fn = reinterpret_cast<LinearForward>(a.address(0));
    if (!a.good) return -1;
    return unlocked([&] {
      return fn(px, pW, pb, pr, M, static_cast<int32_t>(k), static_cast<int32_t>(o), &opt, py, pp, ws, wsb, s);
    });
  });
}

// (address, dy, x, W, dx, dW, workspace, pre, dbias, activation, dx_plan, dw_plan, stream)
PyObject* linear_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 13, [](Args& a) -> long {
    const at::Tensor* dy = a.lead(1);
    const at::Tensor *x = a.tensor(2), *W = a.tensor(3);
    if (!a.good || (!x && !W)) return -1;
    const int64_t M = dy->size(0), o = dy->size(1);
    const at::Tensor* wide = W ? W : x;
    if (wide->dim() != 2) return -1;
    const int64_t k = wide->size(1);
    if (k > INT32_MAX || o > INT32_MAX) return -1;
    kdkl_linear_options opt{};
    const void* pdy = a.matrix(1, M, o, kBf);
    const void* px = a.matrix(2, M, k, kBf);
    const void* pW = a.matrix(3, o, k, kBf);
    void* pdx = a.matrix(4, M, k, kBf);
    void* pdW = a.matrix(5, o, k, kBf);
    size_t wsb = 0;
    void* ws = a.workspace(6, &wsb);
    const void* pp = a.matrix(7, M, o, kBf);
    float* pb = a.vector<float>(8, o, kF32);
    opt.operands = KDKL_BF16;
    opt.activation = a.integer(9);
    opt.dx_plan = a.integer(10);
    opt.dw_plan = a.integer(11);
    void* s = a.stream(12);
    const auto fn = reinterpret_cast<LinearBackward>(a.address(0));
    if (!a.good) return -1;
    return unlocked([&] {
      return fn(pdy, pp, px, pW, M, static_cast<int32_t>(k), static_cast<int32_t>(o), &opt, pdx, pdW, pb, ws, wsb, s);
    });
  });
}

PyMethodDef methods[] = {
    {"rmsnorm_forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rmsnorm_forward)), METH_FASTCALL, nullptr},
    {"rmsnorm_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rmsnorm_backward)), METH_FASTCALL, nullptr},
    {"linear_forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_forward)), METH_FASTCALL, nullptr},
    {"linear_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_backward)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "kdkl_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit_kdkl_binding() { return PyModule_Create(&module); }
