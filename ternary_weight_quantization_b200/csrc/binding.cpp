// The quick way through the Python binding: the checks of a call's tensors
// (type, shape, contiguity, device) and the C call itself in one step.
//
// Each function takes the arguments of the Python function of its name and
// returns the C call's status, or None, before anything is called, where an
// argument is not what the call takes; the Python function then goes through
// the arguments itself and says which one and why. A call checked tensor by
// tensor in Python and made through ctypes takes 8 to 15 us on the host, most
// of these operators' small calls less than that on the GPU (measured with
// norm_forward at 256 x 512: 10.3 us from Python, of which 2.6 us were the
// launch).
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/bitlinear.h"

namespace {

using at::ScalarType;

// Reads the arguments of one call; `ok` turns false at the first that does not
// fit.
struct Call {
  PyObject* const* args;
  int64_t device = -1;
  bool ok = true;

  explicit Call(PyObject* const* a) : args(a) {}

  bool none(int i) const { return args[i] == Py_None; }

  const at::Tensor* tensor(int i) {
    if (!ok || !THPVariable_Check(args[i])) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    if (!t.is_cuda() || t.layout() != at::kStrided || !t.is_contiguous()) {
      ok = false;
      return nullptr;
    }
    if (device < 0) device = c10::cuda::current_device();
    if (t.get_device() != device) {
      ok = false;
      return nullptr;
    }
    return &t;
  }

  // Address of the tensor at i, of this type and shape (None: null, where
  // `optional`).
  void* ptr(int i, ScalarType type, std::initializer_list<int64_t> shape, bool optional = false) {
    if (none(i)) {
      ok = ok && optional;
      return nullptr;
    }
    const at::Tensor* t = tensor(i);
    if (!t || t->scalar_type() != type || t->sizes() != at::IntArrayRef(shape)) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }

  // The workspace at i and its bytes.
  void* scratch(int i, size_t* bytes) {
    *bytes = 0;
    if (none(i)) return nullptr;
    const at::Tensor* t = tensor(i);
    if (!t) return nullptr;
    *bytes = t->nbytes();
    return t->data_ptr();
  }

  // Rows, columns and type (bf16 or fp32) of the tensor at i.
  ScalarType matrix(int i, int64_t* rows, int64_t* cols) {
    const at::Tensor* t = tensor(i);
    if (!t || t->dim() != 2 || (t->scalar_type() != at::kBFloat16 && t->scalar_type() != at::kFloat)) {
      ok = false;
      return at::kFloat;
    }
    *rows = t->size(0);
    *cols = t->size(1);
    return t->scalar_type();
  }

  // Type of the first tensor among these that is there (fp32 if none is).
  ScalarType first_type(std::initializer_list<int> which) {
    for (int i : which) {
      if (none(i)) continue;
      const at::Tensor* t = tensor(i);
      if (t && t->scalar_type() != at::kBFloat16 && t->scalar_type() != at::kFloat) ok = false;
      return t ? t->scalar_type() : at::kFloat;
    }
    return at::kFloat;
  }

  bool flag(int i) {
    const int v = PyObject_IsTrue(args[i]);
    if (v < 0) {
      PyErr_Clear();
      ok = false;
    }
    return v > 0;
  }

  float number(int i) {
    const double v = PyFloat_AsDouble(args[i]);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<float>(v);
  }

  // The call's stream: none given, the current one of the device. (A given
  // stream takes the Python way.)
  void* stream(int i) {
    if (!none(i)) ok = false;
    return ok ? static_cast<void*>(c10::cuda::getCurrentCUDAStream(device).stream()) : nullptr;
  }
};

bl_dtype code(ScalarType t) { return t == at::kFloat ? BL_F32 : BL_BF16; }
int64_t groups(int64_t K) { return (K + 127) / 128; }

// Runs `body`, which returns whether the arguments fit and, if so, sets the
// status; no C++ exception leaves.
template <int kArgs, typename F>
PyObject* run(PyObject* const* args, Py_ssize_t n, F body) {
  if (n != kArgs) Py_RETURN_NONE;
  bl_status status = BL_OK;
  bool made = false;
  try {
    Call c(args);
    made = body(c, &status);
  } catch (...) {
    made = false;
  }
  if (!made) Py_RETURN_NONE;
  return PyLong_FromLong(status);
}

#define BL_CALL(call)          \
  do {                         \
    if (!c.ok) return false;   \
    Py_BEGIN_ALLOW_THREADS     \
    *status = call;            \
    Py_END_ALLOW_THREADS       \
    return true;               \
  } while (0)

// h, W, targets, loss, lse, workspace, stream
PyObject* xent_forward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run<7>(args, n, [](Call& c, bl_status* status) {
    int64_t M = 0, K = 0, V = 0, K2 = 0;
    c.matrix(0, &M, &K);
    c.matrix(1, &V, &K2);
    void* h = c.ptr(0, at::kBFloat16, {M, K});
    void* W = c.ptr(1, at::kBFloat16, {V, K});
    auto* t = static_cast<int64_t*>(c.ptr(2, at::kLong, {M}));
    auto* loss = static_cast<float*>(c.ptr(3, at::kFloat, {M}));
    auto* lse = static_cast<float*>(c.ptr(4, at::kFloat, {M}));
    size_t bytes;
    void* ws = c.scratch(5, &bytes);
    void* st = c.stream(6);
    BL_CALL(bl_linear_xent_forward(h, W, t, M, V, K, loss, lse, ws, bytes, st));
  });
}

// h, W, targets, lse, dloss, dH, dW, workspace, accumulate_dW, stream
PyObject* xent_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run<10>(args, n, [](Call& c, bl_status* status) {
    int64_t M = 0, K = 0, V = 0, K2 = 0;
    c.matrix(0, &M, &K);
    c.matrix(1, &V, &K2);
    void* h = c.ptr(0, at::kBFloat16, {M, K});
    void* W = c.ptr(1, at::kBFloat16, {V, K});
    auto* t = static_cast<int64_t*>(c.ptr(2, at::kLong, {M}));
    auto* lse = static_cast<float*>(c.ptr(3, at::kFloat, {M}));
    auto* dloss = static_cast<float*>(c.ptr(4, at::kFloat, {M}));
    void* dH = c.ptr(5, at::kBFloat16, {M, K}, true);
    const ScalarType wt = c.none(6) ? at::kBFloat16 : c.first_type({6});
    void* dW = c.ptr(6, wt, {V, K}, true);
    size_t bytes;
    void* ws = c.scratch(7, &bytes);
    const int acc = c.flag(8);
    void* st = c.stream(9);
    BL_CALL(bl_linear_xent_backward(h, W, t, lse, dloss, M, V, K, dH, dW, code(wt), acc, ws, bytes, st));
  });
}

// x, codes, scales, stream
PyObject* act8_encode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run<4>(args, n, [](Call& c, bl_status* status) {
    int64_t M = 0, K = 0;
    const ScalarType xt = c.matrix(0, &M, &K);
    void* x = c.ptr(0, xt, {M, K});
    auto* codes = static_cast<int8_t*>(c.ptr(1, at::kChar, {M, K}));
    auto* scales = static_cast<float*>(c.ptr(2, at::kFloat, {M, groups(K)}));
    void* st = c.stream(3);
    BL_CALL(bl_act8_encode(x, code(xt), M, K, codes, scales, st));
  });
}

// codes, scales, x, stream
PyObject* act8_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run<4>(args, n, [](Call& c, bl_status* status) {
    int64_t M = 0, K = 0;
    const ScalarType xt = c.matrix(2, &M, &K);
    auto* codes = static_cast<int8_t*>(c.ptr(0, at::kChar, {M, K}));
    auto* scales = static_cast<float*>(c.ptr(1, at::kFloat, {M, groups(K)}));
    void* x = c.ptr(2, xt, {M, K});
    void* st = c.stream(3);
    BL_CALL(bl_act8_decode(codes, scales, M, K, x, code(xt), st));
  });
}

// x, weight, bias, eps, y, mean, rstd, rms, codes, scales, stream
PyObject* norm_forward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run<11>(args, n, [](Call& c, bl_status* status) {
    int64_t M = 0, K = 0;
    const ScalarType xt = c.matrix(0, &M, &K);
    const ScalarType pt = c.first_type({1, 2});
    void* x = c.ptr(0, xt, {M, K});
    void* w = c.ptr(1, pt, {K}, true);
    void* b = c.ptr(2, pt, {K}, true);
    const float eps = c.number(3);
    void* y = c.ptr(4, xt, {M, K});
    auto* mean = static_cast<float*>(c.ptr(5, at::kFloat, {M}, true));
    auto* rstd = static_cast<float*>(c.ptr(6, at::kFloat, {M}, true));
    const int rms = c.flag(7);
    auto* codes = static_cast<int8_t*>(c.ptr(8, at::kChar, {M, K}, true));
    auto* scales = static_cast<float*>(c.ptr(9, at::kFloat, {M, groups(K)}, true));
    void* st = c.stream(10);
    BL_CALL(bl_norm_forward(x, code(xt), w, b, code(pt), M, K, eps, rms, y, mean, rstd, codes, scales, st));
  });
}

// dy, x, codes, scales, weight, mean, rstd, dx, dweight, dbias, workspace, rms, accumulate, stream
PyObject* norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run<14>(args, n, [](Call& c, bl_status* status) {
    int64_t M = 0, K = 0;
    const ScalarType xt = c.matrix(0, &M, &K);
    const ScalarType pt = c.first_type({4, 8, 9});
    void* dy = c.ptr(0, xt, {M, K});
    void* x = c.ptr(1, xt, {M, K}, true);
    auto* codes = static_cast<int8_t*>(c.ptr(2, at::kChar, {M, K}, true));
    auto* scales = static_cast<float*>(c.ptr(3, at::kFloat, {M, groups(K)}, true));
    void* w = c.ptr(4, pt, {K}, true);
    auto* mean = static_cast<float*>(c.ptr(5, at::kFloat, {M}, true));
    auto* rstd = static_cast<float*>(c.ptr(6, at::kFloat, {M}, true));
    void* dx = c.ptr(7, xt, {M, K}, true);
    void* dw = c.ptr(8, pt, {K}, true);
    void* db = c.ptr(9, pt, {K}, true);
    size_t bytes;
    void* ws = c.scratch(10, &bytes);
    const int rms = c.flag(11), acc = c.flag(12);
    void* st = c.stream(13);
    BL_CALL(bl_norm_backward(dy, x, codes, scales, code(xt), w, code(pt), mean, rstd, M, K, rms, dx, dw, db, acc, ws,
                             bytes, st));
  });
}

// gate, up, y, gate codes, gate scales, up codes, up scales, stream
PyObject* swiglu_forward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run<8>(args, n, [](Call& c, bl_status* status) {
    int64_t M = 0, K = 0;
    const ScalarType xt = c.matrix(0, &M, &K);
    void* gate = c.ptr(0, xt, {M, K});
    void* up = c.ptr(1, xt, {M, K});
    void* y = c.ptr(2, xt, {M, K});
    auto* gc = static_cast<int8_t*>(c.ptr(3, at::kChar, {M, K}, true));
    auto* gs = static_cast<float*>(c.ptr(4, at::kFloat, {M, groups(K)}, true));
    auto* uc = static_cast<int8_t*>(c.ptr(5, at::kChar, {M, K}, true));
    auto* us = static_cast<float*>(c.ptr(6, at::kFloat, {M, groups(K)}, true));
    void* st = c.stream(7);
    BL_CALL(bl_swiglu_forward(gate, up, code(xt), M, K, y, gc, gs, uc, us, st));
  });
}

// dy, gate codes, gate scales, up codes, up scales, dgate, dup, stream
PyObject* swiglu_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return run<8>(args, n, [](Call& c, bl_status* status) {
    int64_t M = 0, K = 0;
    const ScalarType xt = c.matrix(0, &M, &K);
    void* dy = c.ptr(0, xt, {M, K});
    auto* gc = static_cast<int8_t*>(c.ptr(1, at::kChar, {M, K}));
    auto* gs = static_cast<float*>(c.ptr(2, at::kFloat, {M, groups(K)}));
    auto* uc = static_cast<int8_t*>(c.ptr(3, at::kChar, {M, K}));
    auto* us = static_cast<float*>(c.ptr(4, at::kFloat, {M, groups(K)}));
    void* dg = c.ptr(5, xt, {M, K});
    void* du = c.ptr(6, xt, {M, K});
    void* st = c.stream(7);
    BL_CALL(bl_swiglu_backward(dy, gc, gs, uc, us, code(xt), M, K, dg, du, st));
  });
}

#define BL_METHOD(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, nullptr }

PyMethodDef methods[] = {
    BL_METHOD(xent_forward), BL_METHOD(xent_backward), BL_METHOD(act8_encode),    BL_METHOD(act8_decode),
    BL_METHOD(norm_forward), BL_METHOD(norm_backward), BL_METHOD(swiglu_forward), BL_METHOD(swiglu_backward),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
