// Python binding of the entry points around the routed experts
// (sparse_moe_routed_amd._block): argument checks and the call, nothing else.
//
// Every function takes the descriptor structs (ctypes), the arguments of the
// C function in its order -- each a torch tensor, an address or None -- and
// the stream's handle, and returns the status.  What a bare pointer cannot
// tell is checked on tensors: type (MOE_E_DTYPE), size and dense layout
// (MOE_E_SHAPE), memory of the current device (MOE_E_MEMORY).
//
// A small call is bound by its host time.  Through ctypes, with these checks
// in Python, norm_in of one row took 6.1 us a call and combine_norm of 8 rows
// 8.1 us; through here 4.4 and 4.8, the launch itself being 3.6.
#include <Python.h>
#include <hip/hip_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include "moe.h"

namespace {

PyTypeObject* g_shape_type = nullptr;   // ctypes structures of _abi.py
PyTypeObject* g_norm_type = nullptr;

at::ScalarType act_type(int32_t act) {
  if (act == MOE_DT_F32) return at::kFloat;
  return act == MOE_DT_BF16 ? at::kBFloat16 : at::ScalarType::Undefined;   // no tensor has it
}

typedef __int128 Count;   // no product of three int32 sizes wraps

// The arguments of one call: taken in order, the first fault kept.
class Args {
 public:
  Args(PyObject* const* a, Py_ssize_t n) : a_(a), n_(n) {}
  ~Args() {
    for (int i = 0; i < views_; ++i) PyBuffer_Release(&view_[i]);
  }
  const moe_shape* shape() { return static_cast<const moe_shape*>(structure(g_shape_type)); }
  const moe_norm* norm() { return static_cast<const moe_norm*>(structure(g_norm_type)); }

  // address of a tensor of `count` elements
  void* tensor(at::ScalarType type, Count count) {
    return address(next(), [&](const at::Tensor& t) {
      if (t.scalar_type() != type) return MOE_E_DTYPE;
      return t.numel() == count && t.is_contiguous() ? MOE_OK : MOE_E_SHAPE;
    });
  }
  // a workspace and its size, the last two arguments of the C functions that take one
  void* workspace(size_t* bytes) {
    PyObject* o = next();
    PyObject* size = next();
    *bytes = size ? PyLong_AsSize_t(size) : 0;
    if (PyErr_Occurred()) return nullptr;
    return address(o, [&](const at::Tensor& t) {
      return t.is_contiguous() && t.nbytes() >= *bytes ? MOE_OK : MOE_E_WORKSPACE;
    });
  }
  hipStream_t stream() {
    PyObject* o = next();
    return o ? static_cast<hipStream_t>(PyLong_AsVoidPtr(o)) : nullptr;
  }

  // the status of the call `f`, made if nothing was wrong
  template <typename F>
  PyObject* call(F f) {
    if (!PyErr_Occurred() && i_ != n_) PyErr_SetString(PyExc_TypeError, "too many arguments");
    if (PyErr_Occurred()) return nullptr;
    int st = status_ ? status_ : memory_;
    if (!st) {
      Py_BEGIN_ALLOW_THREADS
      st = f();
      Py_END_ALLOW_THREADS
    }
    return PyLong_FromLong(st);
  }

 private:
  // the next argument; null once something has raised
  PyObject* next() {
    if (PyErr_Occurred()) return nullptr;
    if (i_ < n_) return a_[i_++];
    PyErr_SetString(PyExc_TypeError, "too few arguments");
    return nullptr;
  }
  // A tensor's address is taken only if nothing was wrong so far; a fault of
  // its memory is reported after every other one.
  template <typename Check>
  void* address(PyObject* o, Check check) {
    if (!o || o == Py_None) return nullptr;
    if (PyLong_Check(o)) return PyLong_AsVoidPtr(o);
    if (!THPVariable_Check(o)) {
      PyErr_SetString(PyExc_TypeError, "expected a tensor, an address or None");
      return nullptr;
    }
    try {   // a tensor without plain storage throws
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!status_) status_ = check(t);
      if (t.is_cuda()) {
        if (device_ < 0 && hipGetDevice(&device_) != hipSuccess) device_ = -1;
        if (t.get_device() != device_) memory_ = MOE_E_MEMORY;
        return status_ || memory_ ? nullptr : t.data_ptr();
      }
    } catch (const std::exception& e) {
      PyErr_SetString(PyExc_RuntimeError, e.what());
      return nullptr;
    }
    memory_ = MOE_E_MEMORY;
    return nullptr;
  }
  const void* structure(PyTypeObject* type) {
    static const char zeros[64] = {};   // read in place of a struct that is not there
    PyObject* o = next();
    if (!o) return zeros;
    if (!type || !PyObject_TypeCheck(o, type) || PyObject_GetBuffer(o, &view_[views_], PyBUF_SIMPLE)) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "expected a moe_shape / moe_norm");
      return zeros;
    }
    return view_[views_++].buf;
  }
  PyObject* const* a_;
  Py_ssize_t n_, i_ = 0;
  Py_buffer view_[2];
  int views_ = 0;
  int status_ = 0, memory_ = 0, device_ = -1;
};

Count elements(const moe_norm* n) { return static_cast<Count>(n->T) * n->H; }
Count tokens(const moe_shape* s) { return static_cast<Count>(s->T) * s->H; }
Count pairs(const moe_shape* s) { return static_cast<Count>(s->T) * s->top_k; }

void* gate(Args& a, const moe_norm* n) {
  return n->flags & MOE_N_GATE_TOKEN ? a.tensor(at::kFloat, n->T)
                                     : a.tensor(act_type(n->act), elements(n));
}

PyObject* norm_in(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a(argv, argc);
  const moe_norm* n = a.norm();
  const at::ScalarType t = act_type(n->act);
  const Count m = elements(n);
  void* x = a.tensor(t, m);
  void* w = a.tensor(t, n->H);
  void* out = a.tensor(t, m);
  hipStream_t st = a.stream();
  return a.call([&] { return moe_norm_in(n, x, w, out, st); });
}

PyObject* norm_in_backward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a(argv, argc);
  const moe_norm* n = a.norm();
  const at::ScalarType t = act_type(n->act);
  const Count m = elements(n);
  void* dn = a.tensor(t, m);
  void* x = a.tensor(t, m);
  void* w = a.tensor(t, n->H);
  void* dres = a.tensor(t, m);
  void* dx = a.tensor(t, m);
  float* dw = static_cast<float*>(a.tensor(at::kFloat, n->H));
  size_t bytes;
  void* ws = a.workspace(&bytes);
  hipStream_t st = a.stream();
  return a.call([&] { return moe_norm_in_backward(n, dn, x, w, dres, dx, dw, ws, bytes, st); });
}

PyObject* norm_out(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a(argv, argc);
  const moe_norm* n = a.norm();
  const at::ScalarType t = act_type(n->act);
  const Count m = elements(n);
  void* z = a.tensor(t, m);
  void* w = a.tensor(t, n->H);
  void* g = gate(a, n);
  void* res = a.tensor(t, m);
  void* w_next = a.tensor(t, n->H);
  void* out = a.tensor(t, m);
  void* n_next = a.tensor(t, m);
  hipStream_t st = a.stream();
  return a.call([&] { return moe_norm_out(n, z, w, g, res, w_next, out, n_next, st); });
}

PyObject* norm_out_backward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a(argv, argc);
  const moe_norm* n = a.norm();
  const at::ScalarType t = act_type(n->act);
  const Count m = elements(n);
  void* dout = a.tensor(t, m);
  void* z = a.tensor(t, m);
  void* w = a.tensor(t, n->H);
  void* g = gate(a, n);
  void* dz = a.tensor(t, m);
  void* dgate = gate(a, n);
  float* dw = static_cast<float*>(a.tensor(at::kFloat, n->H));
  size_t bytes;
  void* ws = a.workspace(&bytes);
  hipStream_t st = a.stream();
  return a.call([&] { return moe_norm_out_backward(n, dout, z, w, g, dz, dgate, dw, ws, bytes, st); });
}

PyObject* combine_norm(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a(argv, argc);
  const moe_shape* s = a.shape();
  const moe_norm* n = a.norm();
  const at::ScalarType t = act_type(n->act);
  const Count m = elements(n), P = pairs(s);
  void* y = a.tensor(t, P * s->H);
  const int32_t* pair_row = static_cast<int32_t*>(a.tensor(at::kInt, P));
  const float* topk_w = static_cast<float*>(a.tensor(at::kFloat, P));
  void* w = a.tensor(t, n->H);
  void* g = gate(a, n);
  void* res = a.tensor(t, m);
  void* w_next = a.tensor(t, n->H);
  void* z = a.tensor(t, m);
  void* out = a.tensor(t, m);
  void* n_next = a.tensor(t, m);
  hipStream_t st = a.stream();
  return a.call([&] {
    return moe_combine_norm(s, n, y, pair_row, topk_w, w, g, res, w_next, z, out, n_next, st);
  });
}

PyObject* dispatch(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a(argv, argc);
  const moe_shape* s = a.shape();
  const at::ScalarType t = act_type(s->act);
  const Count P = pairs(s);
  void* x = a.tensor(t, tokens(s));
  const int32_t* pair_row = static_cast<int32_t*>(a.tensor(at::kInt, P));
  const float* w = static_cast<float*>(a.tensor(at::kFloat, P));
  void* rows = a.tensor(t, P * s->H);
  hipStream_t st = a.stream();
  return a.call([&] { return moe_dispatch(s, x, pair_row, w, rows, st); });
}

PyObject* dispatch_backward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a(argv, argc);
  const moe_shape* s = a.shape();
  const at::ScalarType t = act_type(s->act);
  const Count P = pairs(s), m = tokens(s);
  void* drows = a.tensor(t, P * s->H);
  const int32_t* pair_row = static_cast<int32_t*>(a.tensor(at::kInt, P));
  const float* w = static_cast<float*>(a.tensor(at::kFloat, P));
  void* x = a.tensor(t, m);
  void* dx_in = a.tensor(t, m);
  void* dx = a.tensor(t, m);
  float* dw = static_cast<float*>(a.tensor(at::kFloat, P));
  hipStream_t st = a.stream();
  return a.call([&] { return moe_dispatch_backward(s, drows, pair_row, w, x, dx_in, dx, dw, st); });
}

PyObject* combine_backward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a(argv, argc);
  const moe_shape* s = a.shape();
  const at::ScalarType t = act_type(s->act);
  const Count P = pairs(s);
  void* dout = a.tensor(t, tokens(s));
  void* y = a.tensor(t, P * s->H);
  const int32_t* pair_row = static_cast<int32_t*>(a.tensor(at::kInt, P));
  const float* w = static_cast<float*>(a.tensor(at::kFloat, P));
  void* dy = a.tensor(t, P * s->H);
  float* dw = static_cast<float*>(a.tensor(at::kFloat, P));
  hipStream_t st = a.stream();
  return a.call([&] { return moe_combine_backward(s, dout, y, pair_row, w, dy, dw, st); });
}

PyObject* route_backward(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a(argv, argc);
  const moe_shape* s = a.shape();
  const Count P = pairs(s);
  const int32_t* ids = static_cast<int32_t*>(a.tensor(at::kInt, P));
  const float* w = static_cast<float*>(a.tensor(at::kFloat, P));
  const float* dw = static_cast<float*>(a.tensor(at::kFloat, P));
  float* dlogits = static_cast<float*>(a.tensor(at::kFloat, static_cast<Count>(s->T) * s->E));
  hipStream_t st = a.stream();
  return a.call([&] { return moe_route_backward(s, ids, w, dw, dlogits, st); });
}

// The ctypes classes of moe_shape and moe_norm, once at import.
PyObject* set_types(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  if (argc != 2 || !PyType_Check(argv[0]) || !PyType_Check(argv[1])) {
    PyErr_SetString(PyExc_TypeError, "expected the moe_shape and moe_norm classes");
    return nullptr;
  }
  Py_INCREF(argv[0]);
  Py_INCREF(argv[1]);
  g_shape_type = reinterpret_cast<PyTypeObject*>(argv[0]);
  g_norm_type = reinterpret_cast<PyTypeObject*>(argv[1]);
  Py_RETURN_NONE;
}

typedef PyObject* (*Fast)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction fast(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef g_methods[] = {
    {"moe_norm_in", fast(norm_in), METH_FASTCALL, nullptr},
    {"moe_norm_in_backward", fast(norm_in_backward), METH_FASTCALL, nullptr},
    {"moe_norm_out", fast(norm_out), METH_FASTCALL, nullptr},
    {"moe_norm_out_backward", fast(norm_out_backward), METH_FASTCALL, nullptr},
    {"moe_combine_norm", fast(combine_norm), METH_FASTCALL, nullptr},
    {"moe_dispatch", fast(dispatch), METH_FASTCALL, nullptr},
    {"moe_dispatch_backward", fast(dispatch_backward), METH_FASTCALL, nullptr},
    {"moe_combine_backward", fast(combine_backward), METH_FASTCALL, nullptr},
    {"moe_route_backward", fast(route_backward), METH_FASTCALL, nullptr},
    {"set_types", fast(set_types), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&g_module); }
