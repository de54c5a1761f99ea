// The training operators' calls on torch tensors, without the interpreter.
//
// A small call's time is the host's: reading and checking each tensor's
// properties and allocating the outputs one by one from Python takes longer
// than the launches (a backward norm from 8 bits on 22 frames: 46 us a call, 13
// of them in the library; 17 from here).  These functions do the same in one step for the
// plain call - tensors of the right type, shape, device and layout, outputs to
// be allocated, the current stream - and return None for any other, which the
// Python functions then take on, or refuse with a message.  A non-zero status
// of the library comes back as an int.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <vector>

#include "fas.h"

namespace {

using at::Tensor;

// The library's functions, as the Python side has loaded them.
struct Api {
  decltype(&fas_backward) backward;
  decltype(&fas_residual_norm) norm;
  decltype(&fas_residual_norm_backward) norm_backward;
  decltype(&fas_residual_norm_backward_workspace) norm_workspace;
  decltype(&fas_checkpoint_pack) pack;
  decltype(&fas_checkpoint_unpack) unpack;
} api;

// What a call needs of its arguments; `ok` once falls and stays.
struct Args {
  bool ok = true;
  c10::DeviceIndex device;
  Args() : device(c10::cuda::current_device()) {}
  const Tensor* tensor(PyObject* o) {
    if (!ok || !THPVariable_Check(o)) return fail();
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided || t.unsafeGetTensorImpl()->is_python_dispatch() ||
        t.get_device() != device || !t.is_contiguous())
      return fail();
    return &t;
  }
  const Tensor* tensor(PyObject* o, at::ScalarType type, at::IntArrayRef shape) {
    const Tensor* t = tensor(o);
    return t && t->scalar_type() == type && t->sizes() == shape ? t : fail();
  }
  const Tensor* fail() {
    ok = false;
    return nullptr;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
};

Tensor empty(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}
PyObject* none() { Py_RETURN_NONE; }

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kCodes = at::kFloat8_e4m3fn, kByte = at::kByte;

template <class T = void>
T* ptr(const Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// A tuple of new tensors (undefined: None) or the status.
PyObject* results(int rc, std::initializer_list<const Tensor*> ts) {
  if (rc) return PyLong_FromLong(rc);
  PyObject* tuple = PyTuple_New((Py_ssize_t)ts.size());
  if (!tuple) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor* t : ts) {
    PyObject* o = t->defined() ? THPVariable_Wrap(*t) : none();
    if (!o) {
      Py_DECREF(tuple);
      return nullptr;
    }
    PyTuple_SET_ITEM(tuple, i++, o);
  }
  return tuple;
}

// The frames of a norm: gate [n, width] and their tokens.
struct Frames {
  const Tensor* gate = nullptr;
  std::vector<int32_t> spans;
  int n = 1;
  Frames(Args& a, PyObject* g, PyObject* tokens_of, int64_t tokens, int64_t width) {
    if (!a.ok || g == Py_None) return;
    gate = a.tensor(g);
    if (!gate || gate->dim() != 2 || gate->scalar_type() != kF32 || gate->size(1) != width || gate->size(0) < 1 ||
        gate->size(0) > INT32_MAX) {
      a.fail();
      return;
    }
    n = (int)gate->size(0);
    if (tokens_of == Py_None) {
      if (tokens % n) a.fail();
    } else if (PyLong_CheckExact(tokens_of)) {
      int over = 0;
      const int64_t span = PyLong_AsLongLongAndOverflow(tokens_of, &over);
      if (over || span < 1 || span > tokens || span * n != tokens) a.fail();
    } else if (PyList_CheckExact(tokens_of) || PyTuple_CheckExact(tokens_of)) {
      const Py_ssize_t len = PySequence_Fast_GET_SIZE(tokens_of);
      PyObject** items = PySequence_Fast_ITEMS(tokens_of);
      if (len != n) {
        a.fail();
        return;
      }
      spans.resize(len);
      int64_t sum = 0;
      for (Py_ssize_t i = 0; i < len; ++i) {
        int over = 0;
        const int64_t span = PyLong_CheckExact(items[i]) ? PyLong_AsLongLongAndOverflow(items[i], &over) : 0;
        if (over || span < 1 || span > tokens) {
          a.fail();
          return;
        }
        spans[i] = (int32_t)span;
        sum += span;
      }
      if (sum != tokens) a.fail();
    } else {
      a.fail();
    }
  }
  const int32_t* data() const { return spans.empty() ? nullptr : spans.data(); }
};

// A number argument; falls back for anything but a float or an int.
double number(Args& a, PyObject* o) {
  if (PyFloat_CheckExact(o)) return PyFloat_AS_DOUBLE(o);
  if (PyLong_CheckExact(o)) {
    const double d = PyLong_AsDouble(o);
    if (d == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      a.fail();
    }
    return d;
  }
  a.fail();
  return 0;
}

bool norm_size(const Tensor* x) {
  return x && x->dim() == 2 && x->size(0) >= 1 && x->size(0) <= INT32_MAX && x->size(1) >= 1 && x->size(1) <= INT32_MAX;
}

// (codes, scales) of a tensor of this shape.
struct Held {
  const Tensor *codes = nullptr, *scales = nullptr;
  Held(Args& a, PyObject* o, at::IntArrayRef shape) {
    if (!a.ok || !PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2 || shape.empty() ||
        shape.back() % FAS_CHECKPOINT_BLOCK) {
      a.fail();
      return;
    }
    codes = a.tensor(PyTuple_GET_ITEM(o, 0), kCodes, shape);
    std::vector<int64_t> s = shape.vec();
    s.back() /= FAS_CHECKPOINT_BLOCK;
    scales = a.tensor(PyTuple_GET_ITEM(o, 1), kByte, s);
  }
};
bool holdable(at::IntArrayRef shape, int64_t n) { return !shape.empty() && n > 0 && shape.back() % FAS_CHECKPOINT_BLOCK == 0; }
Tensor empty_scales(const Tensor& x) {
  std::vector<int64_t> s = x.sizes().vec();
  s.back() /= FAS_CHECKPOINT_BLOCK;
  return empty(s, kByte, x);
}

// checkpoint_pack(x) -> (codes, scales)
PyObject* checkpoint_pack(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a;
  const Tensor* x = n == 1 ? a.tensor(v[0]) : nullptr;
  if (!x || (x->scalar_type() != kBf16 && x->scalar_type() != kF32) || !holdable(x->sizes(), x->numel())) return none();
  Tensor codes, scales;
  int rc;
  {
    pybind11::gil_scoped_release free;
    codes = empty(x->sizes(), kCodes, *x);
    scales = empty_scales(*x);
    rc = api.pack(x->data_ptr(), x->scalar_type() == kF32, ptr<uint8_t>(&codes), ptr<uint8_t>(&scales), x->numel(),
                  a.stream());
  }
  return results(rc, {&codes, &scales});
  END_HANDLE_TH_ERRORS
}

// checkpoint_unpack((codes, scales), dtype or None) -> (x,)
PyObject* checkpoint_unpack(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a;
  if (n != 2 || !PyTuple_Check(v[0]) || PyTuple_GET_SIZE(v[0]) != 2) return none();
  const Tensor* codes = a.tensor(PyTuple_GET_ITEM(v[0], 0));
  at::ScalarType type = kBf16;
  if (v[1] != Py_None) {
    if (!THPDtype_Check(v[1])) return none();
    type = reinterpret_cast<THPDtype*>(v[1])->scalar_type;
  }
  if (!codes || (type != kBf16 && type != kF32) || !holdable(codes->sizes(), codes->numel())) return none();
  const Held held(a, v[0], codes->sizes());
  if (!a.ok) return none();
  Tensor x;
  int rc;
  {
    pybind11::gil_scoped_release free;
    x = empty(codes->sizes(), type, *codes);
    rc = api.unpack(ptr<uint8_t>(held.codes), ptr<uint8_t>(held.scales), x.data_ptr(), type == kF32, x.numel(), a.stream());
  }
  return results(rc, {&x});
  END_HANDLE_TH_ERRORS
}

// residual_norm(y, x, gamma_post, gamma_pre, gate, frame_tokens, alpha, eps, checkpoint)
// -> (x_out, h, rstd[, y codes, y scales, x codes, x scales])
PyObject* residual_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a;
  const Tensor* x = n == 9 ? a.tensor(v[1]) : nullptr;
  if (!norm_size(x) || (x->scalar_type() != kBf16 && x->scalar_type() != kF32)) return none();
  const int64_t N = x->size(0), C = x->size(1);
  const Tensor* y = a.tensor(v[0], kBf16, x->sizes());
  const Tensor *post = a.tensor(v[2], kF32, {C}), *pre = a.tensor(v[3], kF32, {C});
  const Frames frames(a, v[4], v[5], N, C);
  const float alpha = (float)number(a, v[6]), eps = (float)number(a, v[7]);
  const bool keep = v[8] == Py_True;
  if (!a.ok || (v[8] != Py_True && v[8] != Py_False) || (keep && !holdable(x->sizes(), x->numel()))) return none();
  Tensor xo, h, rstd, yc, ys, xc, xs;
  int rc;
  {
    pybind11::gil_scoped_release free;
    xo = empty(x->sizes(), x->scalar_type(), *x);
    h = empty(x->sizes(), kBf16, *x);
    rstd = empty({2, N}, kF32, *x);
    if (keep) {
      yc = empty(x->sizes(), kCodes, *x);
      ys = empty_scales(*x);
      xc = empty(x->sizes(), kCodes, *x);
      xs = empty_scales(*x);
    }
    rc = api.norm(y->data_ptr(), x->data_ptr(), x->scalar_type() == kF32, ptr<float>(frames.gate), ptr<float>(post),
                  ptr<float>(pre), alpha, eps, N, (int)C, frames.data(), frames.n, xo.data_ptr(), h.data_ptr(),
                  ptr<float>(&rstd), keep ? ptr<uint8_t>(&yc) : nullptr, keep ? ptr<uint8_t>(&ys) : nullptr,
                  keep ? ptr<uint8_t>(&xc) : nullptr, keep ? ptr<uint8_t>(&xs) : nullptr, a.stream());
  }
  return keep ? results(rc, {&xo, &h, &rstd, &yc, &ys, &xc, &xs}) : results(rc, {&xo, &h, &rstd});
  END_HANDLE_TH_ERRORS
}

// residual_norm_backward(dx_out, dh, y, x_out, rstd, gamma_post, gamma_pre, gate,
// frame_tokens, alpha) -> (dx, dy, dgamma_post, dgamma_pre, dgate)
PyObject* residual_norm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a;
  const Tensor* g = n == 10 ? a.tensor(v[0]) : nullptr;
  if (!norm_size(g) || (g->scalar_type() != kBf16 && g->scalar_type() != kF32)) return none();
  const int64_t N = g->size(0), C = g->size(1);
  const Tensor* dh = a.tensor(v[1], kBf16, g->sizes());
  const Tensor *y = nullptr, *x = nullptr, *yc = nullptr, *ys = nullptr, *xc = nullptr, *xs = nullptr;
  if (PyTuple_Check(v[2])) {
    const Held hy(a, v[2], g->sizes()), hx(a, v[3], g->sizes());
    yc = hy.codes;
    ys = hy.scales;
    xc = hx.codes;
    xs = hx.scales;
  } else {
    y = a.tensor(v[2], kBf16, g->sizes());
    x = a.tensor(v[3], g->scalar_type(), g->sizes());
  }
  const Tensor *rstd = a.tensor(v[4], kF32, {2, N}), *post = a.tensor(v[5], kF32, {C}), *pre = a.tensor(v[6], kF32, {C});
  const Frames frames(a, v[7], v[8], N, C);
  const float alpha = (float)number(a, v[9]);
  if (!a.ok) return none();
  Tensor dx, dy, dpost, dpre, dgate;
  int rc;
  {
    pybind11::gil_scoped_release free;
    int64_t bytes = 0;
    rc = api.norm_workspace(N, (int)C, frames.data(), frames.n, &bytes);
    if (!rc) {
      dx = empty(g->sizes(), g->scalar_type(), *g);
      dy = empty(g->sizes(), kBf16, *g);
      dpost = empty({C}, kF32, *g);
      dpre = empty({C}, kF32, *g);
      if (frames.gate) dgate = empty(frames.gate->sizes(), kF32, *g);
      const Tensor workspace = empty({bytes}, kByte, *g);
      rc = api.norm_backward(g->data_ptr(), dh->data_ptr(), ptr(y), ptr(x), g->scalar_type() == kF32, ptr<uint8_t>(yc),
                             ptr<uint8_t>(ys), ptr<uint8_t>(xc), ptr<uint8_t>(xs), ptr<float>(rstd),
                             ptr<float>(frames.gate), ptr<float>(post), ptr<float>(pre), alpha, N, (int)C, frames.data(),
                             frames.n, dx.data_ptr(), dy.data_ptr(), frames.gate ? ptr<float>(&dgate) : nullptr,
                             ptr<float>(&dpost), ptr<float>(&dpre), workspace.data_ptr(), bytes, a.stream());
    }
  }
  return results(rc, {&dx, &dy, &dpost, &dpre, &dgate});
  END_HANDLE_TH_ERRORS
}

// backward(q, k, v, out, lse, dout, shape, lse_shape, workspace bytes a row)
// -> (dq, dk, dv)
PyObject* backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Args a;
  if (n != 9 || !PyTuple_Check(v[6]) || !PyTuple_Check(v[7]) || PyTuple_GET_SIZE(v[6]) != 3 || PyTuple_GET_SIZE(v[7]) != 2)
    return none();
  int64_t s[3], l[2];
  for (int i = 0; i < 3; ++i) s[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v[6], i));
  for (int i = 0; i < 2; ++i) l[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(v[7], i));
  const int64_t row = PyLong_AsLongLong(v[8]);
  if (PyErr_Occurred()) return nullptr;
  const Tensor* t[6];
  for (int i = 0; i < 6; ++i) t[i] = i == 4 ? a.tensor(v[i], kF32, {l[0], l[1]}) : a.tensor(v[i], kBf16, {s[0], s[1], s[2]});
  if (!a.ok) return none();
  Tensor dq, dk, dv;
  int rc;
  {
    pybind11::gil_scoped_release free;
    dq = empty(t[0]->sizes(), kBf16, *t[0]);
    dk = empty(t[0]->sizes(), kBf16, *t[0]);
    dv = empty(t[0]->sizes(), kBf16, *t[0]);
    const Tensor workspace = empty({row * l[0] * l[1]}, kByte, *t[0]);
    rc = api.backward(t[0]->data_ptr(), t[1]->data_ptr(), t[2]->data_ptr(), t[3]->data_ptr(), ptr<float>(t[4]),
                      t[5]->data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), a.stream());
  }
  return results(rc, {&dq, &dk, &dv});
  END_HANDLE_TH_ERRORS
}

// bind(the addresses of the library's functions, in Api's order)
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
  void* p[6];
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) p[i] = PyLong_AsVoidPtr(v[i]);
  if (PyErr_Occurred()) return nullptr;
  api.backward = reinterpret_cast<decltype(api.backward)>(p[0]);
  api.norm = reinterpret_cast<decltype(api.norm)>(p[1]);
  api.norm_backward = reinterpret_cast<decltype(api.norm_backward)>(p[2]);
  api.norm_workspace = reinterpret_cast<decltype(api.norm_workspace)>(p[3]);
  api.pack = reinterpret_cast<decltype(api.pack)>(p[4]);
  api.unpack = reinterpret_cast<decltype(api.unpack)>(p[5]);
  return none();
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL(bind), CALL(checkpoint_pack), CALL(checkpoint_unpack), CALL(residual_norm),
                         CALL(residual_norm_backward), CALL(backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() { return PyModule_Create(&module); }
