// The host side of the operators' calls in one step: the checks of operators.py
// that pass for the tensors the parameters were made for, and the call of the
// library's entry point.  Anything else (other tensors, another device, a
// gradient, an explicit stream, a tensor without storage of its own, whose
// accessors throw) is left to the Python checks, which either take the call or say
// what is wrong with it; so this file raises no error of its own, and no C++
// exception leaves it: that would end the process.
//
// A call of an operator on a few rows lasts 2 to 5 us on the GPU; the Python
// checks and ctypes take 12 us on the host, this about 1.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <memory>
#include <vector>

#include "sparsepr.h"

namespace {

// A tensor as the parameters were made for it, or as its fields ask for.
struct Want {
  bool given = false;
  at::ScalarType type = at::kFloat;
  std::vector<int64_t> sizes, strides;  // strides empty: contiguous
};

struct Plan {
  enum Kind { NORM_ROTATE, MASKED, PROJECT } kind;
  std::vector<uint8_t> bytes;  // the parameters when the plan was made
  void* fn;                    // the library's entry point
  std::vector<Want> main;      // the tensors made for, in the order of the call
};

constexpr const char* NAME = "sparsepr.plan";

void destroy(PyObject* capsule) {
  delete static_cast<Plan*>(PyCapsule_GetPointer(capsule, NAME));
}

bool to_want(PyObject* o, Want* w) {
  if (o == Py_None) return true;
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  w->given = true;
  w->type = t.scalar_type();
  w->sizes = t.sizes().vec();
  w->strides = t.strides().vec();
  return true;
}

// plan(kind, address of the parameters, their size, address of the entry point, tensors made for)
PyObject* make_plan(PyObject* args) {
  int kind;
  unsigned long long prm, fn;
  Py_ssize_t size;
  PyObject* tensors;
  if (!PyArg_ParseTuple(args, "iKnKO!", &kind, &prm, &size, &fn, &PyTuple_Type, &tensors))
    return nullptr;
  auto p = std::make_unique<Plan>();
  p->kind = static_cast<Plan::Kind>(kind);
  const auto* now = reinterpret_cast<const uint8_t*>(prm);
  p->bytes.assign(now, now + size);
  p->fn = reinterpret_cast<void*>(fn);
  p->main.resize(PyTuple_GET_SIZE(tensors));
  for (size_t i = 0; i < p->main.size(); ++i)
    if (!to_want(PyTuple_GET_ITEM(tensors, i), &p->main[i])) Py_RETURN_NONE;
  return PyCapsule_New(p.release(), NAME, destroy);
}

// The tensors of one call, checked one after the other; ok is false after the first misfit.
struct Call {
  bool ok = true, grad = c10::GradMode::is_enabled();
  int device = -1;

  const at::Tensor* tensor(PyObject* o) {
    if (!THPVariable_CheckExact(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    // (a tangent counts under no_grad too: only reverse mode is off there)
    if (!t.is_cuda() || (grad && t.requires_grad()) || t._fw_grad(0).defined()) return fail();
    const int d = t.get_device();
    if (device < 0) device = d;
    return d == device ? &t : fail();
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
  void* main(PyObject* o, const Want& w) {
    if (!w.given) {
      if (o != Py_None) fail();
      return nullptr;
    }
    const at::Tensor* t = tensor(o);
    if (!t || t->scalar_type() != w.type || t->sizes() != at::IntArrayRef(w.sizes) ||
        t->strides() != at::IntArrayRef(w.strides)) {
      fail();
      return nullptr;
    }
    return t->data_ptr();
  }
  const at::Tensor* workspace(PyObject* o) {
    const at::Tensor* t = tensor(o);
    return t && t->is_contiguous() ? t : fail();
  }
  void* aux(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> sizes) {
    if (o == Py_None) return nullptr;
    const at::Tensor* t = tensor(o);
    if (!t || t->scalar_type() != type || t->sizes() != at::IntArrayRef(sizes) ||
        !t->is_contiguous()) {
      fail();
      return nullptr;
    }
    return t->data_ptr();
  }
};

// call(plan, address of the parameters, *tensors in the order of the Python function,
// stream): the library's status, or -1 where the call is left to the Python checks.
PyObject* make_call(PyObject* const* a, Py_ssize_t n) {
  auto* p = n > 1 ? static_cast<Plan*>(PyCapsule_GetPointer(a[0], NAME)) : nullptr;
  if (!p) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  const void* now = PyLong_AsVoidPtr(a[1]);
  if (!now) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "parameters without an address");
    return nullptr;
  }
  ++a;  // a[1], a[2] .. are the tensors from here on
  --n;
  const Py_ssize_t want = p->kind == Plan::NORM_ROTATE ? 13 : p->kind == Plan::MASKED ? 14 : 10;
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  if (a[n - 1] != Py_None || memcmp(p->bytes.data(), now, p->bytes.size()))
    return PyLong_FromLong(-1);
  Call c;
  const auto i32 = at::kInt;
  int status = -1;
  auto stream = [&]() -> void* {
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream();
  };
  auto here = [&] { return c.ok && c.device == static_cast<int>(c10::cuda::current_device()); };
  if (p->kind == Plan::NORM_ROTATE) {
    const auto& m = *static_cast<const spr_norm_rotate_params*>(now);
    void* t[4];
    for (int i = 0; i < 4; ++i) t[i] = c.main(a[1 + i], p->main[i]);
    if (!m.Hk && (a[6] != Py_None || a[10] != Py_None)) return PyLong_FromLong(-1);
    if (m.rot && (a[7] == Py_None || a[8] == Py_None)) return PyLong_FromLong(-1);
    const auto type = p->main[0].type;
    void *wq = c.aux(a[5], type, {m.d}), *wk = c.aux(a[6], type, {m.d});
    int64_t rows = 0;
    float *cos = nullptr, *sin = nullptr;
    if (m.rot) {
      if (!THPVariable_CheckExact(a[7])) return PyLong_FromLong(-1);
      const at::Tensor& t0 = THPVariable_Unpack(a[7]);
      if (t0.dim() != 2 || t0.size(0) > INT32_MAX) return PyLong_FromLong(-1);
      rows = t0.size(0);
      cos = static_cast<float*>(c.aux(a[7], at::kFloat, {rows, m.rot / 2}));
      sin = static_cast<float*>(c.aux(a[8], at::kFloat, {rows, m.rot / 2}));
    } else if (a[7] != Py_None || a[8] != Py_None) {
      return PyLong_FromLong(-1);
    }
    auto* pq = static_cast<int32_t*>(c.aux(a[9], i32, {m.B, m.Nq}));
    auto* pk = static_cast<int32_t*>(c.aux(a[10], i32, {m.B, m.Nk}));
    auto* st = static_cast<int32_t*>(c.aux(a[11], i32, {4}));
    if (!here()) return PyLong_FromLong(-1);
    status = reinterpret_cast<decltype(&sparsepr_norm_rotate)>(p->fn)(
        &m, t[0], t[1], wq, wk, cos, sin, (int32_t)rows, pq, pk, t[2], t[3], st, stream());
  } else if (p->kind == Plan::MASKED) {
    const auto& m = *static_cast<const spr_masked_params*>(now);
    void* t[4];
    for (int i = 0; i < 4; ++i) t[i] = c.main(a[1 + i], p->main[i]);
    const at::Tensor* ws = c.workspace(a[5]);
    auto* k_len = static_cast<int32_t*>(c.aux(a[6], i32, {m.B}));
    auto* doc_q = static_cast<int32_t*>(c.aux(a[7], i32, {m.B, m.Nq}));
    auto* doc_k = static_cast<int32_t*>(c.aux(a[8], i32, {m.B, m.Nk}));
    auto* prefix = static_cast<int32_t*>(c.aux(a[9], i32, {m.B}));
    auto* slopes = static_cast<float*>(c.aux(a[10], at::kFloat, {m.Hq}));
    auto* lse = static_cast<float*>(c.aux(a[11], at::kFloat, {m.B, m.Hq, m.Nq}));
    auto* st = static_cast<int32_t*>(c.aux(a[12], i32, {4}));
    if (!doc_q != !doc_k || (prefix && !m.causal) || !here()) return PyLong_FromLong(-1);
    status = reinterpret_cast<decltype(&sparsepr_attend_masked)>(p->fn)(
        &m, t[0], t[1], t[2], k_len, doc_q, doc_k, prefix, slopes, t[3], lse, ws->data_ptr(),
        ws->nbytes(), st, stream());
  } else {
    const auto& m = *static_cast<const spr_project_params*>(now);
    void* t[3];
    for (int i = 0; i < 3; ++i) t[i] = c.main(a[1 + i], p->main[i]);
    const at::Tensor* ws = c.workspace(a[4]);
    const auto type = p->main[0].type;
    const int64_t M = (int64_t)m.Hy * m.dy;
    void *bias = c.aux(a[5], type, {M}), *gate = c.aux(a[6], type, {m.B, M});
    void* res = a[7] == Py_None ? nullptr : c.main(a[7], p->main[3].given ? p->main[3] : p->main[2]);
    auto* st = static_cast<int32_t*>(c.aux(a[8], i32, {4}));
    if (!here()) return PyLong_FromLong(-1);
    status = reinterpret_cast<decltype(&sparsepr_project)>(p->fn)(
        &m, t[0], t[1], bias, gate, res, t[2], ws->data_ptr(), ws->nbytes(), st, stream());
  }
  return PyLong_FromLong(status);
}

// What `f` returns, or `otherwise` where it throws.
template <typename F>
PyObject* guarded(F&& f, PyObject* (*otherwise)()) {
  try {
    return f();
  } catch (...) {
    PyErr_Clear();
    return otherwise();
  }
}
PyObject* plan(PyObject*, PyObject* args) {
  return guarded([&] { return make_plan(args); }, []() -> PyObject* { Py_RETURN_NONE; });
}
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&] { return make_call(a, n); }, [] { return PyLong_FromLong(-1); });
}

PyMethodDef METHODS[] = {
    {"plan", plan, METH_VARARGS, "The plan of a call with the given parameters and tensors."},
    {"call", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call)), METH_FASTCALL,
     "Make the call if the tensors fit the plan; -1 otherwise."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef MODULE = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, METHODS,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&MODULE); }
