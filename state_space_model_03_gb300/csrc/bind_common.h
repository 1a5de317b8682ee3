// What the Python bindings share: argument checks, operands and errors.
#pragma once
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cstring>
#include <string>
#include <vector>

#include "ssfwd_packed.h"

namespace {

const char *(*g_text)(int);
PyObject *g_error;  // api.SSError

// A check that failed: the Python exception is set where it is caught.
struct Refusal {
  PyObject *type;
  std::string what;
};
[[noreturn]] void refuse(PyObject *type, std::string what) { throw Refusal{type, std::move(what)}; }

struct Status {
  int code;
};
void check(int status) {
  if (status != SS_OK) throw Status{status};
}

const at::Tensor *opt(PyObject *o, const char *name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor &need(PyObject *o, const char *name) {
  const at::Tensor *t = opt(o, name);
  if (!t) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return *t;
}
int dtype_of(const at::Tensor &t) {
  switch (t.scalar_type()) {
    case at::kFloat: return SS_F32;
    case at::kHalf: return SS_F16;
    case at::kBFloat16: return SS_BF16;
    default: return -1;
  }
}
const void *ptr(const at::Tensor *t) { return t && t->defined() ? t->data_ptr() : nullptr; }
const float *fptr(const at::Tensor *t) { return static_cast<const float *>(ptr(t)); }
const int32_t *iptr(const at::Tensor *t) { return static_cast<const int32_t *>(ptr(t)); }

// Operands, kept alive for the call where they had to be copied.
struct Held {
  at::Tensor t;
  const at::Tensor *get() const { return t.defined() ? &t : nullptr; }
};
Held rows(const at::Tensor *t) { return !t ? Held{} : Held{t->dim() == 0 || t->stride(-1) == 1 ? *t : t->contiguous()}; }
Held flat(const at::Tensor *t) { return !t ? Held{} : Held{t->contiguous()}; }

void on(const at::Tensor *t, const at::Tensor &x, const char *name) {
  if (t && t->device() != x.device()) refuse(PyExc_ValueError, std::string(name) + " must be on " + x.device().str());
}
void no_grad(std::initializer_list<const at::Tensor *> ts) {
  const bool backward = c10::GradMode::is_enabled();
  for (const at::Tensor *t : ts)
    if (t && ((backward && t->requires_grad()) || t->_fw_grad(0).defined()))
      refuse(PyExc_NotImplementedError, "this operator is forward only: no gradients and no tangents");
}
// A cache was updated in place: what autograd has saved of it is known to be old.
void changed(const at::Tensor *t) {
  if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}
Held int32(const at::Tensor *t, const char *name, int64_t n, const at::Tensor &x) {
  if (!t) return Held{};
  if (t->scalar_type() != at::kInt || t->dim() != 1 || t->size(0) != n)
    refuse(PyExc_TypeError, std::string(name) + " must be int32 (" + std::to_string(n) + ",)");
  on(t, x, name);
  return Held{t->contiguous()};
}
int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
bool flag(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v == 1;
}
void *stream_of(const at::Tensor &x) { return c10::cuda::getCurrentCUDAStream(x.get_device()).stream(); }

// The tables as the operators take them, in a bytes object.
struct Plan {
  ss_packed_tables t;
  int64_t device;
};
const Plan &plan_of(PyObject *o, const at::Tensor &x) {
  if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != (Py_ssize_t)sizeof(Plan)) refuse(PyExc_TypeError, "tables must be a RequestTables");
  const Plan &p = *reinterpret_cast<const Plan *>(PyBytes_AS_STRING(o));
  if (p.t.tokens != x.size(0) || p.device != x.get_device())
    refuse(PyExc_ValueError, "tables are of another batch: x must have num_tokens rows, on their device");
  return p;
}

template <typename F>
PyObject *guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  HANDLE_TH_ERRORS
  try {
    if (given != wanted) refuse(PyExc_TypeError, "wrong number of arguments");
    return f();
  } catch (const Refusal &r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const Status &s) {
    PyObject *e = PyObject_CallFunction(g_error, "is", s.code, g_text(s.code));
    if (e) {
      PyErr_SetObject(g_error, e);
      Py_DECREF(e);
    }
  }
  return nullptr;
  END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

}  // namespace
