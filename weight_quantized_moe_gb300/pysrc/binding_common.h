// What the compiled Python calls share: argument checks, output allocation, the
// tensors' device and stream, and the boundary that no C++ exception crosses.
#pragma once

#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include "moeq.h"

namespace {

PyObject* g_error_class = nullptr;  // binding.MoeqError

// Thrown once the Python error is set.
struct Raised {};

template <typename... Args>
[[noreturn]] void raise(PyObject* type, const char* fmt, Args... args) {
  PyErr_Format(type, fmt, args...);
  throw Raised();
}

void check(int status) {
  if (status == MQ_OK) return;
  PyObject* e = PyObject_CallFunction(g_error_class, "is", status, mq_last_error_message());
  if (e) {
    PyErr_SetObject(g_error_class, e);
    Py_DECREF(e);
  }
  throw Raised();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

void on_cuda(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be on a CUDA device", name);
}

long as_long(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

// MQ_DTYPE_* of a plain tensor; -1 for another type.
int dtype_code(at::ScalarType t) {
  return t == at::kBFloat16 ? MQ_DTYPE_BF16
         : t == at::kHalf   ? MQ_DTYPE_F16
         : t == at::kFloat  ? MQ_DTYPE_F32
                            : -1;
}

at::ScalarType scalar_type(long code) {
  return code == MQ_DTYPE_BF16 ? at::kBFloat16 : code == MQ_DTYPE_F16 ? at::kHalf : at::kFloat;
}

void same_device(const at::Tensor& t, const at::Tensor& first, const char* name) {
  if (t.get_device() != first.get_device())
    raise(PyExc_ValueError, "%s must be on cuda:%d", name, (int)first.get_device());
}

// A dense tensor of a given type, dims (< 0: any) and first's device.
const at::Tensor& dense(PyObject* o, at::ScalarType type, int dims, const at::Tensor& first,
                        const char* name) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type),
          c10::toString(t.scalar_type()));
  on_cuda(t, name);
  if (dims >= 0 && t.dim() != dims) raise(PyExc_ValueError, "%s must have %d dims", name, dims);
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
  same_device(t, first, name);
  return t;
}

// Elements between the rows of a tensor whose rows are dense and evenly spaced.
int64_t row_stride(const at::Tensor& t, const char* name) {
  const int64_t cols = t.size(-1);
  if (t.is_contiguous()) return cols;
  if (cols > 1 && t.stride(-1) != 1)
    raise(PyExc_ValueError, "%s: the elements of a row must be contiguous", name);
  int64_t stride = cols;
  bool first = true;
  int64_t expect = 0;  // stride that the next dim outwards has to have
  for (int64_t d = t.dim() - 2; d >= 0; --d) {
    if (t.size(d) == 1) continue;
    if (first) stride = t.stride(d);
    else if (t.stride(d) != expect)
      raise(PyExc_ValueError, "%s: the rows must be evenly spaced", name);
    first = false;
    expect = t.stride(d) * t.size(d);
  }
  return stride;
}

// The caller's output, checked, or a new one.
at::Tensor output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const at::Tensor& first,
                  const char* name) {
  if (o == Py_None) return at::empty(shape, first.options().dtype(type));
  const at::Tensor& t = dense(o, type, -1, first, name);
  if (t.sizes() != shape) raise(PyExc_ValueError, "%s has the wrong shape", name);
  return t;
}

// After a call that wrote to tensors of the caller (None: not given): their versions count, as
// with any in-place operation, so that a backward pass that saved one refuses to run.
void written(std::initializer_list<PyObject*> os) {
  for (PyObject* o : os)
    if (o != Py_None && !THPVariable_Unpack(o).is_inference())
      THPVariable_Unpack(o).unsafeGetTensorImpl()->bump_version();
}

// Makes the tensors' device current for the rest of a call: the library plans,
// launches and finds its status word on the current device.  (Where it is current
// already, as almost always, one look-up instead of a guard's two.)
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;  // that device's current stream
  explicit OnDevice(const at::Tensor& t) {
    if (c10::cuda::current_device() != t.get_device()) guard.set_device(t.device());
    stream = c10::cuda::getCurrentCUDAStream(t.get_device()).stream();
  }
};

uint8_t* bytes(const at::Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }

PyObject* wrap(const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  if (!o) throw Raised();
  return o;
}

PyObject* wrap_all(std::initializer_list<at::Tensor> ts) {  // (undefined: None)
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Raised();
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      throw Raised();
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

template <typename F>
int call(F&& f) {  // without the interpreter's lock: a full launch queue blocks
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

// A workspace of at least `need` bytes: the caller's, or a new one.
at::Tensor workspace(PyObject* o, size_t need, const at::Tensor& first) {
  if (o != Py_None) return dense(o, at::kByte, -1, first, "workspace");
  if (!need) return at::Tensor();
  return at::empty({(int64_t)need}, first.options().dtype(at::kByte));
}

void int_sizes(std::initializer_list<int64_t> sizes) {
  for (int64_t n : sizes)
    if (n > INT32_MAX) raise(PyExc_ValueError, "a size exceeds 32 bits");
}

PyObject* set_error_class(PyObject* const* a) {
  Py_XDECREF(g_error_class);
  g_error_class = Py_NewRef(a[0]);
  Py_RETURN_NONE;
}

// No C++ exception leaves a call.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
constexpr PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)),
          METH_FASTCALL, nullptr};
}

}  // namespace
