"""The compiled calls of the microscaled operators on pretended CUDA devices.

pysrc/mx_binding.cpp is compiled against stand-ins for CUDA's current device
and streams and for the library, which record what they are called with, so
that a machine without a GPU (or with one) can see on which device and stream a
call would launch.  Tensors are host memory that says it is on cuda:<n>."""

import importlib.machinery
import importlib.util
import os
import subprocess
import sysconfig

import torch

from weight_quantized_moe_gb300 import binding, build

HEADER = r"""
#pragma once
#include <c10/core/Device.h>
namespace fake { inline int current = 0; }
namespace c10::cuda {
inline c10::DeviceIndex current_device() { return (c10::DeviceIndex)fake::current; }
struct CUDAGuard {
  int before;
  explicit CUDAGuard(c10::Device d) : before(fake::current) { fake::current = d.index(); }
  ~CUDAGuard() { fake::current = before; }
  CUDAGuard(const CUDAGuard&) = delete;
  CUDAGuard& operator=(const CUDAGuard&) = delete;
};
struct OptionalCUDAGuard {
  int before = -1;
  void set_device(c10::Device d) {
    if (before < 0) before = fake::current;
    fake::current = d.index();
  }
  ~OptionalCUDAGuard() {
    if (before >= 0) fake::current = before;
  }
};
struct CUDAStream {
  int device;
  void* stream() const { return reinterpret_cast<void*>(intptr_t(100 + device)); }
};
inline CUDAStream getCurrentCUDAStream(c10::DeviceIndex d = -1) { return {d < 0 ? fake::current : d}; }
}  // namespace c10::cuda
"""

SOURCE = r"""
#include "mx_binding.cpp"
#include <vector>

static std::vector<std::pair<int, long>> g_calls;  // (current device, stream)
static int note(void* stream) {
  g_calls.emplace_back(fake::current, (long)reinterpret_cast<intptr_t>(stream));
  return MQ_OK;
}
extern "C" {
const char* mq_last_error_message(void) { return ""; }
int moe_quantize_mx(const void*, int, int64_t, int64_t, int64_t, int, uint8_t*, uint8_t*, void* st) { return note(st); }
int moe_dequantize_mx(const uint8_t*, const uint8_t*, int64_t, int64_t, int, void*, int, void* st) { return note(st); }
int moe_rmsnorm_mx(const void*, const void*, const void*, int, int, int, int, int64_t, int64_t, float, void*, void*,
                   int, uint8_t*, uint8_t*, void* st) { return note(st); }
size_t moe_mx_product_workspace(int64_t, int, int, int) { return 0; }
int moe_mx_product(const uint8_t*, const uint8_t*, int, int64_t, int, int, int, const uint8_t*, const uint8_t*,
                   const int32_t*, void*, int, void*, size_t, void* st) { return note(st); }
size_t moe_mx_forward_workspace(int, int, int, int, int, int) { return 0; }
int moe_mx_forward(const uint8_t*, const uint8_t*, int, int, int, int, int, int, const uint8_t*, const uint8_t*,
                   const uint8_t*, const uint8_t*, const float*, const int32_t*, void*, int, void*, size_t,
                   void* st) { return note(st); }
}

// (host tensor, device) -> the same memory, said to be on cuda:<device>
static PyObject* on_device(PyObject*, PyObject* args) {
  PyObject* o;
  int device;
  if (!PyArg_ParseTuple(args, "Oi", &o, &device)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  c10::Storage storage(c10::Storage::use_byte_size_t(), t.numel() * t.element_size(),
                       c10::DataPtr(t.data_ptr(), c10::Device(c10::DeviceType::CUDA, device)), nullptr, false);
  at::Tensor r = at::detail::make_tensor<c10::TensorImpl>(
      std::move(storage), c10::DispatchKeySet(c10::DispatchKey::CUDA), t.dtype());
  r.unsafeGetTensorImpl()->set_sizes_and_strides(t.sizes(), t.strides());
  return THPVariable_Wrap(r);
}
// the calls so far, and the device that is current now
static PyObject* calls(PyObject*, PyObject*) {
  PyObject* list = PyList_New(0);
  for (const auto& c : g_calls) {
    PyObject* p = Py_BuildValue("(il)", c.first, c.second);
    PyList_Append(list, p);
    Py_DECREF(p);
  }
  g_calls.clear();
  return Py_BuildValue("(Ni)", list, fake::current);
}
static PyMethodDef fake_methods[] = {{"on_device", on_device, METH_VARARGS, nullptr},
                                     {"calls", calls, METH_NOARGS, nullptr},
                                     {nullptr, nullptr, 0, nullptr}};
static PyModuleDef fake_module = {PyModuleDef_HEAD_INIT, "_mx_fake", nullptr, -1, fake_methods,
                                  nullptr, nullptr, nullptr, nullptr};
PyMODINIT_FUNC PyInit__mx_fake(void) { return PyModule_Create(&fake_module); }
"""


def _load(name, path):
    loader = importlib.machinery.ExtensionFileLoader(name, path)
    m = importlib.util.module_from_spec(importlib.util.spec_from_file_location(name, path, loader=loader))
    loader.exec_module(m)
    return m


def compile_fake(folder):
    """(the binding's compiled calls on the stand-ins, the stand-ins' own calls)."""
    for name in ("CUDAGuard.h", "CUDAStream.h"):
        path = os.path.join(folder, "c10", "cuda", name)
        os.makedirs(os.path.dirname(path), exist_ok=True)
        with open(path, "w") as f:
            f.write(HEADER if name == "CUDAGuard.h" else '#include "c10/cuda/CUDAGuard.h"\n')
    src, so = os.path.join(folder, "fake.cpp"), os.path.join(folder, "fake.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    dirs, lib_dir = build._torch_dirs()
    system = [*dirs, sysconfig.get_path("include")]
    r = subprocess.run(
        [build._cxx(), "-O0", "-std=c++17", "-fPIC", "-shared",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", folder,
         "-I", os.path.dirname(build.PYSRC), "-I", os.path.join(build.ROOT, "include"),
         *[a for d in system for a in ("-isystem", d)], src, "-o", so, "-L", lib_dir, "-ltorch_python",
         "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{lib_dir}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    calls, fake = _load("_mx_binding", so), _load("_mx_fake", so)
    calls.set_error_class(binding.MoeqError)
    return calls, fake
