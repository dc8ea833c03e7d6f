"""The compiled calls of the 16-bit operators on pretended CUDA devices, as
mx_fake_device.py has the microscaled ones: the stand-ins for the library record the
device and stream of each call, and how the weights were described."""

import os
import subprocess
import sysconfig

import torch

import mx_fake_device as mx
from weight_quantized_moe_gb300 import binding, build

LIBRARY = r"""
#include "grouped_binding.cpp"
#include <vector>

static std::vector<std::pair<int, long>> g_calls;  // (current device, stream)
static long g_weights[3];
static int note(void* stream) {
  g_calls.emplace_back(fake::current, (long)reinterpret_cast<intptr_t>(stream));
  return MQ_OK;
}
extern "C" {
const char* mq_last_error_message(void) { return ""; }
size_t moe_grouped_product_workspace(int64_t, int, int, int) { return 0; }
size_t moe_grouped_product_grad_workspace(int64_t, int, int, int) { return 0; }
int moe_grouped_product(const void*, int64_t, int, int64_t, int, int, int, const void*, int64_t ws, int64_t we, int tr,
                        const int32_t*, void*, int, void*, size_t, void* st) {
  g_weights[0] = ws, g_weights[1] = we, g_weights[2] = tr;
  return note(st);
}
int moe_grouped_product_grad(const void*, int64_t, const void*, int64_t, int, int64_t, int, int, int, const void*,
                             int64_t, int64_t, int, const int32_t*, void*, void*, int, void*, size_t, void* st) {
  return note(st);
}
size_t moe_lora_product_workspace(int64_t, int, int, int, int, int) { return 0; }
int moe_lora_product(const void*, int64_t, int, int64_t, int, int, int, int, int, const void*, const void*,
                     const int32_t*, const int32_t*, const float*, const void*, int64_t bs, void*, int64_t os, int,
                     void*, size_t, void* st) {
  g_weights[0] = bs, g_weights[1] = os;
  return note(st);
}
}
"""

WEIGHTS = r"""
static PyObject* weights(PyObject*, PyObject*) {
  return Py_BuildValue("(lll)", g_weights[0], g_weights[1], g_weights[2]);
}
"""


def compile_fake(folder):
    """(the compiled calls on the stand-ins, the stand-ins' own calls)."""
    for name in ("CUDAGuard.h", "CUDAStream.h"):
        path = os.path.join(folder, "c10", "cuda", name)
        os.makedirs(os.path.dirname(path), exist_ok=True)
        with open(path, "w") as f:
            f.write(mx.HEADER if name == "CUDAGuard.h" else '#include "c10/cuda/CUDAGuard.h"\n')
    own = mx.SOURCE[mx.SOURCE.index("// (host tensor, device)"):]
    own = own.replace("static PyMethodDef fake_methods[] = {",
                      WEIGHTS + 'static PyMethodDef fake_methods[] = {{"weights", weights, METH_NOARGS, nullptr},\n')
    src, so = os.path.join(folder, "fake.cpp"), os.path.join(folder, "fake.so")
    with open(src, "w") as f:
        f.write(LIBRARY + own)
    dirs, lib_dir = build._torch_dirs()
    system = [*dirs, sysconfig.get_path("include")]
    r = subprocess.run(
        [build._cxx(), "-O0", "-std=c++17", "-fPIC", "-shared",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", folder,
         "-I", os.path.dirname(build.PYSRC), "-I", os.path.join(build.ROOT, "include"),
         *[a for d in system for a in ("-isystem", d)], src, "-o", so, "-L", lib_dir, "-ltorch_python",
         "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{lib_dir}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    calls, fake = mx._load("_grouped_binding", so), mx._load("_mx_fake", so)
    calls.set_error_class(binding.MoeqError)
    return calls, fake
