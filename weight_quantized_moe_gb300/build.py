"""Build libmoeq.so (the C-ABI library) in-tree with nvcc for sm_103a, and
_mx_binding.so (the compiled Python calls of the microscaled operators).

Every ``csrc/*.cu`` is compiled to an object in parallel, then linked into
``weight_quantized_moe_gb300/libmoeq.so``; ``pysrc/mx_binding.cpp`` is compiled
beside them with the host compiler against torch's headers and linked to it.  No fast-math: the quantisers
rely on IEEE division and denormals.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoeq.so")
PYSRC = os.path.join(PKG, "pysrc", "mx_binding.cpp")
PYEXT = os.path.join(PKG, "_mx_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
              "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoeq.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [
        os.path.join(ROOT, "include", "moeq.h"), os.path.abspath(__file__)]


def _newer(made, sources) -> bool:
    if not os.path.exists(made):
        return False
    t = os.path.getmtime(made)
    return all(os.path.getmtime(p) <= t for p in sources)


def _library_up_to_date() -> bool:
    return _newer(LIB, _deps())


def _binding_stamp() -> str:
    """What a binding was compiled against: it fits no other torch or Python."""
    import torch
    return f"torch {torch.__version__} python {sysconfig.get_config_var('EXT_SUFFIX')}"


def _stamp_path() -> str:
    return os.path.join(BUILD, "mx_binding.stamp")


def _binding_up_to_date() -> bool:
    if not _newer(PYEXT, [PYSRC, os.path.join(ROOT, "include", "moeq.h"), os.path.abspath(__file__)]):
        return False
    try:
        with open(_stamp_path()) as f:
            return f.read() == _binding_stamp()
    except (OSError, ImportError):
        return False


def up_to_date() -> bool:
    return _library_up_to_date() and _binding_up_to_date()


def _cxx() -> str:
    for cand in (os.environ.get("CXX"), shutil.which("g++"), shutil.which("c++")):
        if cand:
            return cand
    raise RuntimeError("g++ not found: a C++ compiler is required to build _mx_binding.so")


def _torch_dirs():
    """(torch's include directories, torch's library directory)."""
    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    inc = os.path.join(base, "include")
    return ([inc, os.path.join(inc, "torch", "csrc", "api", "include")],
            os.path.join(base, "lib"))


def _run(cmd, what, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)


def _compile_binding() -> str:
    import torch
    obj = os.path.join(BUILD, "mx_binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    system = [*_torch_dirs()[0], cuda, sysconfig.get_path("include")]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    _run([_cxx(), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", os.path.join(ROOT, "include"),
          *[a for d in system for a in ("-isystem", d)], "-c", PYSRC, "-o", obj],
         "compiling mx_binding.cpp")
    return obj


def _link_binding(obj) -> None:
    lib_dir = _torch_dirs()[1]
    tmp = PYEXT + ".tmp"
    _run([_cxx(), "-shared", "-o", tmp, obj, "-L", PKG, "-lmoeq", "-L", lib_dir, "-ltorch_python",
          "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib_dir}"],
         "linking _mx_binding.so")
    os.replace(tmp, PYEXT)
    with open(_stamp_path(), "w") as f:
        f.write(_binding_stamp())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libmoeq.so and _mx_binding.so, whichever is out of date;
    returns the library's path.  The library needs nvcc only: it is linked before
    anything that is missing for the binding (a C++ compiler, torch) raises."""
    library = force or not _library_up_to_date()
    bind = force or not _binding_up_to_date()
    if not library and not bind:
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        _run(cmd, f"nvcc on {os.path.basename(src)}", verbose)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding) if bind else None
        if library:
            nvcc = _nvcc()
            objs = list(ex.map(compile_one, _sources()))
            tmp = LIB + ".tmp"
            _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], "link")
            os.replace(tmp, LIB)
        if bind:
            _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
