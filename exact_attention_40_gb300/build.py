"""Builds libexattn.so in-tree with nvcc for sm_103a (no cmake, no torch), and
_binding.so, the compiled half of the Python binding, with g++ against the
installed torch's headers.

The translation units compile in parallel, then link into one shared
library next to this file.  Host code is plain C++17, so the same sources
build on x86-64 and aarch64 hosts.  The binding needs torch and Python's headers;
without them the library is built alone, which all but the binding's calls need.
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libexattn.so")
SOURCES = ["api.cu", "prefill.cu", "decode.cu", "norm.cu", "rope.cu", "backward.cu", "rope_axes.cu",
           "decode_fp4.cu", "cache_fp8.cu", "decode_fp8.cu"]
BINDING = os.path.join(HERE, "_binding.so")
BINDING_KEY = os.path.join(HERE, "_build", "binding.key")
HEADER = os.path.join(os.path.dirname(HERE), "include", "exattn.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _torch_dir():
    """Where torch is installed (found without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec is not None else None


def _python_include() -> str:
    return sysconfig.get_paths()["include"]


def _binding_lacks():
    """What the binding cannot be built without and is not here, or None."""
    if _torch_dir() is None:
        return "torch"
    for header in (os.path.join(_torch_dir(), "include", "ATen", "ATen.h"),
                   os.path.join(_python_include(), "Python.h")):
        if not os.path.exists(header):
            return header
    return None


def _binding_key() -> str:
    """The torch and the Python that a binding is built against."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f.read() + str(sysconfig.get_config_var("EXT_SUFFIX"))


def _newer(sources, target) -> bool:
    """Whether the target is missing or older than one of the sources."""
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in sources if os.path.exists(p))


def _lib_stale() -> bool:
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "binding.cpp"]
    return _newer(deps + [HEADER], LIB)


def _binding_stale() -> bool:
    if _binding_lacks() is not None:
        return False
    if _newer([os.path.join(CSRC, "binding.cpp"), HEADER], BINDING) or not os.path.exists(BINDING_KEY):
        return True
    with open(BINDING_KEY) as f:
        return f.read() != _binding_key()


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (what, r.stdout, r.stderr))
    return r


def build(force: bool = False, verbose: bool = False) -> str:
    lib, binding = force or _lib_stale(), _binding_lacks() is None and (force or _binding_stale())
    if force and not binding:
        sys.stderr.write("_binding.so is not built: %s is not installed\n" % _binding_lacks())
    objdir = os.path.dirname(BINDING_KEY)
    if lib or binding:
        os.makedirs(objdir, exist_ok=True)
    nvcc = _nvcc()

    def compile_binding():
        obj = os.path.join(objdir, "binding.o")
        cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
        torch = os.path.join(_torch_dir(), "include")
        dirs = [torch, os.path.join(torch, "torch/csrc/api/include"), _python_include(), cuda]
        _run(["g++", "-O2", "-std=c++17", "-fPIC"] + ["-I" + d for d in dirs]
             + ["-c", os.path.join(CSRC, "binding.cpp"), "-o", obj], "g++ for binding.cpp")
        return obj

    def compile_one(src):
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        r = _run([nvcc] + NVCC_FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj], "nvcc for " + src)
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding_obj = ex.submit(compile_binding) if binding else None
        objs = list(ex.map(compile_one, SOURCES)) if lib else []
    if lib:
        tmp = LIB + ".tmp%d" % os.getpid()
        _run([nvcc] + ARCH + ["-shared", "-o", tmp] + objs, "link of libexattn.so")
        os.replace(tmp, LIB)
    if binding:  # once the library is in place, whatever comes of this
        obj = binding_obj.result()
        # torch's own libraries are in the process before this one is imported
        tmp = BINDING + ".tmp%d" % os.getpid()
        _run(["g++", "-shared", "-o", tmp, obj, "-L" + os.path.dirname(LIB), "-l:libexattn.so", "-Wl,-rpath,$ORIGIN",
              "-L" + os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
              "-lc10_cuda"], "link of _binding.so")
        os.replace(tmp, BINDING)
        with open(BINDING_KEY, "w") as f:
            f.write(_binding_key())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
