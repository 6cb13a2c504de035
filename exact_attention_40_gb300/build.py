"""Builds libexattn.so in-tree with nvcc for sm_103a (no cmake, no torch), and
_binding.so, the compiled half of the Python binding, with g++ against the
installed torch's headers.

The translation units compile in parallel, then link into one shared
library next to this file.  Host code is plain C++17, so the same sources
build on x86-64 and aarch64 hosts.
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
           "decode_fp4.cu"]
BINDING = os.path.join(HERE, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _torch_dir():
    """Where torch is installed (found without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec is not None else None


def _stale() -> bool:
    if not os.path.exists(LIB) or (_torch_dir() is not None and not os.path.exists(BINDING)):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "exattn.h"))
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    nvcc = _nvcc()

    torch_dir = _torch_dir()

    def compile_binding():
        obj = os.path.join(objdir, "binding.o")
        cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
        dirs = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include/torch/csrc/api/include"),
                sysconfig.get_paths()["include"], cuda]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC"] + ["-I" + d for d in dirs]
        cmd += ["-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("g++ failed for binding.cpp:\n%s\n%s" % (r.stdout, r.stderr))
        return obj

    def compile_one(src):
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [nvcc] + NVCC_FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding) if torch_dir is not None else None
        objs = list(ex.map(compile_one, SOURCES))
        binding_obj = binding.result() if binding is not None else None
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    if binding_obj is not None:
        # torch's own libraries are in the process before this one is imported
        tmp = BINDING + ".tmp%d" % os.getpid()
        cmd = ["g++", "-shared", "-o", tmp, binding_obj, "-L" + HERE, "-l:libexattn.so", "-Wl,-rpath,$ORIGIN",
               "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
        os.replace(tmp, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
