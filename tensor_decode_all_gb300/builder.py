"""Build libtda_ar.so from csrc/*.cu for sm_103a, in tree.

Each translation unit is compiled by nvcc in parallel, then linked into one
shared library next to this file (git-ignored); the operators' extension
module (csrc/ops_binding.cpp) is compiled beside them and linked against it.  The CUDA runtime is linked
statically, so the library needs only the CUDA driver at run time.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtda_ar.so")
BINDING = os.path.join(PKG, "_ops_binding.so")      # the extension module of ops.py

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              # IEEE fp32 adds: no fast-math, no flush-to-zero, no contraction
              "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-fmad=false",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                        if f.endswith((".h", ".cuh", ".cpp"))] + [os.path.join(INCLUDE, f) for f in sorted(os.listdir(INCLUDE))]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with ThreadPoolExecutor(max_workers=min(9, (os.cpu_count() or 1) + 1)) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(compile_one, sources()))
        binding_obj = binding.result()
    if verbose or ptxas_verbose:
        for obj, log in results:
            if log.strip():
                sys.stderr.write(f"--- {os.path.basename(obj)}\n{log}")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lrt", "-ldl", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding_obj)
    return LIB


def _torch_dir() -> str:
    """Where torch is installed, without importing it."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found: the operators' binding cannot be built")
    return list(spec.submodule_search_locations)[0]


def _cxx() -> str:
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no C++ compiler: the operators' binding cannot be built")
    return cxx


def _run(what: str, cmd) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")


def _compile_binding() -> str:
    """csrc/ops_binding.cpp against this interpreter's and torch's headers."""
    t, obj = _torch_dir(), os.path.join(BUILD, "ops_binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    _run("the operators' binding", [
        _cxx(), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", os.path.join(CSRC, "ops_binding.cpp"), "-o", obj,
        f"-I{INCLUDE}", f"-I{sysconfig.get_path('include')}", f"-isystem{t}/include",
        f"-isystem{t}/include/torch/csrc/api/include", f"-isystem{cuda}"])
    return obj


def _link_binding(obj: str) -> None:
    t, tmp = os.path.join(_torch_dir(), "lib"), BINDING + f".tmp{os.getpid()}"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "lib64")
    _run("link of the operators' binding", [
        _cxx(), "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:libtda_ar.so", f"-L{t}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
        "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-L{cuda}", "-lcudart", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{t}"])
    os.replace(tmp, BINDING)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="--ptxas-v" in sys.argv))
