"""Build libnsgb300.so in-tree with nvcc for sm_103a, and the Python binding of
its training-step operators (_training.so) against the installed torch.

Each translation unit compiles in parallel into ``_build/``; the shared
library lands next to this file. Rebuilds only when a source or header is
newer than the library, or the binding was built against another torch or
Python. No cmake, one -gencode.
"""

from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libnsgb300.so")
BINDING = os.path.join(PKG, "_training.so")
SOURCES = ["planner.cpp", "api.cu", "runtime.cu", "route.cu", "ns_bf16.cu", "ns_fp32.cu", "pipeline.cu",
           "gemm.cu", "gemm2sm.cu", "gemm32.cu", "prologue.cu", "pack.cu", "small.cu", "noalloc.cu",
           "moe.cu", "qk_rope.cu", "distill.cu", "grad_norm.cu", "block_norm.cu", "moe_few.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libnsgb300.so")
    return cand


def _deps() -> list:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "nsgb300.h"))
    files.append(os.path.abspath(__file__))
    return files


def _torch_dir():
    """Where torch is installed, without importing it; None if it is not, or
    not for CUDA: the library needs no torch, and no such torch has a use for
    the binding."""
    spec = importlib.util.find_spec("torch")
    where = os.path.dirname(spec.origin) if spec and spec.origin else None
    return where if where and os.path.exists(os.path.join(where, "lib", "libc10_cuda.so")) else None


def _binding_of() -> str:
    """What a binding is compiled against: this torch and this Python."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{_torch_dir()}\n{f.read()}"


def _stamp() -> str:
    return os.path.join(BUILD, "binding.txt")


def _stale() -> bool:
    made = [LIB] + ([BINDING, _stamp()] if _torch_dir() else [])
    if not all(os.path.exists(f) for f in made):
        return True
    if _torch_dir():
        with open(_stamp()) as f:
            if f.read() != _binding_of():
                return True
    made = made[:2]
    t = min(os.path.getmtime(f) for f in made)
    return any(os.path.getmtime(f) > t for f in _deps())


def _run(cmd, what) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _compile_binding(nvcc: str) -> str:
    """binding.cpp alone is host code on torch's headers."""
    torch_dir, obj = _torch_dir(), os.path.join(BUILD, "binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], cuda]
    _run(["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE] + [x for d in inc for x in ("-isystem", d)]
         + ["-c", os.path.join(CSRC, "binding.cpp"), "-o", obj], "g++ on binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    tmp = BINDING + ".tmp"
    _run(["g++", "-shared", obj, "-o", tmp, "-L", PKG, "-l:libnsgb300.so", "-Wl,-rpath,$ORIGIN",
          "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], "link of _training.so")
    os.replace(tmp, BINDING)
    with open(_stamp(), "w") as f:
        f.write(_binding_of())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if needed) and return the path of libnsgb300.so."""
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    common = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC] + ARCH

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cu"):
            cmd += ["-Xptxas", "-v"] if verbose else []
        return obj, _run(cmd, f"nvcc on {src}")

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding, nvcc) if _torch_dir() else None
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            if log.strip():
                print(log)
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-shared"] + ARCH + ["-o", tmp] + [o for o, _ in results]
    _run(cmd, "link")
    os.replace(tmp, LIB)
    if binding:
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
