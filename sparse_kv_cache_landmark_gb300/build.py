"""Build libkvo.so in-tree for sm_103a with nvcc (parallel compile, then link), and the native Python binding of the
serving calls, _kvo_binding.so, with g++ against this interpreter's torch."""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkvo.so")
BINDING = os.path.join(PKG, "_kvo_binding.so")
NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def sources():
    return sorted(os.path.join(SRC, f) for f in os.listdir(SRC) if f.endswith(".cu"))


def _newer(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_object() -> str:
    """Compile csrc/binding.cpp (host code only); returns the object file."""
    src, obj = os.path.join(SRC, "binding.cpp"), os.path.join(BUILD, "binding.o")
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    if _newer(obj, [src, os.path.join(ROOT, "include", "kvo.h"), os.path.join(torch, "version.py")]):
        inc = [os.path.join(ROOT, "include"), os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
        r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", *[f"-I{i}" for i in inc], "-c", src, "-o", obj],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for {src}:\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    if not _newer(BINDING, [obj, LIB]):
        return
    torch = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "lib")
    # libkvo.so has no soname, so that a C program linked with its path starts without an rpath; the binding finds it beside itself
    r = subprocess.run(["g++", "-shared", "-o", BINDING, obj, f"-L{PKG}", "-l:libkvo.so", "-Wl,-rpath,$ORIGIN", f"-L{torch}",
                        "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking the binding failed:\n{r.stderr}")


def build(verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(SRC, f) for f in os.listdir(SRC) if f.endswith(".cuh")]
    headers.append(os.path.join(ROOT, "include", "kvo.h"))
    srcs = sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        if not (ptxas_info or _newer(obj, [src] + headers)):
            return ""
        cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if ptxas_info:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return r.stderr

    with ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as ex:
        binding = ex.submit(_binding_object)
        logs = list(ex.map(compile_one, zip(srcs, objs)))
    if verbose or ptxas_info:
        for lg in logs:
            if lg:
                sys.stderr.write(lg)
    if _newer(LIB, objs):
        cmd = [NVCC, *ARCH, "-shared", "-cudart", "shared", "-o", LIB, *objs,
               "-Xlinker", "-rpath,/usr/local/cuda/lib64"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
    _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="--ptxas" in sys.argv))
