"""Build libkvo.so in-tree for sm_103a with nvcc (parallel compile, then link), and the native Python binding of the
serving calls, _kvo_binding.so, with g++ against this interpreter's torch.  The library alone needs neither torch nor
its headers: the binding is left out where torch is not installed, or with ``binding=False`` (--no-binding)."""
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
STAMP = os.path.join(BUILD, "binding.stamp")          # the torch and the interpreter that binding.o was compiled against
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


def _torch_dir():
    """The folder of the installed torch, or None."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _binding_object(torch: str) -> str:
    """Compile csrc/binding.cpp (host code only); returns the object file."""
    src, obj = os.path.join(SRC, "binding.cpp"), os.path.join(BUILD, "binding.o")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    with open(os.path.join(torch, "version.py")) as f:
        against = f"{torch}\n{sysconfig.get_config_var('SOABI')}\n{f.read()}"
    stamp = ""
    if os.path.exists(STAMP):
        with open(STAMP) as f:
            stamp = f.read()
    if stamp != against or _newer(obj, [src, os.path.join(ROOT, "include", "kvo.h")]):
        if os.path.exists(STAMP):
            os.remove(STAMP)
        inc = [os.path.join(ROOT, "include"), os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
        r = subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", *[f"-I{i}" for i in inc], "-c", src, "-o", obj],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for {src} (libkvo.so needs no torch headers: build(binding=False)):\n{r.stderr}")
        with open(STAMP, "w") as f:
            f.write(against)
    return obj


def _link_binding(obj: str, torch: str) -> None:
    if not _newer(BINDING, [obj, STAMP, LIB]):
        return
    # libkvo.so has no soname, so that a C program linked with its path starts without an rpath; the binding finds it beside itself
    r = subprocess.run(["g++", "-shared", "-o", BINDING, obj, f"-L{PKG}", "-l:libkvo.so", "-Wl,-rpath,$ORIGIN", f"-L{torch}/lib",
                        "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking the binding failed:\n{r.stderr}")


def build(verbose: bool = False, ptxas_info: bool = False, binding: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    torch = _torch_dir() if binding else None
    if binding and torch is None:
        sys.stderr.write("no torch: libkvo.so is built without its Python binding\n")
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
        obj = ex.submit(_binding_object, torch) if torch else None
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
    if obj:
        _link_binding(obj.result(), torch)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_info="--ptxas" in sys.argv, binding="--no-binding" not in sys.argv))
