"""Builds libmoe_gb300.so in-tree with nvcc for sm_103a (one translation unit
per .cu file, compiled in parallel, linked with the static CUDA runtime), and
_binding.so, the attention side's calls for this interpreter and its torch."""
from __future__ import annotations

import os
import platform
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build", platform.machine())
LIB = os.path.join(PKG, "libmoe_gb300.so")
BINDING = os.path.join(PKG, "_binding.so")
SOURCES = ["route.cu", "gemm.cu", "slice.cu", "mx.cu", "api.cu", "noalloc.cu", "qk_norm_rope.cu",
           "prefix_attention.cu", "linear.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, extra_flags=()) -> str:
    """Compile (when sources changed) and return the path of the library."""
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    headers.append(os.path.join(INCLUDE, "moe.h"))
    nvcc = _nvcc()
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if _stale(o, [s] + headers):
            jobs.append([nvcc, *ARCH, *FLAGS, *extra_flags, "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {cmd[-3]}")

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_binding_object, run)
        list(ex.map(run, jobs))
        binding_obj, binding_key, linked_with = binding.result()
    stamp = os.path.join(BUILD, "lib.stamp")
    if jobs or _stale(LIB, objs) or not os.path.exists(stamp):
        tmp = LIB + ".tmp"
        run([nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", *objs, "-o", tmp])
        os.replace(tmp, LIB)
        with open(stamp, "w") as f:
            f.write(platform.machine())
    _link(BINDING, binding_obj, binding_key, linked_with, run)
    return LIB


def _same(path: str, text: str) -> bool:
    if not os.path.exists(path):
        return False
    with open(path) as f:
        return f.read() == text


def _binding_object(run):
    """Compiles csrc/binding.cpp; -> (object, what it was compiled for, the
    linker's arguments)."""
    import torch
    at = os.path.dirname(torch.__file__)
    lib, inc_torch = os.path.join(at, "lib"), os.path.join(at, "include")
    key = f"{platform.machine()} {torch.__version__} {sys.version}"
    src, obj = os.path.join(CSRC, "binding.cpp"), os.path.join(BUILD, "binding.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    stamp = os.path.join(BUILD, "binding.compiled")
    if _stale(obj, [src, os.path.join(INCLUDE, "moe.h")]) or not _same(stamp, key):
        inc = [a for p in (inc_torch, os.path.join(inc_torch, "torch", "csrc", "api", "include"),
                           sysconfig.get_paths()["include"], INCLUDE, cuda) for a in ("-I", p)]
        run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *inc,
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-c", src, "-o", obj])
        with open(stamp, "w") as f:
            f.write(key)
    return obj, key, ["-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{lib}"]


def _link(target: str, obj: str, key: str, args, run) -> None:
    stamp = os.path.join(BUILD, "binding.stamp")
    if not _stale(target, [obj]) and _same(stamp, key):
        return
    tmp = target + ".tmp"
    run([os.environ.get("CXX", "g++"), "-shared", obj, "-o", tmp, "-L", PKG, "-l:libmoe_gb300.so", *args,
         "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, target)
    with open(stamp, "w") as f:
        f.write(key)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
