"""Build in-tree: libpa_decode.so, nvcc for sm_103a, one object per .cu in parallel; and
_bind.so, the compiled binding of the operators that serving loops call per token."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpa_decode.so")
BIND = os.path.join(PKG, "_bind.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                     "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa_decode.so")
    return path


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return hs + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _text(path: str) -> str:
    with open(path) as f:
        return f.read()


def _run(cmd, what: str):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_bind(force: bool) -> str:
    """csrc/pa_bind.cpp -> an object named after the torch it is compiled against."""
    import torch
    src = os.path.join(CSRC, "pa_bind.cpp")
    obj = os.path.join(BUILD, f"pa_bind-{torch.__version__}.o")
    if force or _stale(obj, [src] + _headers()):
        inc = os.path.join(os.path.dirname(torch.__file__), "include")
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
        _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
              "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
              "-isystem", cuda, "-isystem", sysconfig.get_paths()["include"], "-c", src, "-o", obj], "g++")
    return obj


def _link_bind(obj: str):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libpa_decode.so", "-Wl,-rpath,$ORIGIN", "-L", libs,
          "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"], "link of _bind.so")
    os.replace(tmp, BIND)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile csrc, link libpa_decode.so and _bind.so; returns the former's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    headers = _headers()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    todo = [(s, o) for s, o in zip(srcs, objs) if force or _stale(o, [s] + headers)]
    exe = nvcc()

    def compile_one(so):
        s, o = so
        cmd = [exe, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {s}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return o

    with cf.ThreadPoolExecutor(max_workers=min(len(todo), os.cpu_count() or 4) + 1) as ex:
        bind = ex.submit(_compile_bind, force)
        list(ex.map(compile_one, todo))
        bind_obj = bind.result()
    if force or todo or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [exe, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    # Which torch's object _bind.so holds: another torch's may be older than the link.
    linked, name = os.path.join(BUILD, "bind-linked"), os.path.basename(bind_obj)
    if force or _stale(BIND, [bind_obj]) or not os.path.exists(linked) or _text(linked) != name:
        _link_bind(bind_obj)
        with open(linked, "w") as f:
            f.write(name)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
