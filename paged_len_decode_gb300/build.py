"""Build libvh.so in-tree from csrc/*.cu with nvcc for sm_103a, and the
CPython binding _vh_bind.so from csrc/bind.cpp.

Each translation unit compiles in parallel into _build/, then nvcc links a
shared library with the CUDA runtime linked statically (so the library loads
on a machine without a GPU; CUDA calls then report that no device exists).
The binding is host code against torch's C++ headers and links libvh.so.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libvh.so")
BIND = os.path.join(HERE, "_vh_bind.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--use_fast_math",
              "-Xptxas", "-O3"] + ARCH


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_dir() -> str:
    # found without importing torch: the compiler runs meanwhile
    import importlib.util

    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch not found")
    return list(spec.submodule_search_locations)[0]


def _bind_stamp() -> str:
    """What the binding is built against besides its sources: torch (found without
    importing it) and this Python."""
    d = _torch_dir()
    version = os.path.join(d, "version.py")
    with open(version) as f:
        return f"{d}\n{f.read()}\n{sys.version}\n{sysconfig.get_config_var('EXT_SUFFIX')}\n"


def _bind_stale(obj: str, deps: list[str], stamp: str) -> bool:
    """Whether the binding's object has to be compiled anew; `stamp` is the file
    that says what it was built against."""
    if _stale(obj, deps) or not os.path.exists(stamp):
        return True
    with open(stamp) as f:
        return f.read() != _bind_stamp()


def _compile_bind(src: str, obj: str, stamp: str) -> str:
    t = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    inc = [t, os.path.join(t, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], cuda]
    cmd = ["g++", "-O1", "-std=c++17", "-fPIC", "-fvisibility=hidden", *[f"-I{d}" for d in inc], "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(_bind_stamp())
    return r.stderr


def _link_bind(obj: str) -> None:
    libs = os.path.join(_torch_dir(), "lib")
    tmp = BIND + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-l:libvh.so", f"-L{libs}", "-ltorch_python",
                        "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                     + glob.glob(os.path.join(HERE, "..", "include", "*.h")))
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    bind_src, bind_obj = os.path.join(CSRC, "bind.cpp"), os.path.join(BUILD, "bind.o")
    bind_deps, stamp = [bind_src, os.path.join(HERE, "..", "include", "vh.h")], os.path.join(BUILD, "bind.stamp")

    def compile_one(src, obj):
        if src == bind_src:
            return _compile_bind(src, obj, stamp) if force or _bind_stale(obj, bind_deps, stamp) else ""
        if not force and not _stale(obj, [src] + headers):
            return ""
        cmd = [cc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return r.stderr

    jobs = [(bind_src, bind_obj), *zip(srcs, objs)]
    with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
        logs = list(ex.map(lambda so: compile_one(*so), jobs))
    if verbose:
        for log in logs:
            if log:
                sys.stderr.write(log)
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        r = subprocess.run([cc, "-shared", *ARCH, "-Xlinker", "-soname=libvh.so", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if force or _stale(BIND, [bind_obj, LIB]):
        _link_bind(bind_obj)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
