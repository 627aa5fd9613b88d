"""Build libskgemm.so in-tree with nvcc for sm_103a, and the torch binding
_skg_torch.so next to it.

Each .cu under csrc/ is one translation unit; they compile in parallel
(one -gencode, no cmake) and link into a shared library with the CUDA
runtime linked statically, so loading the library needs no GPU. The binding
(csrc/skg_torch.cpp, host code) compiles against the installed torch at the
same time and links to libskgemm.so beside it; without torch the library alone is
built.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libskgemm.so")
BINDING = os.path.join(PKG, "_skg_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libskgemm.so")
    return nvcc


def _newest_header() -> float:
    hdrs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(h) for h in hdrs)


def _stale(target: str, objs) -> bool:
    """Whether target is missing or older than one of the objects it is linked of."""
    return not os.path.exists(target) or \
        os.path.getmtime(target) < max(os.path.getmtime(o) for o in objs)


def _read(path: str) -> str:
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def torch_dir():
    """The folder of the installed torch; None without one (the library needs none, and the
    binding is then not built)."""
    try:
        spec = importlib.util.find_spec("torch")
    except (ImportError, ValueError):
        return None
    return os.path.dirname(spec.origin) if spec is not None and spec.origin else None


def _binding_job(force: bool, torch_dir: str):
    """(compile command or None, object, link command) of the torch binding; the object's
    name carries torch's version, whose headers it is compiled against."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        version = "".join(c if c.isalnum() else "_" for c in
                          next(line for line in f if line.startswith("__version__")))
    src = os.path.join(CSRC, "skg_torch.cpp")
    obj = os.path.join(BUILD, f"skg_torch_{version}.o")
    fresh = os.path.exists(obj) and os.path.getmtime(obj) >= max(
        os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "skgemm.h")))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I",
           os.path.join(torch_dir, "include"), "-I",
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), "-I", cuda,
           "-I", sysconfig.get_paths()["include"], "-c", src, "-o", obj]
    lib = os.path.join(torch_dir, "lib")
    link = ["g++", "-shared", obj, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
            "-ltorch", "-ltorch_python", "-L", PKG, "-l:libskgemm.so", "-Wl,-rpath,$ORIGIN",
            f"-Wl,-rpath,{lib}"]
    return (cmd if force or not fresh else None), obj, link


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile (incrementally) and link libskgemm.so and, where torch is installed, the
    binding; returns the library's path."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_time = _newest_header()
    jobs = []
    objs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or not os.path.exists(obj) or \
                os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time):
            jobs.append([nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj])

    def run(cmd):
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            print(res.stdout + res.stderr)
        return res

    torch = torch_dir()
    if torch:
        binding, binding_obj, binding_link = _binding_job(force, torch)
        if binding:
            jobs.insert(0, binding)  # the longest one
    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            list(ex.map(run, jobs))
    if _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    if torch:
        # The link line names the object and torch's libraries: kept beside the objects, it
        # shows a binding that was linked for another torch.
        line, linked = " ".join(binding_link), os.path.join(BUILD, "skg_torch.linked")
        if _stale(BINDING, [binding_obj]) or _read(linked) != line:
            tmp = BINDING + f".tmp{os.getpid()}"
            run([*binding_link, "-o", tmp])
            os.replace(tmp, BINDING)
            with open(linked, "w") as f:
                f.write(line)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
