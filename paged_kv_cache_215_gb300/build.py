"""Build the CUDA library libpkv.so in-tree (paged_kv_cache_215_gb300/_build/).

Each .cu file is compiled by nvcc for sm_103a in parallel, the host C++ file by
g++, and the objects are linked into one shared library against the CUDA
runtime.  No CMake, no setuptools: one nvcc invocation per translation unit.
The module that checks torch tensors for the short calls (csrc/binding) is built
beside it against the installed torch, and again when that changes.  Without a torch
for CUDA and Python's headers it is left out: the C library needs neither.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
SO = os.path.join(BUILD, "libpkv.so")
BINDING = os.path.join(BUILD, "pkv_tensors.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _cuda_home() -> str:
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return os.environ.get("CUDA_HOME", "/usr/local/cuda")


def _sources():
    cus = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    cpps = sorted(glob.glob(os.path.join(CSRC, "*.cpp")))
    deps = cus + cpps + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return cus, cpps, deps


def _stale(deps, target=SO) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps + [__file__])


def _torch():
    """The installed torch's folder and version (without importing it), or None where
    the binding cannot be built: no torch, one without CUDA, or no Python headers."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    where = os.path.dirname(spec.origin)
    for needed in (os.path.join(where, "lib", "libc10_cuda.so"),
                   os.path.join(where, "include", "c10", "cuda", "CUDAStream.h"),
                   os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(needed):
            return None
    try:
        return where, importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:      # not installed as a package
        return where, where


def _binding_job():
    """(command that compiles the binding, its object), or None if it is up to date or
    cannot be built."""
    src = os.path.join(CSRC, "binding", "pkv_tensors.cpp")
    torch = _torch()
    if torch is None:
        return None
    where, version = torch
    stamp = BINDING + ".torch"
    built = open(stamp).read() if os.path.exists(stamp) else ""
    if built == version and not _stale([src, os.path.join(INCLUDE, "pkv.h")], BINDING):
        return None
    obj = os.path.join(BUILD, "pkv_tensors.cpp.o")
    inc = [INCLUDE, os.path.join(_cuda_home(), "include"), os.path.join(where, "include"),
           os.path.join(where, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
            *[x for i in inc for x in ("-isystem" if i != INCLUDE else "-I", i)],
            "-c", src, "-o", obj], obj


def _link_binding(obj):
    where, version = _torch()
    lib = os.path.join(where, "lib")
    _run(["g++", "-shared", "-o", BINDING + ".tmp", obj, "-L", BUILD, "-l:libpkv.so", "-L", lib,
          "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda",
          "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib])
    os.replace(BINDING + ".tmp", BINDING)
    with open(BINDING + ".torch", "w") as f:
        f.write(version)


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("build failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    return r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    cus, cpps, deps = _sources()
    os.makedirs(BUILD, exist_ok=True)
    binding = _binding_job()
    if not force and not _stale(deps):
        if binding:
            _run(binding[0])
            _link_binding(binding[1])
        return SO
    cuda = _cuda_home()
    nvcc = os.path.join(cuda, "bin", "nvcc")
    inc = ["-I", INCLUDE, "-I", CSRC, "-I", os.path.join(cuda, "include")]
    jobs = []
    for src in cus:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
               "-Xcompiler", "-fvisibility=hidden", *inc, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        jobs.append((cmd, obj))
    for src in cpps:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *inc, "-c", src,
               "-o", obj]
        jobs.append((cmd, obj))
    if binding:
        jobs.insert(0, binding)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        logs = list(ex.map(lambda j: _run(j[0]), jobs))
    if verbose:
        for l in logs:
            if l.strip():
                print(l)
    tmp = SO + ".tmp"
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *[j[1] for j in jobs if j is not binding],
          "-L", os.path.join(cuda, "lib64"), "-lcudart",
          "-Xlinker", "-rpath=" + os.path.join(cuda, "lib64")])
    os.replace(tmp, SO)
    if binding:
        _link_binding(binding[1])
    return SO


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
