"""Build the CUDA library in-tree: csrc/*.cu -> _build/libmoe_router.so, and
the Python extension that ops.py calls: csrc/ops_binding.cpp -> _build/_moe_ops.so.

nvcc compiles each translation unit for sm_103a in parallel, then links a
shared library against the shared CUDA runtime.  g++ compiles the extension
against the installed PyTorch and links it to that library.  Rebuilds only
when a source or header is newer than the results.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmoe_router.so")
BINDING_SRC = os.path.join(CSRC, "ops_binding.cpp")
BINDING = os.path.join(BUILD, "_moe_ops.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-I", INCLUDE]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + [BINDING_SRC] + glob.glob(os.path.join(CSRC, "*.h")) +
            glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BINDING)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(d) <= t for d in _deps())


def _binding_commands():
    """Compile and link commands of the extension, and the file they make."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    obj = os.path.join(BUILD, "ops_binding.o")
    abi = "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi())
    compile_cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", abi,
                   "-I", INCLUDE, "-I", os.path.join(root, "include"),
                   "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                   "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
                   "-c", BINDING_SRC, "-o", obj]
    tmp = BINDING + ".%d.tmp" % os.getpid()
    link_cmd = ["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-l:libmoe_router.so",
                "-Wl,-rpath,$ORIGIN", "-L", os.path.join(root, "lib"), "-ltorch_python",
                "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10"]
    return compile_cmd, link_cmd, tmp


def _run(cmd, what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s%s" % (what, r.stdout, r.stderr))
    return r.stdout + r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = _sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(src_obj):
        src, obj = src_obj
        log = _run([cc] + NVCC_FLAGS + ["-c", src, "-o", obj], "nvcc on %s" % src)
        if verbose:
            print(log)
        return obj

    compile_binding, link_binding, tmp_binding = _binding_commands()
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        binding = ex.submit(_run, compile_binding, "g++ on %s" % BINDING_SRC)
        list(ex.map(compile_one, zip(srcs, objs)))
        binding.result()
    tmp = LIB + ".%d.tmp" % os.getpid()
    _run([cc] + ARCH + ["-shared", "-cudart", "shared", "-Xlinker", "-soname=libmoe_router.so",
                        "-o", tmp] + objs, "link")
    os.replace(tmp, LIB)
    _run(link_binding, "link of the extension")
    os.replace(tmp_binding, BINDING)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
